"""64-bit forms of the operators around the bf16 cache (sd_qk_norm_rope, sd_window_attend,
sd_prefix_attend), and how far a result may be from them."""
import math

import torch

D = 128
HALF = torch.finfo(torch.bfloat16).eps / 2  # 2^-8: one rounding to bf16
F32 = torch.finfo(torch.float32).eps / 2    # 2^-24


def visible(p, n, window, sink, device):
    """[queries][n]: what queries at positions p see."""
    i = torch.arange(n, device=device)
    p = p[:, None]
    return (i <= p) & ((i < sink) | (i > p - window))


def attention(q, K, V, see, scale):
    """(out, lse, tolerance of out, tolerance of lse) of q [rows][128] over K, V [n][128]; see
    bool [rows][n].  Tokens that no row sees are left out, and a row's unseen tokens count
    as absent whatever they hold."""
    q, K, V = q.double(), K.double(), V.double()
    out = torch.zeros_like(q)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(q)
    ltol = torch.zeros_like(lse)
    if not see.shape[1]:
        return out, lse, tol, ltol
    sets, which = torch.unique(see, dim=0, return_inverse=True)
    for s in range(sets.shape[0]):
        at = sets[s].nonzero()[:, 0]
        if not len(at):
            continue
        rows = (which == s).nonzero()[:, 0]
        k, v = K[at], V[at]
        z = (q[rows] @ k.T) * scale
        lse[rows] = torch.logsumexp(z, -1)
        w = torch.exp(z - lse[rows, None])
        out[rows] = w @ v
        # a score is a sum of 128 exact products in fp32, then scaled: off by 2^-24 for every
        # addition, of the sum of their sizes (and as much again for exp2's argument)
        zerr = 2 * (D + 4) * F32 * ((q[rows].abs() @ k.abs().T) * scale).amax(-1)
        # a sum over the tokens; exp2.approx and the factors of a raised maximum: 2^-21
        serr = len(at) * F32 + 2.0 ** -21
        size = w @ v.abs()
        # each weight rounded to bf16, the result too
        tol[rows] = HALF * (size + out[rows].abs()) + 2 * (zerr + serr)[:, None] * size + 1e-30
        # log2 and its factor, of the value itself
        ltol[rows] = zerr + serr + 4 * F32 * lse[rows].abs() + 2.0 ** -20
    return out, lse, tol, ltol


def check(got, ref, tol, what):
    got = got.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities"
    ok = ~nan & ~inf
    bad = (got - ref).abs()[ok] - tol[ok]
    if bad.numel():
        assert bad.max() <= 0, f"{what}: {bad.max():.3e} over its tolerance"


def norm_rope(x, weight, eps, pos, inv_freq, rot, pairs):
    """x [..., tokens, 128] at positions pos [tokens], in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if rot:
        a = pos.double()[:, None] * inv_freq
        c, s = torch.cos(a), torch.sin(a)
        one = torch.arange(rot // 2, device=x.device) * (2 if pairs else 1)
        two = one + (1 if pairs else rot // 2)
        u, v = x[..., one], x[..., two]
        x = x.clone()
        x[..., one], x[..., two] = u * c - v * s, v * c + u * s
    return x


def norm_rope_tol(ref, x, weight, eps, pos, inv_freq, rot, pairs):
    """One rounding to bf16, and fp32 arithmetic: 128 squares summed, rsqrt, two products, a
    sine and cosine of 2^-22 and their two products, of the sizes that a pair mixes."""
    size = norm_rope(x.double().abs(), weight if weight is None else weight.abs(), eps, pos,
                     torch.zeros_like(inv_freq) if rot else inv_freq, rot, pairs).abs()
    if rot:
        one = torch.arange(rot // 2, device=x.device) * (2 if pairs else 1)
        two = one + (1 if pairs else rot // 2)
        both = size[..., one] + size[..., two]
        size = size.clone()
        size[..., one], size[..., two] = both, both
    # the angle's own rounding: 64 bits of position * inv_freq in turns
    turn = float(pos.double().abs().max()) * 2.0 ** -51 if rot and pos.numel() else 0.0
    return HALF * ref.abs() + (64 * F32 + turn) * size + 1e-38
