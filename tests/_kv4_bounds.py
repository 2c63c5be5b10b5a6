"""Attention over a 4-bit cache in 64 bits with a bound per output in which each token counts
by its own weight, so that tokens of no weight loosen nothing (those of _kv4.attend take
one logit error, the largest, for all).

u = 2^-24, a rounding to nearest of fp32; an addition counts 2 u (a tensor core truncates).
  logit i: at most 140 roundings of terms whose magnitudes sum to zmass_i, and eight more of
    sums that hold the running maximum M, |M| <= max(|z_i|, |z_top|) + 10 (M is raised to a
    tile's maximum whenever a token exceeds it by more than that):
      dz_i = 280 u zmass_i + 8 u (max(|z_i|, |z_top|) + 10)
  weight p_i: r_i = e^dz_i - 1 + 2^-20 (exponential, product with the step, the two 11-bit
    parts, the factors that join states: each below 2^-22).
    A weight below 2^-124 of the largest may become 0: r_i = 1 (p = 2^(z - M) is flushed
    below 2^-126, and M is at most one above the largest logit).
  The parts' last place is 2^-24 (f16), where the largest weight p s seen so far stands at
    2^7 or above, and a factor of p s may be subnormal, with 2^-26 in the same units: 1.5
    2^-25 / 2^7 of it per token, times |c - 7.5| <= 7.5:
      floor_g = count 11.25 2^-32 max_i p_i s_ig
  sums over `count` tokens: chains of count / 8 + 64 additions, ch = 2 u (count / 8 + 64).
  With a_i = |c - 7.5| s + |m + 7.5 s| the magnitude that token i adds to an output (p
  normalised), and P = sum p_i r_i + ch:
    |d out| <= 1.25 (sum p_i (r_i + ch) a_i + floor_g + |out| P)     (P < 0.1)
    |d lse| <= 1.25 P + 4 u (|lse| + 1)
"""
import numpy as np

import _kv4 as kv

U = 2.0 ** -24


def attend_row(qb, k, v, rec, tok, scale):
    """As _kv4.attend_row: out, lse in 64 bits and their bounds for one KV head."""
    G = qb.shape[0]
    if len(tok) == 0:
        return np.zeros((G, 128)), np.full(G, -np.inf), np.zeros((G, 128)), np.zeros(G)
    q = kv.bf16_val(qb).astype(np.float64)
    kc, km = kv.parts(k[tok], rec[tok, :4])
    vc, vm = kv.parts(v[tok], rec[tok, 4:])
    vs = np.repeat(kv.bf16_val(rec[tok, 4::2]).astype(np.float64), 64, -1)  # [n][128]
    scale = float(np.float32(scale))
    z = q @ (kc + km).T * scale
    zmass = np.abs(q) @ (kc + np.abs(km)).T * abs(scale)
    top = z.max(-1, keepdims=True)
    with np.errstate(under="ignore"):
        p = np.exp(z - top)
    l = p.sum(-1, keepdims=True)
    p /= l
    out, lse = p @ (vc + vm), (top + np.log(l))[:, 0]
    dz = 280 * U * zmass + 8 * U * (np.maximum(np.abs(z), np.abs(top)) + 10)
    pr = p * (np.expm1(np.minimum(dz, 600)) + 2.0 ** -20 + (p * l < 2.0 ** -124))
    ch = 2 * U * (len(tok) / 8 + 64)
    P = pr.sum(-1) + ch
    assert P.max() < 0.1, "the case says nothing"
    a = np.abs(vc - 7.5 * vs) + np.abs(vm + 7.5 * vs)
    floor = len(tok) * 11.25 * 2.0 ** -32 * np.stack([(p[g][:, None] * vs).max(0) for g in range(G)])
    return (out, lse, 1.25 * ((pr + ch * p) @ a + floor + np.abs(out) * P[:, None]),
            1.25 * P + 4 * U * (np.abs(lse) + 1))


def attend(qb, k, v, rec, toks, scale):
    """All rows, as _kv4.attend."""
    B, hq = qb.shape[:2]
    hkv = k.shape[1]
    G = hq // hkv
    res = [np.zeros((B, hq, 128)), np.zeros((B, hq)), np.zeros((B, hq, 128)), np.zeros((B, hq))]
    for b in range(B):
        for h in range(hkv):
            r = attend_row(qb[b, h * G:(h + 1) * G], k[b, h], v[b, h], rec[b, h],
                           np.asarray(toks[b * hkv + h], np.int64), scale)
            for to, x in zip(res, r):
                to[b, h * G:(h + 1) * G] = x
    return res


def check(out, lse, ref, tight=2.0 ** -8):
    """Outputs and lse within their bounds, which are at most `tight` of the largest output
    of each row's group of 64 channels (a bound near the output would pass anything) or
    2^-100, what is as good as 0."""
    ro, rl, bo, bl = ref
    g = lambda x: x.reshape(*x.shape[:-1], 2, 64).max(-1)  # noqa: E731
    assert np.all(g(bo) <= np.maximum(tight * g(np.abs(ro)), 2.0 ** -100)), (g(bo) / np.maximum(g(np.abs(ro)), 1e-300)).max()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    over = np.abs(out - ro) - bo
    assert over.max() <= 0, (over.max(), (np.abs(out - ro) / np.maximum(bo, 1e-300)).max())
    assert np.all(np.abs(lse - rl) <= bl), (np.abs(lse - rl) / bl).max()
