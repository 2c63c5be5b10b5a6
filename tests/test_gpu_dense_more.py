"""GPU tests of the operators around the bf16 cache beyond their values one by one: the
precision that single tokens are given, every token's part in long rows, and the operators
together with the sparse step, the 4-bit cache and one workspace."""
import math

import pytest
import torch

from _dense import D, F32, HALF, attention, check, norm_rope, visible
from test_gpu_dense import SCALE, check_prefix, check_window, i32, normal, run_prefix, run_window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_decode_gb300 import build as b
    b.build()
    import top_sparse_decode_gb300 as m
    m.lib()
    return m


def check_norm(out, ref, parts, what):
    """The 2-norm of out's error, over that of rounding the result alone.  Roundings are
    independent, so their squares add.  A weight of two parts is off by 2^-16 of itself at
    most, a 128th of what the result's own rounding may be: 1.0001, and 1.02 leaves room for
    the fp32 sums.  A weight of one part is rounded as the result is: sqrt(2)."""
    base = float((ref.bfloat16().double() - ref).norm())
    ratio = float((out.double() - ref).norm()) / base
    assert ratio <= (1.02 if parts == 2 else 1.6), (what, ratio)


@pytest.mark.parametrize("fallback", [False, True])
@pytest.mark.parametrize("G,n", [(1, 3000), (4, 500), (8, 9000), (2, 40000)])
def test_single_token_precision(sd, G, n, fallback):
    """Single tokens' weights have 16 bits: out's error is that of its own rounding; so have the
    weights of a sequence's own tokens.  Many tokens' weights and a prefix's have 8."""
    prev = sd.sd_set_fallback_paths(fallback)
    try:
        B, hkv = 4, 4
        for m, parts in ((1, 2), (5, 1)):
            q, K, V, out, lse = run_window(sd, B, hkv, G, n, n, m, n - m, None, None, n, 0)
            p = torch.arange(n - m, n, device="cuda")
            see = visible(p, n, n, 0, "cuda")
            z = torch.einsum("bhgtd,bhnd->bhgtn", q.double().unflatten(1, (hkv, G)), K.double())
            w = torch.softmax((z * SCALE).masked_fill(~see, -math.inf), -1)
            ref = torch.einsum("bhgtn,bhnd->bhgtd", w, V.double()).flatten(1, 2)
            check_norm(out, ref, parts, f"m = {m}")
        q, Kp, Vp, K, V, out, lse = run_prefix(sd, B, hkv, G, 0, 0, n, n, None)
        z = torch.einsum("bhgd,bhnd->bhgn", q.double().unflatten(1, (hkv, G)), K.double())
        ref = torch.einsum("bhgn,bhnd->bhgd", torch.softmax(z * SCALE, -1), V.double())
        check_norm(out, ref.flatten(1, 2), 2, "own tokens")
        q, Kp, Vp, K, V, out, lse = run_prefix(sd, B, hkv, G, n, n, 0, 0, None)
        z = torch.einsum("bhgd,hnd->bhgn", q.double().unflatten(1, (hkv, G)), Kp.double())
        ref = torch.einsum("bhgn,hnd->bhgd", torch.softmax(z * SCALE, -1), Vp.double())
        check_norm(out, ref.flatten(1, 2), 1, "prefix")
    finally:
        sd.sd_set_fallback_paths(prev)


def apart(V):
    """Each token alone in its channel of every 128."""
    n = V.shape[-2]
    V[:] = 0.0
    V[..., torch.arange(n, device="cuda"), torch.arange(n, device="cuda") % D] = 1.0


@pytest.mark.parametrize("case", [
    (1, 1, 4, 9000, 9000, 1, 8999, None, None, 7000, 130),
    (1, 1, 4, 9000, 9000, 700, 8300, None, None, 5000, 200),
    (1, 2, 1, 6000, 6000, 2000, 4000, None, [1777], 3333, 77),
    (2, 1, 8, 7000, 7000, 13, 6900, [0, 87], None, 7000, 0),
    (1, 8, 2, 5000, 5000, 5000, 0, None, None, 4100, 1),
], ids=range(5))
def test_every_token_counts(sd, case):
    """Values that set tokens apart under nearly equal weights: a channel of out is the sum of
    1 / 70 of the row's tokens at most, of which none may be missing, and none doubled (1 / 70
    is more than the two roundings of 2^-8 that the bound holds)."""
    check_window(case, run_window(sd, *case, scale=1e-3, prep=lambda q, K, V: apart(V)),
                 scale=1e-3, some=80)


@pytest.mark.parametrize("case", [(3, 2, 4, 8765, 8800, 100, 128, [100, 0, 37]),
                                  (40, 1, 8, 5003, 5003, 0, 0, None),
                                  (2, 1, 1, 0, 0, 8001, 8001, [8001, 8000])], ids=range(3))
def test_every_token_of_a_prefix_counts(sd, case):
    """The same for prefixes: with queries this small the weights are nearly equal."""
    def prep(q, Kp, Vp, K, V):
        q *= 1e-2
        pad = Vp[:, case[3]:].clone()
        apart(Vp)
        Vp[:, case[3]:] = pad
        if V is not None:
            own = V.clone()
            apart(V)
            V[~torch.isfinite(own.float())] = math.inf  # behind a sequence's end, as before
    check_prefix(case, run_prefix(sd, *case, prep=prep))


@pytest.mark.parametrize("kind", ["planes", "quest"])
def test_prompt_then_sparse_steps(sd, kind):
    """A prompt through norm, rotation and window attention into the cache; its keys indexed;
    then tokens one at a time: written, appended to the index, selected from and attended.
    The index is that of the cache as it stands, and every result the 64-bit attention's over
    what was selected."""
    from top_sparse_decode_gb300.pipeline import DecodeStep, StepConfig, build_index
    B, hkv, G, cap, m = 2, 2, 4, 704, 600
    hq = hkv * G
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    w = torch.ones(D, device="cuda")
    rope = sd.make_rope(freq, w, w)
    K, V = (torch.zeros((B, hkv, cap, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def write(m, at, seed):
        x = normal((B, m, hq + 2 * hkv, D), seed).transpose(1, 2)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        qo = torch.zeros((B, hq, m, D), dtype=torch.bfloat16, device="cuda")
        sd.sd_qk_norm_rope(sd.make_shape(B, hq, hkv, cap), rope, q, qo, k, v, K, V, m, first=at)
        return qo
    q = write(m, 0, 1)
    shape = sd.make_shape(B, hq, hkv, m, D, cap)
    out, lse = torch.zeros_like(q), torch.zeros((B, hq, m), device="cuda")
    ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, m, 256, 4)),
                     dtype=torch.uint8, device="cuda")
    sd.sd_window_attend(shape, q, K, V, m, 256, 4, SCALE, out, lse, ws)
    check_window((B, hkv, G, m, cap, m, 0, None, None, 256, 4), (q, K, V, out, lse), some=80)

    sel = dict(k=64, sink=4, local=32) if kind == "planes" else dict(k=8, sink=0, local=1)
    kid = sd.SD_IDX_PLANES if kind == "planes" else sd.SD_IDX_MINMAX
    sigma2 = torch.rand((hkv, D), device="cuda")
    index = build_index(StepConfig(kid, B, hq, hkv, m, n_cap=cap, **sel), K)
    bufs = (index["planes"], index["scales"]) if kind == "planes" else (index["summ"], None)
    for n in range(m + 1, m + 42):
        q = write(1, n - 1, n)[:, :, 0].contiguous()
        sd.sd_append_index(kid, sd.make_shape(B, hq, hkv, n, D, cap), n - 1, K, None, *bufs)
        if n % 8 and n != m + 1:
            continue
        cfg = StepConfig(kid, B, hq, hkv, n, n_cap=cap, **sel)
        step = DecodeStep(cfg, K, V, index, sigma2=sigma2)
        fresh = DecodeStep(cfg, K, V, build_index(cfg, K), sigma2=sigma2)
        step.run(q)
        fresh.run(q)
        torch.cuda.synchronize()
        assert torch.equal(step.count, fresh.count)
        for b in range(B):
            for h in range(hkv):
                r = b * hkv + h
                at = step.idx[r, :step.count[r]].long()
                assert torch.equal(at, fresh.idx[r, :len(at)].long())
                assert len(torch.unique(at)) == len(at) and int(at.max()) < n
                see = torch.ones((G, len(at)), dtype=torch.bool, device="cuda")
                o, e, tol, ltol = attention(q[b, h * G:(h + 1) * G], K[b, h, at], V[b, h, at],
                                            see, SCALE)
                check(step.out[b, h * G:(h + 1) * G], o, tol, "out")
                check(step.lse[b, h * G:(h + 1) * G], e, ltol, "lse")


def test_rows_on_the_way_to_the_4_bit_cache(sd):
    """Rows normed and rotated into a buffer of their own, turned by their places in the
    sequence, and written to the 4-bit cache: the same codes as by way of the bf16 cache."""
    B, hkv, G, n, m = 2, 2, 4, 300, 70
    hq = hkv * G
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    w = torch.ones(D, device="cuda")
    rope = sd.make_rope(freq, w, w)
    shape, buf = sd.make_shape(B, hq, hkv, n), sd.make_shape(B, hq, hkv, m)
    pos, length = i32([17, 230]), i32([70, 33])
    x = normal((B, m, hq + 2 * hkv, D), 3).transpose(1, 2)
    q, k, v = x.split([hq, hkv, hkv], dim=1)
    caches = [torch.zeros((B, hkv, t, D), dtype=torch.bfloat16, device="cuda")
              for t in (n, n, m, m)]
    outs = [torch.zeros((B, hq, m, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sd.sd_qk_norm_rope(shape, rope, q, outs[0], k, v, *caches[:2], m, pos=pos, length=length)
    sd.sd_qk_norm_rope(buf, rope, q, outs[1], k, v, *caches[2:], m, length=length, rotary=pos)
    assert torch.equal(*outs) and outs[0].abs().max() > 0
    a, b = sd.Kv4Cache(B, hkv, n), sd.Kv4Cache(B, hkv, n)
    sd.sd_kv4_write(shape, b, *caches[2:], m, pos=pos, length=length)
    for s, (at, l) in enumerate(((17, 70), (230, 33))):
        assert torch.equal(caches[0][s, :, at:at + l], caches[2][s, :, :l])
    sd.sd_kv4_write(shape, a, *caches[:2], n)
    for s, (at, l) in enumerate(((17, 70), (230, 33))):
        for x, y in ((a.k, b.k), (a.v, b.v), (a.scale, b.scale)):
            assert torch.equal(x[s, :, at:at + l], y[s, :, at:at + l])


def test_answers_over_a_document(sd):
    """One workspace, as large as the largest call needs, through a document's prompt in an odd
    chunk and a long one, and steps of several answers over it: each token normed, rotated by
    its place behind the document, written and attended."""
    B, hkv, G, p, n, window = 3, 2, 4, 901, 24, 901
    hq = hkv * G
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    w = torch.ones(D, device="cuda")
    rope = sd.make_rope(freq, w, w)
    doc, own = sd.make_shape(1, hq, hkv, p), sd.make_shape(B, hq, hkv, n)
    need = [sd.sd_window_attend_workspace_size(doc, m, window) for m in (33, 868)]
    need.append(sd.sd_prefix_attend_workspace_size(own, p))
    ws = torch.empty(max(16, *need), dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    Kp, Vp = torch.zeros((1, hkv, p, D), **bf), torch.zeros((1, hkv, p, D), **bf)
    K, V = torch.zeros((B, hkv, n, D), **bf), torch.zeros((B, hkv, n, D), **bf)
    at = 0
    for m in (33, 868):
        x = normal((1, m, hq + 2 * hkv, D), m).transpose(1, 2)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        qo, out = torch.zeros((1, hq, m, D), **bf), torch.zeros((1, hq, m, D), **bf)
        lse = torch.zeros((1, hq, m), device="cuda")
        sd.sd_qk_norm_rope(doc, rope, q, qo, k, v, Kp, Vp, m, first=at)
        sd.sd_window_attend(doc, qo, Kp, Vp, m, window, 0, SCALE, out, lse, ws, first=at)
        check_window((1, hkv, G, p, p, m, at, None, None, window, 0), (qo, Kp, Vp, out, lse),
                     some=60)
        at += m
    lens = i32([0, 5, 11])
    K[1, :, :5], V[1, :, :5] = normal((hkv, 5, D), 70), normal((hkv, 5, D), 71)
    K[2, :, :11], V[2, :, :11] = normal((hkv, 11, D), 72), normal((hkv, 11, D), 73)
    for step in range(6):
        x = normal((B, 1, hq + 2 * hkv, D), 80 + step).transpose(1, 2)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        qo = torch.zeros((B, hq, 1, D), **bf)
        sd.sd_qk_norm_rope(own, rope, q, qo, k, v, K, V, 1, pos=lens, rotary=lens + p)
        for b in range(B):
            r = lens[b:b + 1] + p
            kr = norm_rope(k[b], w, 1e-6, r, freq, 128, False)
            got = K[b, :, int(lens[b])].double()[:, None]
            assert ((got - kr).abs() <= HALF * kr.abs() + 256 * F32 * 16).all()
        lens += 1
        out, lse = torch.zeros((B, hq, D), **bf), torch.zeros((B, hq), device="cuda")
        sd.sd_prefix_attend(own, qo, Kp, Vp, p, K, V, SCALE, out, lse, ws, end=lens)
        check_prefix((B, hkv, G, p, p, n, n, lens.tolist()),
                     (qo[:, :, 0], Kp[0], Vp[0], K, V, out, lse))
    sd.sd_device_status()
