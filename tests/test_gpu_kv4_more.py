"""GPU tests of the 4-bit K/V cache beyond the ordinary sizes and values: calls that are longer
than the cache, values and queries at the ends of their range with the bounds of _kv4_bounds.py,
ranges and selections that the kernel before writes, calls captured first, every step."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _kv4 as kv
import _kv4_bounds as kb
from _helpers import dev, host

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module")
def sd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_sparse_decode_gb300 import build as b
    b.build()
    import top_sparse_decode_gb300 as m
    m.lib()
    return m


def bits(t):
    return host(t.contiguous().view(torch.int16), np.uint16)


@pytest.mark.parametrize("with_length", [False, True])
def test_move_longer_than_the_cache(sd, with_length):
    """The largest m (2^31 - 1, a broadcast token) with nearly all of it in front of the cache,
    in it, or behind it: the tokens that have a place are moved, and only they."""
    rng = np.random.default_rng(3)
    B, h, n, m = 4, 2, 64, 2 ** 31 - 1
    K, V = kv.tokens(rng, (B, h, 1)), kv.tokens(rng, (B, h, 1))
    ek, ev, er = kv.encode(K, V)
    pos = np.array([-(m - 40), -(m - 3), 5, -m], np.int32)
    length = np.full(B, m, np.int32) if with_length else None
    c = sd.Kv4Cache(B, h, n)
    shp = sd.make_shape(B, h, h, n)
    wide = [dev(x).view(torch.bfloat16).expand(B, h, m, 128) for x in (K, V)]
    sd.sd_kv4_write(shp, c, *wide, m, pos=dev(pos), length=None if length is None else dev(length))
    torch.cuda.synchronize()
    for got, e in ((host(c.k, np.uint8), ek), (host(c.v, np.uint8), ev), (bits(c.scale), er)):
        for b, (lo, hi) in enumerate(((0, 40), (0, 3), (5, n), (0, 0))):
            want = np.zeros((h, n, e.shape[-1]), e.dtype)
            want[:, lo:hi] = e[b]
            assert np.array_equal(got[b], want), b


def test_read_in_front_of_the_cache(sd):
    """A read whose positions are all but seven in front of the cache."""
    rng = np.random.default_rng(4)
    n, m = 32, 1 << 20
    K, V = kv.tokens(rng, (1, 1, n)), kv.tokens(rng, (1, 1, n))
    k, v, rec = kv.encode(K, V)
    c = sd.Kv4Cache(1, 1, n, k=dev(k), v=dev(v), scale=dev(rec))
    out = torch.full((2, 1, 1, m, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    sd.sd_kv4_read(sd.make_shape(1, 1, 1, n), c, out[0], out[1], m,
                   pos=dev(np.array([7 - m], np.int32)))
    torch.cuda.synchronize()
    assert bool((out[:, :, :, :m - 7] == 7.0).all())
    for i, x in enumerate((kv.read(k, rec[..., :4]), kv.read(v, rec[..., 4:]))):
        assert np.array_equal(bits(out[i, 0, 0, m - 7:]), x[0, 0, :7])


@pytest.fixture(params=[False, True], ids=["chosen", "stream"])
def path(sd, request):
    """The kernel the library chooses, then the streaming one for every size."""
    before = sd.sd_set_fallback_paths(request.param)
    yield
    sd.sd_set_fallback_paths(before)


def attend_both(sd, q, k, v, rec, scale):
    """Dense attention and attention over all tokens listed in turn: [(out, lse)] x 2."""
    B, h, n = k.shape[:3]
    hq = q.shape[1]
    shp = sd.make_shape(B, hq, h, n)
    c = sd.Kv4Cache(B, h, n, k=dev(k), v=dev(v), scale=dev(rec))
    ws = torch.full((max(sd.sd_kv4_attend_workspace_size(shp),
                         sd.sd_kv4_gather_attend_workspace_size(shp, n)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    idx = dev(np.tile(np.arange(n, dtype=np.int32), (B * h, 1)))
    cnt = dev(np.full(B * h, n, np.int32))
    res = []
    for gather in (False, True):
        out = torch.full((B, hq, 128), 9.0, device="cuda")
        lse = torch.full((B, hq), 9.0, device="cuda")
        if gather:
            sd.sd_kv4_gather_attend(shp, dev(q), c, idx, n, cnt, n, scale, out, lse, ws)
        else:
            sd.sd_kv4_attend(shp, dev(q), c, scale, out, lse, ws)
        torch.cuda.synchronize()
        res.append((host(out, np.float32), host(lse, np.float32)))
    return res


def check_both(sd, q, k, v, rec, scale, tight=2.0 ** -8):
    B, h, n = k.shape[:3]
    ref = kb.attend(q, k, v, rec, [np.arange(n)] * (B * h), scale)
    for out, lse in attend_both(sd, q, k, v, rec, scale):
        kb.check(out, lse, ref, tight)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("below", [20, 60, 83, 300])
@pytest.mark.parametrize("wide", [1e10, 1e30, 1e38])
def test_wide_values_of_little_weight(sd, path, G, below, wide):
    """A group of values that is constant in every token, but for one token of a wide range
    whose logit is far below the others': first, in the middle, last, or the only one of its
    tile's second half.  What it adds is tiny or 0, and never NaN."""
    rng = np.random.default_rng(int(below) + G)
    B, h, n = 5, 1, 333
    qf = rng.standard_normal((B, 1, 128)) + 0.05 * rng.standard_normal((B, h * G, 128))
    K = 0.3 * rng.standard_normal((B, h, n, 128))
    V = rng.standard_normal((B, h, n, 128))
    V[:, :, :, 64:] = np.array([0, 2.5, 0, -1, 0]).reshape(B, 1, 1, 1)
    for b, at in enumerate((0, 100, n - 1, 20, 31)):
        base = qf[b].mean(0)
        K[b, :, at] = -below / SCALE / (base @ base) * base
        V[b, :, at] = rng.uniform(-1, 1, 128) * wide
    q = kv.bf16_bits(qf.astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K.astype(np.float32)), kv.bf16_bits(V.astype(np.float32)))
    check_both(sd, q, k, v, rec, SCALE, tight=2.0 ** -6)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("wide", [100, 113, 120, 126])
def test_wide_keys(sd, path, G, wide):
    """Keys of a range of 2^wide, tiny queries and a small scale: ordinary logits of factors
    whose products in another order pass the fp32 range."""
    rng = np.random.default_rng(wide + G)
    B, h, n = 2, 2, 333
    qf = rng.uniform(-1, 1, (B, h * G, 128)) * 2.0 ** (27 - wide)
    K = rng.uniform(-1, 1, (B, h, n, 128)) * 2.0 ** wide
    V = rng.standard_normal((B, h, n, 128))
    q = kv.bf16_bits(qf.astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K.astype(np.float32)), kv.bf16_bits(V.astype(np.float32)))
    check_both(sd, q, k, v, rec, SCALE * 2.0 ** -24, tight=2.0 ** -6)


@pytest.mark.parametrize("n,mc", [(300, 64), (4096, 700)])
def test_ranges_written_by_the_kernel_before(sd, n, mc):
    """begin, end, count and idx come from the kernel just before the attention (at sizes that
    take the cluster kernel, which starts while that one runs) and change from pass to pass;
    eagerly and in a graph."""
    rng = np.random.default_rng(n)
    B, h, G = 3, 4, 4
    shp = sd.make_shape(B, h * G, h, n)
    q = kv.tokens(rng, (B, h * G), spread=False)
    k, v, rec = kv.encode(kv.tokens(rng, (B, h, n)), kv.tokens(rng, (B, h, n)))
    c = sd.Kv4Cache(B, h, n, k=dev(k), v=dev(v), scale=dev(rec))
    passes = []
    for _ in range(4):
        begin = rng.integers(0, n // 2, B).astype(np.int32)
        end = (begin + rng.integers(1, n // 2, B)).astype(np.int32)
        idx = rng.integers(0, n, (B * h, mc)).astype(np.int32)
        cnt = rng.integers(1, mc + 1, B * h).astype(np.int32)
        dense = [np.arange(begin[b], end[b]) for b in range(B) for _ in range(h)]
        passes.append(([dev(x) for x in (begin, end, idx, cnt)],
                       kv.attend(q, k, v, rec, dense, SCALE),
                       kv.attend(q, k, v, rec, [idx[r, :cnt[r]] for r in range(B * h)], SCALE)))
    feed = [torch.zeros_like(x) for x in passes[0][0]]
    now = [torch.zeros_like(x) for x in feed]
    dq = dev(q)
    outs = [torch.zeros((B, h * G, 128), device="cuda") for _ in range(2)]
    lses = [torch.zeros((B, h * G), device="cuda") for _ in range(2)]
    ws = torch.empty(max(sd.sd_kv4_attend_workspace_size(shp),
                         sd.sd_kv4_gather_attend_workspace_size(shp, mc)), dtype=torch.uint8,
                     device="cuda")

    def work():
        torch._foreach_copy_(now[:2], feed[:2])
        sd.sd_kv4_attend(shp, dq, c, SCALE, outs[0], lses[0], ws, begin=now[0], end=now[1])
        torch.add(feed[2], 0, out=now[2])
        torch.add(feed[3], 0, out=now[3])
        sd.sd_kv4_gather_attend(shp, dq, c, now[2], mc, now[3], mc, SCALE, outs[1], lses[1], ws)

    def check(i):
        torch.cuda.synchronize()
        for j in range(2):
            kv.check(host(outs[j], np.float32), host(lses[j], np.float32), passes[i][1 + j])

    for i in (0, 1, 2, 3, 1):
        for to, x in zip(feed, passes[i][0]):
            to.copy_(x)
        torch.cuda._sleep(200000)
        work()
        check(i)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for i in (2, 0, 3, 1):
        for to, x in zip(feed, passes[i][0]):
            to.copy_(x)
        graph.replay()
        check(i)


FIRST = """
import torch, top_sparse_decode_gb300 as sd
B, h, G, n = 2, 2, 4, {n}
shp, c = sd.make_shape(B, h * G, h, n), sd.Kv4Cache(B, h, n)
x = torch.randn((B, h, n, 128), device="cuda").bfloat16()
q = torch.randn((B, h * G, 128), device="cuda").bfloat16()
out, lse = torch.zeros((B, h * G, 128), device="cuda"), torch.zeros((B, h * G), device="cuda")
ws = torch.empty(sd.sd_kv4_attend_workspace_size(shp), dtype=torch.uint8, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sd.sd_kv4_write(shp, c, x, x, n)
    sd.sd_kv4_attend(shp, q, c, 0.08, out, lse, ws)
graph.replay()
torch.cuda.synchronize()
got = out.clone(), lse.clone()
sd.sd_kv4_attend(shp, q, c, 0.08, out, lse, ws)
torch.cuda.synchronize()
assert torch.equal(got[0], out) and torch.equal(got[1], lse) and bool((out != 0).any())
print("captured first")
"""


@pytest.mark.parametrize("n", [500, 40000])
def test_first_calls_captured(sd, n):
    """The library's very first calls are made inside a capture (what it asks the device once
    it asks there)."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(n=n)], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("small", [0, -40, -60])
def test_small_values_after_wide_ones(sd, path, G, small):
    """The first tile's values have a range of 2^100 and its logits lie 400 below those of
    all that follow, whose values are of size 2^small: a warp that has met the wide ones
    weighs the others as exactly as any."""
    rng = np.random.default_rng(G)
    B, h, n = 20, 8, 1000  # several tiles a warp with either kernel
    some = 2
    qf = rng.standard_normal((B, h, 1, 128)) + 0.05 * rng.standard_normal((B, h, G, 128))
    K = 0.3 * rng.standard_normal((B, h, n, 128)).astype(np.float32)
    V = rng.standard_normal((B, h, n, 128)).astype(np.float32) * np.float32(2.0 ** small)
    base = qf.mean(2)
    K[:, :, :32] = (-400 / SCALE / (base * base).sum(-1, keepdims=True) * base)[:, :, None]
    V[:, :, :32] = rng.uniform(-1, 1, (B, h, 32, 128)) * 2.0 ** 100
    q = kv.bf16_bits(qf.reshape(B, h * G, 128).astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K), kv.bf16_bits(V))
    ref = kb.attend(q[:some], k[:some], v[:some], rec[:some], [np.arange(n)] * (some * h), SCALE)
    for out, lse in attend_both(sd, q, k, v, rec, SCALE):
        kb.check(out[:some], lse[:some], ref, tight=2.0 ** -6)
        assert np.isfinite(out).all()


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("below", [10, 20, 28])
def test_wide_queries(sd, path, G, below):
    """Query channels of up to `below` powers of two under the head's largest, with a key that
    shows only them: exact all the same (the keys are 0 and their group's minimum in the
    large channels, so that a logit holds nothing else)."""
    rng = np.random.default_rng(below + G)
    B, h, n = 2, 2, 333
    big = np.arange(128) % 16 == 3
    qf = np.where(big, 1.5, rng.uniform(1, 2, (B, h * G, 128)) * 2.0 ** -below)
    K = np.where(big, 0, rng.uniform(0, 4, (B, h, n, 128)))
    V = rng.standard_normal((B, h, n, 128))
    q = kv.bf16_bits(qf.astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K.astype(np.float32)), kv.bf16_bits(V.astype(np.float32)))
    assert not kv.bf16_val(rec[..., 1:4:2]).any()  # the minima
    check_both(sd, q, k, v, rec, 2.0 ** (below - 4), tight=2.0 ** -7)


@pytest.mark.parametrize("G", [4, 8])
def test_huge_values_of_no_weight(sd, path, G):
    """Ordinary tokens, and three of enormous values and a weight of 0 at the front."""
    rng = np.random.default_rng(G)
    B, h, n = 2, 2, 900
    qf = np.repeat(rng.standard_normal((B, h, 128)), G, 1)
    K, V = rng.standard_normal((2, B, h, n, 128))
    K[:, :, :3] = -40 * qf[:, ::G, None]
    V[:, :, :3] *= 1e30
    q = kv.bf16_bits(qf.astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K.astype(np.float32)), kv.bf16_bits(V.astype(np.float32)))
    check_both(sd, q, k, v, rec, SCALE, tight=2.0 ** -6)


@pytest.mark.parametrize("G", [4, 8])
def test_long_flat_tail(sd, G):
    """One token of a wide step that carries half of the mass, then thousands of equal ones
    that carry the rest, in rows that a warp works on alone: the smallest weights that count
    against a large one (their 22 bits end at 2^-25 / 2^7 of it)."""
    g = torch.Generator(device="cuda").manual_seed(G)
    B, h, n = 400, 8, 4096      # rows in plenty for the streaming kernel
    some = [0, 1, 133, B - 1]
    c = sd.Kv4Cache(B, h, n)
    shp = sd.make_shape(B, h * G, h, n)
    base = torch.randn(128, device="cuda", generator=g)
    first = base * (math.log(n) / SCALE / float(base @ base))  # logit log(n), the others 0
    for t in range(0, n, 512):
        V = torch.randn((B, h, 512, 128), device="cuda", generator=g)
        K = torch.zeros_like(V)
        if t == 0:
            K[:, :, 0] = first
            V[:, :, 0] *= 4
        sd.sd_kv4_write(shp, c, K.bfloat16(), V.bfloat16(), 512, first=t)
        del K, V
    qb = base.bfloat16().expand(B, h * G, 128).contiguous()
    out, lse = torch.empty((B, h * G, 128), device="cuda"), torch.empty((B, h * G), device="cuda")
    ws = torch.empty(sd.sd_kv4_attend_workspace_size(shp), dtype=torch.uint8, device="cuda")
    sd.sd_kv4_attend(shp, qb, c, SCALE, out, lse, ws)
    torch.cuda.synchronize()
    s = torch.tensor(some, device="cuda")
    q, k, v = bits(qb[s]), host(c.k[s], np.uint8), host(c.v[s], np.uint8)
    ref = kb.attend(q, k, v, bits(c.scale[s]), [np.arange(n)] * (len(some) * h), SCALE)
    kb.check(host(out[s], np.float32), host(lse[s], np.float32), ref)


def test_steps_of_every_significand(sd):
    """Steps s of all 128 bf16 significands and of exponents over the whole range, with channels
    on, next to and between the borders of codes (m + (c + 1/2) s): the quotients are
    rounded as an IEEE division's, so every code is that of the plain format."""
    rng = np.random.default_rng(5)
    sig = np.arange(128, 256)
    ex = np.concatenate((np.arange(-100, 118, 7), [117]))
    s = (sig[:, None] * 2.0 ** (ex[None] - 7.0)).reshape(-1)              # [groups]
    off = rng.integers(0, 16, s.size)                                     # m = -off s / 4 or so
    lo = kv.bf16_val(kv.bf16_bits((-off * s / 4).astype(np.float32))).astype(np.float64)
    x = np.empty((s.size, 64))
    x[:] = lo[:, None] + (rng.integers(0, 15, x.shape) + 0.5 + rng.choice(
        [0, 2.0 ** -9, -2.0 ** -9, 2.0 ** -7, -2.0 ** -7], x.shape)) * s[:, None]
    x[:, 0] = lo
    x[:, 1] = lo + 15 * s                                                 # the group's largest
    x = kv.bf16_bits(x.astype(np.float32))
    n = s.size // 2
    rows = x.reshape(n, 128)
    codes, steps, _ = kv.quantise(rows)
    got = kv.bf16_bits(steps.reshape(-1)) & 0x7F
    assert set(got.tolist()) == set(range(128)) and (steps > 0).all()
    # ties are among them: a quotient that is not the division's would show there
    d = kv.bf16_val(rows).astype(np.float64).reshape(n, 2, 64)
    qt = (d - d.min(-1, keepdims=True)) / steps[..., None]
    assert ((qt - np.floor(qt)) == 0.5).sum() > 1000
    c = sd.Kv4Cache(1, 1, n)
    t = dev(rows).view(1, 1, n, 128)
    sd.sd_kv4_write(sd.make_shape(1, 1, 1, n), c, t, t, n)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.k, np.uint8)[0, 0], kv.pack(codes))
    assert np.array_equal(host(c.v, np.uint8)[0, 0], kv.pack(codes))
    assert np.array_equal(bits(c.scale)[0, 0, :, 0:4:2], kv.bf16_bits(steps))
