"""GPU tests of the 4-bit K/V cache: sd_kv4_write and sd_kv4_read bit for bit, sd_kv4_attend
and sd_kv4_gather_attend against 64-bit attention over the same cache within the worst-case
bounds of _kv4.py."""
import math

import numpy as np
import pytest
import torch

import _kv4 as kv
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


@pytest.fixture(params=[False, True], ids=["chosen", "stream"])
def path(sd, request):
    """The kernel the library chooses, then the streaming one for every size."""
    before = sd.sd_set_fallback_paths(request.param)
    yield
    sd.sd_set_fallback_paths(before)


def cache_of(sd, k, v, rec):
    B, h, n = k.shape[:3]
    return sd.Kv4Cache(B, h, n, k=dev(k), v=dev(v), scale=dev(rec))


def filled(rng, B, h, ncap):
    """A cache of random bytes and of scale records of every kind (a write's target)."""
    return (rng.integers(0, 256, (B, h, ncap, 64)).astype(np.uint8),
            rng.integers(0, 256, (B, h, ncap, 64)).astype(np.uint8),
            rng.integers(0, 65536, (B, h, ncap, 8)).astype(np.uint16))


def same_bits(a, b):
    """bf16 bits equal; -0 is as +0 and one NaN as another (the format fixes neither)."""
    def plain(x):
        return np.where(x == 0x8000, 0, np.where((x & 0x7FFF) > 0x7F80, 0x7FC0, x))
    return np.array_equal(plain(a), plain(b))


def special_rows(x):
    """Groups that are constant, tied, not finite, overflowing or tiny, in row-major rows."""
    f = kv.bf16_val(x).copy().reshape(-1, 128)
    for r in range(0, f.shape[0], 7):
        kind = (r // 7) % 7
        if kind == 0:
            f[r] = 2.5
        elif kind == 1:
            f[r, :64] = np.arange(64) % 31 / 2  # ties at half steps (s = 1)
        elif kind == 2:
            f[r, 3] = np.nan
        elif kind == 3:
            f[r, 120] = -np.inf
        elif kind == 4:
            f[r, 0], f[r, 1] = 3.0e38, -3.0e38
        elif kind == 5:
            f[r, :] *= np.float32(3e-30)
        else:
            f[r, :] *= np.float32(1e36)
    return kv.bf16_bits(f).reshape(x.shape)


@pytest.mark.parametrize("B,h,m,n,ncap", [(1, 1, 1, 1, 1), (3, 2, 1, 50, 64), (2, 4, 7, 33, 33),
                                          (1, 2, 129, 200, 256), (5, 8, 67, 100, 130)])
def test_write_bits(sd, B, h, m, n, ncap):
    rng = np.random.default_rng(B * 1000 + m)
    K, V = special_rows(kv.tokens(rng, (B, h, m))), kv.tokens(rng, (B, h, m))
    ref = filled(rng, B, h, ncap)
    c = cache_of(sd, *ref)
    pos = rng.integers(-3, n, B).astype(np.int32)
    length = rng.integers(0, m + 3, B).astype(np.int32)
    pos[0], length[0] = min(2, n - 1), m
    if B > 1:
        length[1] = 0
    first = 1 if n > 1 else 0
    ek, ev, er = kv.encode(K, V)
    for b in range(B):
        for t in range(min(m, length[b])):
            p = first + pos[b] + t
            if 0 <= p < n:
                ref[0][b, :, p], ref[1][b, :, p], ref[2][b, :, p] = ek[b, :, t], ev[b, :, t], er[b, :, t]
    shp = sd.make_shape(B, h, h, n, 128, ncap)
    sd.sd_kv4_write(shp, c, dev(K), dev(V), m, pos=dev(pos), length=dev(length), first=first)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.k, np.uint8), ref[0])
    assert np.array_equal(host(c.v, np.uint8), ref[1])
    assert same_bits(host(c.scale.view(torch.int16), np.uint16), ref[2])


def test_write_strides(sd):
    """Token-major projections ([B][m][hkv][d], K and V in one array), a broadcast head, one
    half only."""
    rng = np.random.default_rng(7)
    B, h, m, n = 2, 4, 19, 40
    kvt = kv.tokens(rng, (B, m, 2, h))  # [B][m][2][h][128]
    t = dev(kvt)
    K, V = t[:, :, 0].transpose(1, 2), t[:, :, 1].transpose(1, 2)
    shp = sd.make_shape(B, h, h, n)
    c = sd.Kv4Cache(B, h, n)
    sd.sd_kv4_write(shp, c, K, V, m, first=5)
    ek, ev, er = kv.encode(np.swapaxes(kvt[:, :, 0], 1, 2), np.swapaxes(kvt[:, :, 1], 1, 2))
    assert np.array_equal(host(c.k, np.uint8)[:, :, 5:5 + m], ek)
    assert np.array_equal(host(c.v, np.uint8)[:, :, 5:5 + m], ev)
    assert same_bits(host(c.scale.view(torch.int16), np.uint16)[:, :, 5:5 + m], er)
    assert not host(c.k, np.uint8)[:, :, :5].any() and not host(c.k, np.uint8)[:, :, 5 + m:].any()
    # one head broadcast over all, keys only: the values and their scales stay
    one = K[:, :1].expand(B, h, m, 128)
    before = host(c.v, np.uint8).copy(), host(c.scale.view(torch.int16), np.uint16).copy()
    sd.sd_kv4_write(shp, c, one, None, m, first=5)
    bk = np.broadcast_to(np.swapaxes(kvt[:, :, 0], 1, 2)[:, :1], (B, h, m, 128))
    assert np.array_equal(host(c.k, np.uint8)[:, :, 5:5 + m], kv.encode(bk, bk)[0])
    assert np.array_equal(host(c.v, np.uint8), before[0])
    assert np.array_equal(host(c.scale.view(torch.int16), np.uint16)[..., 4:], before[1][..., 4:])
    # a longer source than m: its own strides count
    c2 = sd.Kv4Cache(B, h, n)
    full = K.contiguous()
    sd.sd_kv4_write(shp, c2, full, full, 3)
    assert np.array_equal(host(c2.k, np.uint8)[:, :, :3], ek[:, :, :3])


@pytest.mark.parametrize("B,h,m,n,ncap", [(1, 1, 1, 1, 1), (3, 2, 5, 50, 64), (2, 4, 133, 140, 160)])
def test_read_bits(sd, B, h, m, n, ncap):
    rng = np.random.default_rng(B * 77 + m)
    K, V = special_rows(kv.tokens(rng, (B, h, ncap))), kv.tokens(rng, (B, h, ncap))
    k, v, rec = kv.encode(K, V)
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(B, h, h, n, 128, ncap)
    pos = rng.integers(-3, n, B).astype(np.int32)
    length = rng.integers(0, m + 2, B).astype(np.int32)
    pos[0], length[0] = 0, m
    mark = kv.bf16_bits(np.float32(7.0))
    rk = np.full((B, h, m, 128), mark, np.uint16)
    rv = rk.copy()
    ok, ov = dev(rk), dev(rv)
    sd.sd_kv4_read(shp, c, ok, ov, m, pos=dev(pos), length=dev(length))
    fk, fv = kv.read(k, rec[..., :4]), kv.read(v, rec[..., 4:])
    for b in range(B):
        for t in range(min(m, length[b])):
            p = pos[b] + t
            if 0 <= p < n:
                rk[b, :, t], rv[b, :, t] = fk[b, :, p], fv[b, :, p]
    assert same_bits(host(ok, np.uint16), rk)
    assert same_bits(host(ov, np.uint16), rv)
    # values only, into a token-major output
    tm = torch.zeros((B, m, h, 128), dtype=torch.bfloat16, device="cuda")
    sd.sd_kv4_read(shp, c, None, tm.transpose(1, 2), m)
    got = np.swapaxes(host(tm.view(torch.int16), np.uint16), 1, 2)
    assert same_bits(got, np.concatenate(
        (fv[:, :, :min(m, n)], np.zeros((B, h, m - min(m, n), 128), np.uint16)), 2))


def run_attend(sd, shp, q, c, begin=None, end=None, lse=True, ws=None, scale=SCALE):
    B, hq = q.shape[:2]
    out = torch.full((B, hq, 128), 9.0, device="cuda")
    ls = torch.full((B, hq), 9.0, device="cuda") if lse else None
    if ws is None:
        ws = torch.full((sd.sd_kv4_attend_workspace_size(shp),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    sd.sd_kv4_attend(shp, dev(q), c, scale, out, ls, ws,
                     begin=None if begin is None else dev(begin),
                     end=None if end is None else dev(end))
    torch.cuda.synchronize()
    return host(out, np.float32), host(ls, np.float32) if lse else None


def run_gather(sd, shp, q, c, idx, cnt, max_count, lse=True, scale=SCALE):
    B, hq = q.shape[:2]
    out = torch.full((B, hq, 128), 9.0, device="cuda")
    ls = torch.full((B, hq), 9.0, device="cuda") if lse else None
    ws = torch.full((sd.sd_kv4_gather_attend_workspace_size(shp, max_count),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    sd.sd_kv4_gather_attend(shp, dev(q), c, dev(idx), idx.shape[1], dev(cnt), max_count, scale,
                            out, ls, ws)
    torch.cuda.synchronize()
    return host(out, np.float32), host(ls, np.float32) if lse else None


def setup(rng, B, h, G, ncap):
    q = kv.tokens(rng, (B, h * G), spread=False)
    k, v, rec = kv.encode(kv.tokens(rng, (B, h, ncap)), kv.tokens(rng, (B, h, ncap)))
    return q, k, v, rec


def ranges(B, h, n, begin, end):
    b0 = np.zeros(B, np.int64) if begin is None else np.maximum(begin, 0)
    e0 = np.full(B, n) if end is None else np.minimum(end, n)
    return [np.arange(b0[b], max(b0[b], e0[b])) for b in range(B) for _ in range(h)]


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 64, 127, 257, 1000, 4099])
def test_attend_lengths(sd, path, n, G):
    rng = np.random.default_rng(n * 10 + G)
    q, k, v, rec = setup(rng, 2, 2, G, n + 5)
    rec[:, :, n:] = 0x7FC0  # NaN behind the last token
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(2, 2 * G, 2, n, 128, n + 5)
    ref = kv.attend(q, k, v, rec, ranges(2, 2, n, None, None), SCALE)
    out, lse = run_attend(sd, shp, q, c)
    kv.check(out, lse, ref)
    out2, _ = run_attend(sd, shp, q, c, lse=False)
    assert np.array_equal(out, out2)


@pytest.mark.parametrize("B,h,G,n", [(7, 1, 4, 300), (40, 2, 8, 130), (130, 4, 2, 70),
                                     (9, 8, 1, 1025), (600, 1, 4, 40)])
def test_attend_ragged(sd, path, B, h, G, n):
    """Ranges of every kind: empty, inverted, outside [0, n), one token, all."""
    rng = np.random.default_rng(B)
    q, k, v, rec = setup(rng, B, h, G, n + 3)
    begin = rng.integers(-5, n, B).astype(np.int32)
    end = (begin + rng.integers(-2, n + 5, B)).astype(np.int32)
    begin[0], end[0] = 0, 0
    begin[1], end[1] = n - 1, n + 1000
    begin[2], end[2] = -7, 2 ** 31 - 1
    begin[3], end[3] = n, 2 * n
    begin[4], end[4] = 17, 18
    toks = ranges(B, h, n, begin, end)
    for b in range(B):  # NaN in everything outside the range
        inside = np.zeros(n + 3, bool)
        inside[toks[b * h]] = True
        rec[b, :, ~inside] = 0x7FC0
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(B, h * G, h, n, 128, n + 3)
    out, lse = run_attend(sd, shp, q, c, begin, end)
    kv.check(out, lse, kv.attend(q, k, v, rec, toks, SCALE))
    # begin or end alone
    for bb, ee in ((begin, None), (None, end)):
        tk = ranges(B, h, n, bb, ee)
        clean = rec.copy()
        clean[np.repeat(np.isnan(kv.bf16_val(rec)).any(-1, keepdims=True), 8, -1)] = 0x3F80
        out, lse = run_attend(sd, shp, q, cache_of(sd, k, v, clean), bb, ee)
        kv.check(out, lse, kv.attend(q, k, v, clean, tk, SCALE))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("B,h,mc", [(1, 1, 1), (2, 2, 17), (3, 2, 64), (2, 8, 530), (64, 2, 129),
                                    (300, 1, 33)])
def test_gather(sd, path, B, h, mc, G):
    """Any order, duplicates, indices outside [0, n), counts of -1, 0 and above max_count."""
    rng = np.random.default_rng(mc * 31 + G)
    n, ncap, stride = 700, 704, mc + 3
    q, k, v, rec = setup(rng, B, h, G, ncap)
    rows = B * h
    idx = rng.integers(0, n, (rows, stride)).astype(np.int32)
    bad = rng.random((rows, stride)) < 0.1
    idx[bad] = rng.choice([-1, n, n + 3, 2 ** 31 - 1, -2 ** 31], bad.sum())
    cnt = rng.integers(0, mc + 5, rows).astype(np.int32)
    cnt[0] = mc
    for i, x in enumerate((0, -1, 1, 16, mc + 100)):
        if i + 1 < rows:
            cnt[i + 1] = x
    if rows > 7:
        idx[7] = 5  # the same token again and again
    toks = []
    for r in range(rows):
        t = idx[r, :max(0, min(cnt[r], mc))]
        toks.append(t[(t >= 0) & (t < n)])
    listed = np.zeros((B, h, ncap), bool)
    for r in range(rows):
        listed[r // h, r % h, toks[r]] = True
    rec[~listed] = 0x7FC0  # NaN in every token that is not selected
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(B, h * G, h, n, 128, ncap)
    ref = kv.attend(q, k, v, rec, toks, SCALE)
    out, lse = run_gather(sd, shp, q, c, idx, cnt, mc)
    kv.check(out, lse, ref)
    out2, _ = run_gather(sd, shp, q, c, idx, cnt, mc, lse=False)
    assert np.array_equal(out, out2)


def test_gather_none(sd, path):
    rng = np.random.default_rng(1)
    q, k, v, rec = setup(rng, 2, 2, 4, 64)
    shp = sd.make_shape(2, 8, 2, 64)
    idx = np.zeros((4, 1), np.int32)
    out, lse = run_gather(sd, shp, q, cache_of(sd, k, v, rec), idx, np.full(4, 5, np.int32), 0)
    assert not out.any() and np.all(np.isneginf(lse))


@pytest.mark.parametrize("gather", [False, True])
def test_nan_stays_in_its_row_and_group(sd, path, gather):
    """A NaN value makes its group of outputs NaN, a NaN key its whole KV head; other rows,
    also those that follow in the same call, are untouched."""
    rng = np.random.default_rng(11)
    B, h, G, n = 6, 2, 4, 200
    q, k, v, rec = setup(rng, B, h, G, n)
    rec[1, 0, 20, 4:6] = 0x7FC0      # values, group 0
    rec[2, 1, 150, 6:8] = 0x7FC0     # values, group 1
    rec[3, 0, 0, 0:2] = 0x7FC0       # keys
    rec[4, 1, n - 1, 2:4] = 0x7FC0
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(B, h * G, h, n)
    idx = np.tile(np.arange(n, dtype=np.int32), (B * h, 1))
    ref = kv.attend(q, k, v, rec, [idx[0]] * (B * h), SCALE)
    if gather:
        out, lse = run_gather(sd, shp, q, c, idx, np.full(B * h, n, np.int32), n)
    else:
        out, lse = run_attend(sd, shp, q, c)
    kv.check(out, lse, ref)
    assert np.isnan(out).any() and np.isfinite(out).any()


@pytest.mark.parametrize("case", ["sharp", "flat", "growing", "big_v", "tiny", "zero_q",
                                  "negative_scale", "big_q", "huge_unweighted"])
def test_attend_ranges_of_values(sd, path, case):
    """Logits that differ by hundreds, maxima that grow along the cache, values whose scales
    differ by many powers of two, queries and caches at the ends of the range."""
    rng = np.random.default_rng(5)
    B, h, G, n = 2, 2, 4, 900
    qf = rng.standard_normal((B, h * G, 128))
    K = rng.standard_normal((B, h, n, 128))
    V = rng.standard_normal((B, h, n, 128))
    scale = SCALE
    if case == "sharp":
        qf *= 12
    elif case == "flat":
        qf *= 1e-4
    elif case == "growing":
        K += qf[:, ::G, None] * np.linspace(-4, 4, n)[None, None, :, None]
    elif case == "big_v":
        V *= 2.0 ** rng.integers(-30, 31, (B, h, n, 1))
    elif case == "tiny":
        K *= 1e-20
        V *= 1e-25
        qf *= 1e-12
    elif case == "zero_q":
        qf[:, ::2] = 0
    elif case == "negative_scale":
        scale = -0.2
    elif case == "big_q":
        qf *= 2.0 ** np.linspace(-20, 20, 128)
        K /= 2.0 ** np.linspace(-20, 20, 128) * 8
    else:  # the first tokens: enormous values whose weight is 0
        K[:, :, :3] = -400 * np.repeat(qf[:, ::G], 1, 1)[:, :, None]
        qf = np.repeat(qf[:, ::G], G, 1)
        V[:, :, :3] *= 1e30
    q = kv.bf16_bits(qf.astype(np.float32))
    k, v, rec = kv.encode(kv.bf16_bits(K.astype(np.float32)), kv.bf16_bits(V.astype(np.float32)))
    shp = sd.make_shape(B, h * G, h, n)
    ref = kv.attend(q, k, v, rec, ranges(B, h, n, None, None), scale)
    c = cache_of(sd, k, v, rec)
    out, lse = run_attend(sd, shp, q, c, scale=scale)
    kv.check(out, lse, ref)
    idx = np.tile(np.arange(n, dtype=np.int32), (B * h, 1))
    out, lse = run_gather(sd, shp, q, c, idx, np.full(B * h, n, np.int32), n, scale=scale)
    kv.check(out, lse, ref)


def test_offsets_past_32_bits(sd):
    """The last rows of a cache of 2.7 GB of codes per array: write, read, both attentions."""
    rng = np.random.default_rng(13)
    h, ncap, G = 40, 1 << 20, 4
    c = sd.Kv4Cache(1, h, ncap)
    c.scale.fill_(float("nan"))  # whatever is read by mistake shows
    m, n = 37, ncap
    K, V = kv.tokens(rng, (1, h, m)), kv.tokens(rng, (1, h, m))
    shp = sd.make_shape(1, h * G, h, n)
    sd.sd_kv4_write(shp, c, dev(K), dev(V), m, first=n - m)
    k, v, rec = kv.encode(K, V)
    ok = torch.zeros((1, h, m, 128), dtype=torch.bfloat16, device="cuda")
    ov = torch.zeros_like(ok)
    sd.sd_kv4_read(shp, c, ok, ov, m, first=n - m)
    assert same_bits(host(ok.view(torch.int16), np.uint16), kv.read(k, rec[..., :4]))
    assert same_bits(host(ov.view(torch.int16), np.uint16), kv.read(v, rec[..., 4:]))
    q = kv.tokens(rng, (1, h * G), spread=False)
    ref = kv.attend(q, k, v, rec, [np.arange(m)] * h, SCALE)
    out, lse = run_attend(sd, shp, q, c, np.array([n - m], np.int32), None)
    kv.check(out, lse, ref)
    idx = np.tile(np.arange(n - m, n, dtype=np.int32), (h, 1))
    out, lse = run_gather(sd, shp, q, c, idx, np.full(h, m, np.int32), m)
    kv.check(out, lse, ref)


def test_streams_and_graphs(sd):
    """A side stream, and two captured graphs that share a workspace, replayed in turn with
    new inputs; the same bits as eager calls."""
    rng = np.random.default_rng(17)
    B, h, G, n = 3, 4, 4, 1500
    q, k, v, rec = setup(rng, B, h, G, n)
    c = cache_of(sd, k, v, rec)
    shp = sd.make_shape(B, h * G, h, n)
    end = np.array([n, 700, 3], np.int32)
    idx = np.stack([rng.permutation(n)[:600] for _ in range(B * h)]).astype(np.int32)
    cnt = np.full(B * h, 600, np.int32)
    eager_a = run_attend(sd, shp, q, c, end=end)
    eager_g = run_gather(sd, shp, q, c, idx, cnt, 600)
    dq, de, di, dc = dev(q), dev(end), dev(idx), dev(cnt)
    out, lse = torch.zeros((B, h * G, 128), device="cuda"), torch.zeros((B, h * G), device="cuda")
    ws = torch.empty(max(sd.sd_kv4_attend_workspace_size(shp),
                         sd.sd_kv4_gather_attend_workspace_size(shp, 600)), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sd.sd_kv4_attend(shp, dq, c, SCALE, out, lse, ws, end=de, stream=side)
    side.synchronize()
    assert np.array_equal(host(out, np.float32), eager_a[0])
    ga, gg = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        sd.sd_kv4_attend(shp, dq, c, SCALE, out, lse, ws, end=de)
    with torch.cuda.graph(gg):
        sd.sd_kv4_gather_attend(shp, dq, c, di, 600, dc, 600, SCALE, out, lse, ws)
    for g, want in ((ga, eager_a), (gg, eager_g), (ga, eager_a), (ga, eager_a), (gg, eager_g)):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out, np.float32), want[0])
        assert np.array_equal(host(lse, np.float32), want[1])
    q2 = kv.tokens(rng, (B, h * G), spread=False)
    dq.copy_(dev(q2))
    de.copy_(dev(np.array([1, n, 900], np.int32)))
    ga.replay()
    torch.cuda.synchronize()
    ref = kv.attend(q2, k, v, rec, ranges(B, h, n, None, np.array([1, n, 900])), SCALE)
    kv.check(host(out, np.float32), host(lse, np.float32), ref)


def test_decode_loop(sd):
    """Prompts written at once, then a token per sequence and step: written, read back,
    attended; every step against the plain cache."""
    rng = np.random.default_rng(19)
    B, h, G, ncap = 3, 2, 4, 96
    c = sd.Kv4Cache(B, h, ncap)
    lens = np.array([40, 1, 63], np.int32)
    K, V = kv.tokens(rng, (B, h, 63)), kv.tokens(rng, (B, h, 63))
    shp = sd.make_shape(B, h * G, h, ncap)
    sd.sd_kv4_write(shp, c, dev(K), dev(V), 63, length=dev(lens))
    k, v, rec = (np.zeros((B, h, ncap, w), t) for w, t in ((64, np.uint8), (64, np.uint8),
                                                          (8, np.uint16)))
    ek, ev, er = kv.encode(K, V)
    for b in range(B):
        for to, x in ((k, ek), (v, ev), (rec, er)):
            to[b, :, :lens[b]] = x[b, :, :lens[b]]
    for _ in range(6):
        K, V = kv.tokens(rng, (B, h, 1)), kv.tokens(rng, (B, h, 1))
        sd.sd_kv4_write(shp, c, dev(K), dev(V), 1, pos=dev(lens))
        ek, ev, er = kv.encode(K, V)
        for b in range(B):
            k[b, :, lens[b]], v[b, :, lens[b]], rec[b, :, lens[b]] = (x[b, :, 0] for x in (ek, ev, er))
        lens += 1
        assert np.array_equal(host(c.k, np.uint8), k) and np.array_equal(host(c.v, np.uint8), v)
        q = kv.tokens(rng, (B, h * G), spread=False)
        out, lse = run_attend(sd, shp, q, c, end=lens)
        kv.check(out, lse, kv.attend(q, k, v, rec, ranges(B, h, ncap, None, lens), SCALE))


def values(codes, rec, dtype):
    """What a cache's rows stand for (torch, on the GPU): [..., 128] in `dtype`."""
    w = codes.contiguous().view(torch.int32)[..., None]
    c = ((w >> torch.arange(0, 32, 4, device="cuda")) & 15).to(dtype)      # [..., 16, 8]
    c = c.unflatten(-2, (8, 2)).transpose(-3, -2).flatten(-2)              # [..., 2, 64]
    sm = rec.to(dtype).unflatten(-1, (2, 2))
    return (c * sm[..., :1] + sm[..., 1:]).flatten(-2)


@pytest.mark.parametrize("B,h,G,n", [(1, 1, 4, 300), (3, 2, 8, 5000), (2, 2, 1, 20000),
                                     (1, 2, 4, 300000), (1, 1, 8, 600000)])
def test_as_exact_as_fp32(sd, B, h, G, n):
    """The error against 64 bits, in the 2-norm, is at most twice that of the plain fp32
    computation on the same cache (both round alike: one fp32 rounding per operation).
    Worst-case bounds would pass a loss of many bits here: outputs of flat attention are
    means of values that change sign, so a bias in the sums shows."""
    g = torch.Generator(device="cuda").manual_seed(n)
    c = sd.Kv4Cache(B, h, n)
    shp = sd.make_shape(B, h * G, h, n)
    for t in range(0, n, 65536):
        m = min(65536, n - t)
        kv2 = torch.randn((2, B, h, m, 128), device="cuda", generator=g).bfloat16()
        sd.sd_kv4_write(shp, c, kv2[0], kv2[1], m, first=t)
    q = torch.randn((B, h * G, 128), device="cuda", generator=g).bfloat16()
    got = {}
    out, lse = torch.empty((B, h * G, 128), device="cuda"), torch.empty((B, h * G), device="cuda")
    ws = torch.empty(max(sd.sd_kv4_attend_workspace_size(shp),
                         sd.sd_kv4_gather_attend_workspace_size(shp, n)), dtype=torch.uint8,
                     device="cuda")
    sd.sd_kv4_attend(shp, q, c, SCALE, out, lse, ws)
    got["attend"] = out.clone(), lse.clone()
    idx = torch.stack([torch.randperm(n, device="cuda", generator=g) for _ in range(B * h)]).int()
    cnt = torch.full((B * h,), n, dtype=torch.int32, device="cuda")
    sd.sd_kv4_gather_attend(shp, q, c, idx, n, cnt, n, SCALE, out, lse, ws)
    got["gather"] = out.clone(), lse.clone()

    def plain(dtype):
        K, V = values(c.k, c.scale[..., :4], dtype), values(c.v, c.scale[..., 4:], dtype)
        z = (q.to(dtype).unflatten(1, (h, G)) @ K.transpose(-1, -2)) * SCALE
        top = z.amax(-1, keepdim=True)
        p = torch.exp(z - top)
        l = p.sum(-1, keepdim=True)
        return ((p @ V) / l).flatten(1, 2).double(), (torch.log(l) + top).flatten(1).double()

    ref, fp32 = plain(torch.float64), plain(torch.float32)
    for name, pair in got.items():
        for x, y, f in zip(pair, ref, fp32):
            err = float((x.double() - y).norm() / y.norm())
            base = float((f - y).norm() / y.norm())
            assert err <= max(2 * base, 2e-7), (name, err, base)


@pytest.mark.parametrize("kind", ["planes", "quest"])
def test_step_over_the_cache(sd, kind):
    """A sparse decode step whose only K and V are the 4-bit cache: written, its keys read
    back for the index, the step run eagerly and as a graph.  The selection is the bf16
    step's over the values read back, the attention is the plain one's over it."""
    from top_sparse_decode_gb300.pipeline import DecodeStep, StepConfig, build_index
    rng = np.random.default_rng(23)
    B, h, G, n = 2, 2, 4, 4096
    kw = dict(k=64, sink=4, local=32) if kind == "planes" else dict(k=8, sink=0, local=1)
    cfg = StepConfig(sd.SD_IDX_PLANES if kind == "planes" else sd.SD_IDX_MINMAX, B, h * G, h, n,
                     **kw)
    shp = sd.make_shape(B, h * G, h, n)
    c = sd.Kv4Cache(B, h, n)
    sd.sd_kv4_write(shp, c, dev(kv.tokens(rng, (B, h, n))), dev(kv.tokens(rng, (B, h, n))), n)
    K = torch.empty((B, h, n, 128), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    sd.sd_kv4_read(shp, c, K, V, n)
    index = build_index(cfg, K)
    sigma2 = torch.rand((h, 128), device="cuda")
    q = kv.tokens(rng, (B, h * G), spread=False)
    dq = dev(q)
    step = DecodeStep(cfg, None, None, index, sigma2=sigma2, kv4=c)
    bf16 = DecodeStep(cfg, K, V, index, sigma2=sigma2)
    step.run(dq)
    bf16.run(dq)
    torch.cuda.synchronize()
    assert torch.equal(step.idx, bf16.idx) and torch.equal(step.count, bf16.count)
    idx, cnt = host(step.idx, np.int32), host(step.count, np.int32)
    toks = [idx[r, :cnt[r]] for r in range(B * h)]
    k, v = host(c.k, np.uint8), host(c.v, np.uint8)
    rec = host(c.scale.view(torch.int16), np.uint16)
    ref = kv.attend(q, k, v, rec, toks, step.scale)
    out, lse = host(step.out, np.float32).copy(), host(step.lse, np.float32).copy()
    kv.check(out, lse, ref)
    # the other step's K and V are rounded to bf16, 2^-9 of a value at most: logits move by
    # dz <= 2^-9 scale sum |q k|, weights by e^(2 dz), outputs by both over the largest |v|
    zm = (torch.from_numpy(kv.bf16_val(q)).cuda().abs().unflatten(1, (h, G)) @
          K.float().abs().transpose(-1, -2)).amax().item() * step.scale
    far = (2 * math.expm1(2 * 2.0 ** -9 * zm) + 2.0 ** -9) * V.float().abs().amax().item()
    assert np.abs(host(bf16.out, np.float32) - out).max() <= far
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(dq)
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host(step.out, np.float32), out)
    with pytest.raises(ValueError):
        DecodeStep(cfg, None, None, index, sigma2=sigma2)
    if kind == "planes":
        with pytest.raises(ValueError):
            DecodeStep(StepConfig(cfg.kind, B, h * G, h, n, select_attend=True), K, V, index,
                       sigma2=sigma2, kv4=c)



def test_two_streams_at_once(sd):
    """Calls on two streams at the same time, each with a workspace of its own."""
    rng = np.random.default_rng(31)
    B, h, G, n = 4, 4, 4, 9000
    q, k, v, rec = setup(rng, B, h, G, n)
    c, shp = cache_of(sd, k, v, rec), sd.make_shape(B, h * G, h, n)
    dq = dev(q)
    ends = [dev(np.array(e, np.int32)) for e in ((n, 1, 4500, 0), (77, n, n, 8999))]
    want = [run_attend(sd, shp, q, c, end=host(e, np.int32)) for e in ends]
    streams = [torch.cuda.Stream() for _ in ends]
    outs = [torch.zeros((B, h * G, 128), device="cuda") for _ in ends]
    lses = [torch.zeros((B, h * G), device="cuda") for _ in ends]
    ws = [torch.empty(sd.sd_kv4_attend_workspace_size(shp), dtype=torch.uint8, device="cuda")
          for _ in ends]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            sd.sd_kv4_attend(shp, dq, c, SCALE, outs[i], lses[i], ws[i], end=ends[i], stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(host(outs[i], np.float32), want[i][0])
        assert np.array_equal(host(lses[i], np.float32), want[i][1])


def test_arrays_at_16_bytes(sd):
    """Cache arrays, q and outputs that start 16 bytes into an allocation."""
    rng = np.random.default_rng(37)
    B, h, G, n = 2, 3, 4, 301
    q, k, v, rec = setup(rng, B, h, G, n)

    def off(x):
        t = dev(x).contiguous().view(torch.uint8).flatten()
        buf = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda")
        buf[16:] = t
        return buf[16:]

    c = sd.Kv4Cache(B, h, n, k=off(k), v=off(v), scale=off(rec))
    shp = sd.make_shape(B, h * G, h, n)
    out = torch.zeros(B * h * G * 128 + 4, device="cuda")[4:]
    lse = torch.zeros(B * h * G + 1, device="cuda")[1:]
    ws = torch.zeros(sd.sd_kv4_attend_workspace_size(shp) + 16, dtype=torch.uint8, device="cuda")[16:]
    ref = kv.attend(q, k, v, rec, ranges(B, h, n, None, None), SCALE)
    sd.sd_kv4_attend(shp, off(q), c, SCALE, out, lse, ws)
    torch.cuda.synchronize()
    kv.check(host(out, np.float32).reshape(B, h * G, 128), host(lse, np.float32).reshape(B, h * G), ref)
    idx = np.stack([rng.permutation(n)[:100] for _ in range(B * h)]).astype(np.int32)
    sd.sd_kv4_gather_attend(shp, off(q), c, dev(idx), 100, dev(np.full(B * h, 100, np.int32)), 100,
                            SCALE, out, lse, ws)
    torch.cuda.synchronize()
    ref = kv.attend(q, k, v, rec, list(idx), SCALE)
    kv.check(host(out, np.float32).reshape(B, h * G, 128), host(lse, np.float32).reshape(B, h * G), ref)
    K = off(kv.tokens(rng, (B, h, n))).view(torch.bfloat16).view(B, h, n, 128)
    sd.sd_kv4_write(shp, c, K, K, n)
    ek = kv.encode(host(K.contiguous().view(torch.int16), np.uint16),
                   host(K.contiguous().view(torch.int16), np.uint16))
    assert np.array_equal(host(c.k, np.uint8).reshape(ek[0].shape), ek[0])
    assert np.array_equal(host(c.v, np.uint8).reshape(ek[1].shape), ek[1])


def test_many_rows(sd, path):
    """20,000 rows, most of them empty or of one token."""
    rng = np.random.default_rng(41)
    B, h, G, n = 5000, 4, 2, 40
    q, k, v, rec = setup(rng, B, h, G, n)
    c, shp = cache_of(sd, k, v, rec), sd.make_shape(B, h * G, h, n)
    end = rng.choice([0, 0, 1, 33, 40], B).astype(np.int32)
    out, lse = run_attend(sd, shp, q, c, end=end)
    some = np.concatenate((np.arange(40), rng.integers(0, B, 60)))
    toks = [np.arange(end[b]) for b in some for _ in range(h)]
    kv.check(out[some], lse[some], kv.attend(q[some], k[some], v[some], rec[some], toks, SCALE))
    none = end == 0
    assert not out[none].any() and np.all(np.isneginf(lse[none]))
    assert np.all(np.isfinite(lse[~none]))


def test_fallback_switch(sd):
    """sd_set_fallback_paths(1): the streaming kernel also where clusters would run, with the
    same results within the bounds."""
    rng = np.random.default_rng(29)
    for B, h, G, n in ((1, 1, 4, 5), (3, 2, 8, 333), (2, 8, 2, 100)):
        q, k, v, rec = setup(rng, B, h, G, n)
        c = cache_of(sd, k, v, rec)
        shp = sd.make_shape(B, h * G, h, n)
        end = rng.integers(0, n + 1, B).astype(np.int32)
        ref = kv.attend(q, k, v, rec, ranges(B, h, n, None, end), SCALE)
        before = sd.sd_set_fallback_paths(True)
        try:
            out, lse = run_attend(sd, shp, q, c, end=end)
        finally:
            sd.sd_set_fallback_paths(before)
        kv.check(out, lse, ref)


def test_order_after_other_work(sd):
    """Each call follows what its stream holds before it: copies (as memcpy and as kernels),
    an event of another stream, its own kernels; eagerly and captured, with inputs that
    change from pass to pass."""
    rng = np.random.default_rng(43)
    B, h, G, n = 4, 4, 4, 700
    shp = sd.make_shape(B, h * G, h, n)
    src = [dev(kv.tokens(rng, (2, B, h, n))) for _ in range(3)]
    q = kv.tokens(rng, (B, h * G), spread=False)
    dq = dev(q)
    want = []
    for x in src:
        b = host(x, np.uint16)
        k, v, rec = kv.encode(b[0], b[1])
        want.append((kv.read(k, rec[..., :4]), kv.attend(q, k, v, rec, ranges(B, h, n, None, None),
                                                         SCALE)))
    c = sd.Kv4Cache(B, h, n)
    X = torch.zeros_like(src[0])
    K2, V2 = torch.zeros_like(X[0]), torch.zeros_like(X[0])
    out, lse = torch.zeros((B, h * G, 128), device="cuda"), torch.zeros((B, h * G), device="cuda")
    ws = torch.empty(sd.sd_kv4_attend_workspace_size(shp), dtype=torch.uint8, device="cuda")

    def work():
        sd.sd_kv4_write(shp, c, X[0], X[1], n)
        sd.sd_kv4_read(shp, c, K2, V2, n)
        sd.sd_kv4_attend(shp, dq, c, SCALE, out, lse, ws)

    def check(i):
        torch.cuda.synchronize()
        assert same_bits(host(K2, np.uint16), want[i][0]), i
        kv.check(host(out, np.float32), host(lse, np.float32), want[i][1])

    side = torch.cuda.Stream()
    for i in (0, 1, 2, 1):
        torch.cuda._sleep(200000)
        X.copy_(src[i])                      # a device copy
        work()
        check(i)
        torch.cuda._sleep(200000)
        torch.add(src[i], 0, out=X)          # a kernel
        work()
        check(i)
        X.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(400000)
            X.copy_(src[i])
        torch.cuda.current_stream().wait_stream(side)
        work()
        check(i)
    feed = src[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X.copy_(feed)
        work()
    for i in (2, 0, 1):
        feed.copy_(src[i])
        graph.replay()
        graph.replay()
        check(i)
