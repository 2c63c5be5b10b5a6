"""sd_qk_norm_rope, sd_window_attend and sd_prefix_attend against their 64-bit forms
(_dense.py), at the sizes, masks and layouts where they can go wrong."""
import math
import os
import subprocess
import sys

import pytest
import torch

from _dense import D, attention, check, norm_rope, norm_rope_tol, visible

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module")
def sd():
    import top_sparse_decode_gb300 as m
    m.lib()
    return m


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- norm, rotation, cache -------------------------------------------------------------
ROPE = [
    # B, hkv, G, n, n_cap, m, first, pos, length, rotary, rot, pairs, norms
    (1, 1, 1, 1, 1, 1, 0, None, None, None, 128, False, "qk"),
    (2, 2, 4, 40, 64, 5, 3, [0, 30], [5, 2], None, 128, False, "qk"),
    (3, 8, 4, 700, 700, 333, 0, [0, 300, 690], [333, 0, 333], None, 64, True, "qk"),
    (2, 1, 8, 50, 50, 7, 0, [-3, 48], None, [1 << 20, (1 << 31) - 20], 128, True, "q"),
    (2, 4, 2, 64, 64, 64, 0, None, [-1, 70], [5, -9], 32, False, "k"),
    (1, 2, 1, 33, 40, 33, 0, None, None, None, 0, False, "qk"),
    (5, 8, 8, 9, 16, 1, 0, [0, 8, 9, 4, -1], None, None, 16, False, ""),
    (700, 1, 2, 16, 16, 9, 0, None, None, None, 128, False, "qk"),
    (16, 2, 2, 300, 300, 300, 0, None, None, None, 112, True, "qk"),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_norm_rope(sd, case, layout):
    B, hkv, G, n, cap, m, first, pos, length, rotary, rot, pairs, norms = ROPE[case]
    hq = hkv * G
    if layout == "fused":  # one array [B][m][hq + 2 hkv][128] and q_out [B][m][hq][128]
        x = normal((B, m, hq + 2 * hkv, D), case, 2.0).transpose(1, 2)
        q, k, v = x.split([hq, hkv, hkv], dim=1)
        qo = torch.full((B, m, hq, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    else:
        q, k, v = (normal((B, h, m, D), case + j, 2.0) for j, h in enumerate((hq, hkv, hkv)))
        qo = torch.full((B, hq, m, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qw = 1 + 0.3 * normal((D,), 50).float() if "q" in norms else None
    kw = 1 + 0.3 * normal((D,), 51).float() if "k" in norms else None
    freq = None if rot == 0 else 10000.0 ** (
        -torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    K = torch.full((B, hkv, cap, D), 3.0, dtype=torch.bfloat16, device="cuda")
    V = torch.full_like(K, 5.0)
    rope = sd.make_rope(freq, qw, kw, eps=1e-5, pairs=pairs)
    before = sd.sd_launch_count()
    sd.sd_qk_norm_rope(sd.make_shape(B, hq, hkv, n, D, cap), rope, q, qo, k, v, K, V, m,
                       pos=i32(pos), length=i32(length), rotary=i32(rotary), first=first)
    assert sd.sd_launch_count() == before + 1
    Kr, Vr, qr = K.double() * 0 + 3.0, V.double() * 0 + 5.0, qo.double() * 0 + 7.0
    Kt, qt = torch.zeros_like(Kr), torch.zeros_like(qr)
    for b in range(B):
        l = m if length is None else max(0, min(m, length[b]))
        at = first + (pos[b] if pos else 0)
        r = torch.arange(l, device="cuda") + (rotary[b] if rotary else at)
        args = (1e-5, r, freq, rot, pairs)
        qr[b, :, :l] = norm_rope(q[b, :, :l], qw, *args)
        qt[b, :, :l] = norm_rope_tol(qr[b, :, :l], q[b, :, :l], qw, *args)
        kk = norm_rope(k[b, :, :l], kw, *args)
        kt = norm_rope_tol(kk, k[b, :, :l], kw, *args)
        lo, hi = max(0, -at), max(0, min(l, n - at))
        if lo < hi:
            Kr[b, :, at + lo:at + hi] = kk[:, lo:hi]
            Kt[b, :, at + lo:at + hi] = kt[:, lo:hi]
            Vr[b, :, at + lo:at + hi] = v[b, :, lo:hi].double()
    check(qo, qr, qt, "q")
    check(K, Kr, Kt, "K")
    assert torch.equal(V.double(), Vr)


def test_norm_rope_in_place_and_sides(sd):
    """q turned in its own array; keys alone; values alone; a broadcast input."""
    B, hkv, G, m = 2, 2, 2, 20
    shape = sd.make_shape(B, hkv * G, hkv, m)
    freq = torch.rand(64, device="cuda", dtype=torch.float64)
    rope = sd.make_rope(freq, None, torch.ones(D, device="cuda"))
    q, k = normal((B, hkv * G, m, D), 1), normal((1, hkv, m, D), 2).expand(B, -1, -1, -1)
    pos = torch.arange(m, device="cuda")
    ref = norm_rope(q, None, 0, pos, freq, 128, False)
    tol = norm_rope_tol(ref, q, None, 0, pos, freq, 128, False)
    sd.sd_qk_norm_rope(shape, rope, q, q, None, None, None, None, m)
    check(q, ref, tol, "q in place")
    K, V = (torch.zeros((B, hkv, m, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sd.sd_qk_norm_rope(shape, rope, None, None, k, None, K, None, m)
    ref = norm_rope(k, torch.ones(D, device="cuda"), 1e-6, pos, freq, 128, False)
    check(K, ref, norm_rope_tol(ref, k, torch.ones(D, device="cuda"), 1e-6, pos, freq, 128, False),
          "keys alone")
    v = torch.full_like(K, math.nan)
    v[0, 0, 0, 0] = -math.inf
    v.view(torch.int16)[0, 0, 0, 1] = 0x7F81  # a NaN's own bits pass
    sd.sd_qk_norm_rope(shape, rope, None, None, None, v, None, V, m)
    assert torch.equal(V.view(torch.int16), v.view(torch.int16))


def test_norm_rope_keeps_rows_apart(sd):
    """A row that is not finite, all zeros, or tiny changes no other."""
    m = 24
    shape = sd.make_shape(1, 4, 2, m)
    freq = torch.rand(32, device="cuda", dtype=torch.float64)
    w = torch.ones(D, device="cuda")
    rope = sd.make_rope(freq, w, w, eps=0.0)
    q = normal((1, 4, m, D), 3)
    q[0, 1, 5, 7] = math.inf
    q[0, 2, 6, 9] = math.nan
    q[0, 3, 7] = normal((D,), 4, 1e-15)
    pos = torch.arange(m, device="cuda")
    out = torch.zeros_like(q)
    sd.sd_qk_norm_rope(shape, rope, q, out, None, None, None, None, m)
    ref = norm_rope(q, w, 0.0, pos, freq, 64, False)
    tol = norm_rope_tol(ref, q, w, 0.0, pos, freq, 64, False)
    keep = torch.ones((1, 4, m), dtype=torch.bool, device="cuda")
    keep[0, 1, 5] = keep[0, 2, 6] = False
    check(out[keep], ref[keep], tol[keep], "q")
    assert not torch.isfinite(out[0, 2, 6]).any()


# ---- window attention --------------------------------------------------------------------
def run_window(sd, B, hkv, G, n, cap, m, first, pos, length, window, sink, scale=SCALE, seed=0,
               layout="token", prep=None, ws_fill=None):
    hq = hkv * G
    if layout == "token":
        q = normal((B, m, hq, D), seed).transpose(1, 2)
        out = torch.full((B, m, hq, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    else:
        q = normal((B, hq, m + 3, D), seed)[:, :, 1:m + 1]
        out = torch.full((B, hq, m + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")[:, :, 2:]
    K, V = normal((B, hkv, cap, D), seed + 1), normal((B, hkv, cap, D), seed + 2)
    if cap > n:  # what lies behind n is not read
        K[:, :, n:], V[:, :, n:] = math.nan, math.nan
    if prep:
        prep(q, K, V)
    lse = torch.full((B, hq, m), 7.0, device="cuda")
    shape = sd.make_shape(B, hq, hkv, n, D, cap)
    ws = torch.full((max(16, sd.sd_window_attend_workspace_size(shape, m, window, sink)),),
                    255 if ws_fill is None else ws_fill, dtype=torch.uint8, device="cuda")
    sd.sd_window_attend(shape, q, K, V, m, window, sink, scale, out, lse, ws, pos=i32(pos),
                        length=i32(length), first=first)
    sd.sd_device_status()
    return q, K, V, out, lse


def check_window(case, got, scale=SCALE, some=None):
    B, hkv, G, n, cap, m, first, pos, length, window, sink = case
    q, K, V, out, lse = got
    for b in range(B):
        l = m if length is None else max(0, min(m, length[b]))
        assert (out[b, :, l:] == 7.0).all() and (lse[b, :, l:] == 7.0).all()
        t = torch.arange(l, device="cuda")
        if some and l > some:  # a spread of the rows
            t = torch.unique(torch.cat((t[:70], t[-70:], t[::max(1, l // some)])))
        if not len(t):
            continue
        p = t + first + (pos[b] if pos else 0)
        see = visible(p, n, window, sink, "cuda").repeat_interleave(G, 0)
        for h in range(hkv):
            rows = q[b, h * G:(h + 1) * G][:, t].transpose(0, 1).flatten(0, 1)
            o, e, tol, ltol = attention(rows, K[b, h, :n], V[b, h, :n], see, scale)
            check(out[b, h * G:(h + 1) * G][:, t].transpose(0, 1).flatten(0, 1), o, tol,
                  f"out of ({b}, {h})")
            check(lse[b, h * G:(h + 1) * G][:, t].T.flatten(), e, ltol, f"lse of ({b}, {h})")


WINDOW = [
    # B, hkv, G, n, n_cap, m, first, pos, length, window, sink
    (1, 1, 1, 1, 1, 1, 0, None, None, 1, 0),
    (1, 1, 4, 5, 8, 5, 0, None, None, 2, 1),
    (1, 2, 8, 129, 129, 1, 128, None, None, 129, 0),
    (2, 1, 2, 257, 300, 1, 0, [256, 0], None, 100, 7),
    (3, 2, 4, 1000, 1024, 1, 0, [999, 499, -1], None, 300, 128),
    (4, 2, 4, 700, 700, 1, 0, [699, 700, 5000, 2147483647], [1, 0, 1, 1], 64, 4),
    (2, 8, 4, 5000, 5000, 1, 4999, None, None, 1 << 40, 0),
    (1, 2, 8, 9000, 9000, 1, 8999, None, None, 8500, 200),
    (2, 2, 4, 300, 310, 300, 0, None, None, 300, 0),
    (2, 1, 1, 600, 600, 600, 0, None, [600, 311], 77, 3),
    (1, 2, 2, 513, 513, 385, 128, None, None, 128, 128),
    (3, 2, 8, 500, 520, 67, 0, [0, 200, 480], [67, 33, 67], 50, 20),
    (2, 1, 8, 400, 400, 30, 0, [-20, 395], None, 1, 0),
    (1, 1, 4, 2000, 2000, 130, 1870, None, None, 1900, 0),
    (2, 2, 4, 3000, 3000, 2, 0, [2998, 17], None, 2500, 300),
    (1, 1, 2, 4000, 4000, 8, 3992, None, None, 4000, 0),
    (5, 1, 4, 64, 64, 64, 0, None, [0, 1, 64, 63, -5], 16, 1 << 33),
    (1, 4, 1, 1300, 1300, 1300, 0, None, None, 1, 0),
    (1, 1, 8, 200, 200, 40, 0, [300], None, 64, 10),
]


@pytest.mark.parametrize("case", WINDOW, ids=range(len(WINDOW)))
@pytest.mark.parametrize("layout", ["token", "head"])
def test_window(sd, case, layout):
    check_window(case, run_window(sd, *case, layout=layout))


@pytest.mark.parametrize("case", [
    (1, 2, 4, 4096, 4096, 4096, 0, None, None, 1000, 128),
    (2, 1, 8, 3500, 3500, 3500, 0, None, [3500, 1234], 3500, 0),
    (1, 8, 4, 20000, 20000, 1, 19999, None, None, 20000, 0),
    (1, 1, 4, 30000, 30000, 200, 29800, None, None, 30000, 0),
    (40, 4, 2, 900, 900, 1, 0, [(37 * i) % 900 for i in range(40)], None, 512, 64),
], ids=range(5))
def test_window_long(sd, case):
    check_window(case, run_window(sd, *case, seed=9), some=200)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("m", [1, 3, 31, 64, 65, 128, 129, 257])
def test_window_row_counts(sd, G, m):
    case = (1, 1, G, 700, 700, m, 700 - m, None, None, 200, 5)
    check_window(case, run_window(sd, *case, seed=G + m))


@pytest.mark.parametrize("m", [1, 4, 100, 300])
def test_window_unseen_tokens_reach_nothing(sd, m):
    """Tokens outside every query's window hold NaN and infinities."""
    first, window, sink, n = 300, 90, 11, 700

    def spoil(q, K, V):
        lo = first - window + 1
        for x in (K, V):
            x[:, :, sink:lo:2] = math.nan
            x[:, :, sink + 1:lo:2] = math.inf
            x[:, :, first + m:] = -math.inf
    case = (2, 2, 4, n, n, m, first, None, None, window, sink)
    got = run_window(sd, *case, prep=spoil)
    assert torch.isfinite(got[3].float()).all()
    check_window(case, got)


def median_us(call, reps=21):
    """Median time of a call, from events around each."""
    for _ in range(3):
        call()
    marks = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
             for _ in range(reps)]
    for a, b in marks:
        a.record()
        call()
        b.record()
    torch.cuda.synchronize()
    return sorted(a.elapsed_time(b) for a, b in marks)[reps // 2] * 1e3


@pytest.mark.parametrize("G", [1, 4, 8])
def test_window_unseen_tokens_cost_nothing(sd, G):
    """Between the first tokens and the window, and behind the sequence, the cache holds NaN,
    as one that was never written there may: the tiles that reach into these cells take no
    longer for it.  (Rows computed again by themselves take more than ten times as long.)"""
    first, window, sink, n, m = 1000, 256, 4, 4096, 2048
    case = (1, 4, G, n, n, m, first, None, [m - 5], window, sink)

    def spoil(q, K, V):
        for x in (K, V):
            x[:, :, sink:first - window + 1] = math.nan
            x[:, :, first + m - 5:] = math.nan
    clean, got = run_window(sd, *case), run_window(sd, *case, prep=spoil)
    check_window(case, got, some=200)
    shape, times, length = sd.make_shape(1, 4 * G, 4, n), [], i32([m - 5])
    ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, m, window, sink)),
                     dtype=torch.uint8, device="cuda")
    for q, K, V, out, lse in (clean, got):
        times.append(median_us(lambda: sd.sd_window_attend(
            shape, q, K, V, m, window, sink, SCALE, out, lse, ws, length=length, first=first)))
    assert times[1] <= 2 * times[0], times


@pytest.mark.parametrize("where", [0, 127, 128, 200, 255, 399])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_window_bad_value_reaches_who_sees_it(sd, where, bad):
    """One value of V that is not finite: the queries that see its token get it in that
    channel, every other result is as without it."""
    case = (1, 2, 4, 400, 400, 400, 0, None, None, 150, 2)
    clean = run_window(sd, *case)

    def spoil(q, K, V):
        V[0, 0, where, 17] = bad
    got = run_window(sd, *case, prep=spoil)
    check_window(case, got)
    see = visible(torch.arange(400, device="cuda"), 400, 150, 2, "cuda")[:, where]
    hit = ~torch.isfinite(got[3][0, :4, :, 17].float())
    assert torch.equal(hit, see.expand(4, -1))
    other = torch.ones(D, dtype=torch.bool, device="cuda")
    other[17] = False
    for b, a in ((got[3][0, :4][:, ~see], clean[3][0, :4][:, ~see]),
                 (got[3][0, 4:], clean[3][0, 4:])):
        # rows of a tile that holds the value may be summed in another order
        assert ((b.float() - a.float()).abs() <= 2.0 ** -5).all()


@pytest.mark.parametrize("case", [
    # m = 20 and 300: parts joined by a kernel of their own; 1,500: more items than SMs
    (1, 2, 4, 3000, 3000, 20, 2980, None, None, 2000, 9),
    (1, 1, 8, 3000, 3000, 300, 2700, None, None, 3000, 0),
    (3, 8, 4, 1500, 1500, 1500, 0, None, [1500, 1, 777], 300, 130),
    (2, 2, 1, 900, 900, 900, 0, None, None, 900, 0),
    (1, 1, 2, 700, 700, 650, 0, [-30], None, 90, 3),
], ids=range(5))
def test_window_many_bad_values(sd, case):
    """Values that are not finite all over V: rows see some of them and have others in their
    tiles."""
    def spoil(q, K, V):
        g = torch.Generator(device="cuda").manual_seed(5)
        hit = torch.rand(V.shape, device="cuda", generator=g)
        V[hit < 1e-4] = math.nan
        V[(hit > 1e-4) & (hit < 4e-4)] = math.inf
        V[hit > 1 - 3e-4] = -math.inf
    got = run_window(sd, *case, prep=spoil)
    check_window(case, got)
    bad = ~torch.isfinite(got[3].float())
    assert bad.any() and not bad.all()


def test_window_long_prompt_early_infinity(sd):
    """An infinity in V at the first token of a long prompt, which every row sees: its channel
    infinite in every row, every other right, nothing given up, in bounded time.  (Measured:
    13.4 ms, 0.96 ms without the infinity.)"""
    n = 32768
    case = (1, 1, 4, n, n, n, 0, None, None, n, 0)

    def spoil(q, K, V):
        V[0, 0, 0, 17] = math.inf
    got = run_window(sd, *case, prep=spoil)
    q, K, V, out, lse = got
    assert (out[..., 17] == math.inf).all()
    assert int((~torch.isfinite(out.float())).sum()) == 4 * n
    check_window(case, got, some=100)
    shape = sd.make_shape(1, 4, 1, n)

    def call():
        sd.sd_window_attend(shape, q, K, V, n, n, 0, SCALE, out, lse, None)
    bad = median_us(call, reps=5)
    V[0, 0, 0, 17] = 0.0
    clean = median_us(call, reps=5)
    print(f"{bad:.0f} us, {clean:.0f} us without the infinity")
    assert bad <= 40 * clean
    sd.sd_device_status()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_prefix_bad_value(sd, bad):
    """A prefix's value that is not finite reaches every sequence of its KV head, in its
    channel."""
    case = (17, 4, 8, 777, 800, 33, 33, None)

    def spoil(q, Kp, Vp, K, V):
        Vp[2, 770, 5] = bad
        V[3, 0, 20, 90] = bad
    got = run_prefix(sd, *case, prep=spoil)
    check_prefix(case, got)
    assert int((~torch.isfinite(got[5].float())).sum()) == 17 * 8 + 8


@pytest.mark.parametrize("m", [1, 20, 200])
def test_window_largest_values_without_weight(sd, m):
    """The largest values of V, at tokens whose weights are 0 in fp32, are not seen in out."""
    n = 600
    case = (1, 2, 4, n, n, m, n - m, None, None, n, 0)

    def spoil(q, K, V):
        q[..., 0] = 8.0
        K[..., 0] = 0.0
        K[:, :, 5:n - m:40, 0] = -400.0  # scores some 280 below the others'
        V[:, :, 5:n - m:40] = 3.3e38
    got = run_window(sd, *case, prep=spoil)
    assert got[3].float().abs().max() < 10
    check_window(case, got)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [1, 40, 600, 9000])
def test_single_token_bad_value(sd, n, bad):
    """Single tokens, and the own tokens behind a prefix: a value of V that is not finite comes
    out as itself in its channel, whatever the weights of its token, and in no other."""
    where = sorted({0, n // 3, n // 2, n - 1})

    def spoil(q, K, V):
        for j, w in enumerate(where):
            V[0, :, w, 10 * j + 3] = bad
    case = (2, 2, 4, n, n, 1, n - 1, None, None, n, 0)
    got = run_window(sd, *case, prep=spoil)
    check_window(case, got)
    assert int((~torch.isfinite(got[3].float())).sum()) == 8 * len(where)
    case = (2, 2, 4, 300, 300, n, n, None)
    check_prefix(case, run_prefix(sd, *case, prep=lambda q, Kp, Vp, K, V: spoil(q, K, V)))


def test_window_bad_key(sd):
    """A key that is not finite makes its own readers' scores NaN or infinite, and nothing
    else."""
    case = (1, 1, 4, 300, 300, 300, 0, None, None, 100, 0)

    def spoil(q, K, V):
        K[0, 0, 130, 3] = math.nan
    got = run_window(sd, *case, prep=spoil)
    see = visible(torch.arange(300, device="cuda"), 300, 100, 0, "cuda")[:, 130]
    assert torch.equal(torch.isnan(got[3][0].float()).all(-1), see.expand(4, -1))
    assert torch.equal(torch.isnan(got[4][0]), see.expand(4, -1))


def test_window_empty_scores(sd):
    """Keys of minus infinity leave a row without weight: out 0, lse -inf."""
    case = (1, 1, 2, 200, 200, 200, 0, None, None, 20, 0)

    def spoil(q, K, V):
        q[..., 0] = 1.0
        K[0, 0, :40] = 0.0
        K[0, 0, :40, 0] = -math.inf
    got = run_window(sd, *case, prep=spoil)
    assert (got[3][0, :, :40] == 0).all() and (got[4][0, :, :40] == -math.inf).all()
    assert torch.isfinite(got[3].float()).all()


@pytest.mark.parametrize("m", [1, 200])
@pytest.mark.parametrize("grow", [0.0, 0.5, 30.0, -30.0])
def test_window_rising_scores(sd, m, grow):
    """Scores that rise (or fall) along the sequence, so that the running maximum moves at
    every tile."""
    n = 1000

    def spoil(q, K, V):
        q[..., 0] = 8.0
        K[..., 0] = (torch.arange(n, device="cuda") * (grow / 128)).bfloat16()
    case = (1, 2, 4, n, n, m, n - m, None, None, n, 0)
    check_window(case, run_window(sd, *case, prep=spoil))


@pytest.mark.parametrize("scale", [0.0, 1e-3, 4.0])
def test_window_scales(sd, scale):
    case = (1, 1, 4, 500, 500, 150, 350, None, None, 400, 9)
    check_window(case, run_window(sd, *case, scale=scale), scale=scale)


@pytest.mark.parametrize("scale", [0.0, 2e-38, 1e-30])
def test_window_small_scales(sd, scale):
    """Scales far below 1 with products as far above it (0: every visible token counts alike)."""
    for m in (1, 20, 300):
        case = (1, 1, 4, 600, 600, m, 600 - m, None, None, 500, 9)

        def spoil(q, K, V):
            q[..., 0] = 3e18
            K[..., 0] *= 1.5e19 if scale < 1e-35 else 3e11
        check_window(case, run_window(sd, *case, scale=scale, prep=spoil), scale=scale)


@pytest.mark.parametrize("scale", [1e3, 1e6, 3e8, 1e30])
@pytest.mark.parametrize("low", [-100, -300, 40])
def test_window_wide_scores(sd, scale, low):
    """Whole numbers as scores, times a scale that sets them far apart: a row's result is the
    mean of the values of its largest score, however far that is from 0.  (The scores are
    exact; the scale, log2 e, ln 2 and the products with them are rounded, 2^-24 each.
    Weights of equal scores are equal, of others below 2^-126 from a scale of 1e3 on.)"""
    for m, n, window in ((1, 900, 900), (20, 900, 700), (150, 400, 400), (500, 500, 130)):
        case = (1, 2, 4, n, n, m, n - m, None, None, window, 3)

        def spoil(q, K, V):
            g = torch.Generator(device="cuda").manual_seed(m)
            q[..., 1:] = 0.0
            q[..., 0] = 1.0
            K[..., 0] = torch.randint(low, low + 201, K.shape[:3], device="cuda", generator=g,
                                      dtype=torch.int32).bfloat16()
            K[:, :, n // 2, 0] = K[:, :, n // 2 - 1, 0]
        q, K, V, out, lse = run_window(sd, *case, scale=scale, prep=spoil)
        see = visible(torch.arange(n - m, n, device="cuda"), n, window, 3, "cuda")
        for h in range(2):
            z = K[0, h, :, 0].double().expand(m, -1).masked_fill(~see, -math.inf)
            top = z.amax(-1, keepdim=True)
            w = (z == top).double()
            count = w.sum(-1, keepdim=True)
            ref, size = w @ V[0, h].double() / count, w @ V[0, h].double().abs() / count
            check(out[0, 4 * h:4 * h + 4], ref.expand(4, -1, -1),
                  (2.0 ** -8 * (ref.abs() + size) + 2.0 ** -20 * size + 1e-30).expand(4, -1, -1),
                  "out")
            want = (top * scale + torch.log(count))[:, 0]
            check(lse[0, 4 * h:4 * h + 4], want.expand(4, -1),
                  (8 * 2.0 ** -24 * want.abs() + 2.0 ** -18).expand(4, -1), "lse")


def test_window_repeats_and_graph(sd):
    """The same bits again, from another workspace's contents and from a replayed graph."""
    for case in ((2, 2, 4, 3000, 3000, 1, 2999, None, None, 2900, 0),
                 (1, 1, 4, 3000, 3000, 300, 2700, None, None, 3000, 0)):
        a = run_window(sd, *case, ws_fill=0)
        b = run_window(sd, *case, ws_fill=255)
        assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])
        B, hkv, G, n, cap, m, first = case[:7]
        shape = sd.make_shape(B, hkv * G, hkv, n)
        ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, m, case[9], 0)),
                         dtype=torch.uint8, device="cuda")
        q, K, V = a[:3]
        out, lse = torch.zeros_like(a[3]), torch.zeros_like(a[4])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                sd.sd_window_attend(shape, q, K, V, m, case[9], 0, SCALE, out, lse, ws,
                                    first=first)
        for _ in range(3):
            out.zero_()
            lse.zero_()
            g.replay()
            assert torch.equal(out, a[3]) and torch.equal(lse, a[4])


@pytest.mark.parametrize("off", [0, 16])
def test_bases_on_16_bytes(sd, off):
    """Inputs, outputs and workspaces that start on 16 bytes and no more."""
    def at16(shape, dtype, fill=None):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        raw = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        skip = off - raw.data_ptr() % 256 + 256
        x = raw[skip:skip + n].view(dtype).view(shape)
        assert x.data_ptr() % 256 == off
        if fill is not None:
            x.copy_(fill)
        return x
    B, hkv, G, n, window = 1, 2, 4, 3000, 2900
    hq = hkv * G
    K, V = (at16((B, hkv, n, D), torch.bfloat16, normal((B, hkv, n, D), s)) for s in (1, 2))
    shape = sd.make_shape(B, hq, hkv, n)
    for m in (1, 20, 300):
        q = at16((B, hq, m, D), torch.bfloat16, normal((B, hq, m, D), 3))
        out, lse = at16((B, hq, m, D), torch.bfloat16), at16((B, hq, m), torch.float32)
        ws = at16((max(16, sd.sd_window_attend_workspace_size(shape, m, window)),), torch.uint8)
        sd.sd_window_attend(shape, q, K, V, m, window, 0, SCALE, out, lse, ws, first=n - m)
        check_window((B, hkv, G, n, n, m, n - m, None, None, window, 0), (q, K, V, out, lse))
    p, own = 1500, 40
    q = at16((B, hq, D), torch.bfloat16, normal((B, hq, D), 4))
    out, lse = at16((B, hq, D), torch.bfloat16), at16((B, hq), torch.float32)
    Kp, Vp = (at16((hkv, p, D), torch.bfloat16, normal((hkv, p, D), s)) for s in (5, 6))
    Ko, Vo = (at16((B, hkv, own, D), torch.bfloat16, normal((B, hkv, own, D), s)) for s in (7, 8))
    shape = sd.make_shape(B, hq, hkv, own)
    ws = at16((max(16, sd.sd_prefix_attend_workspace_size(shape, p)),), torch.uint8)
    sd.sd_prefix_attend(shape, q, Kp, Vp, p, Ko, Vo, SCALE, out, lse, ws)
    check_prefix((B, hkv, G, p, p, own, own, None), (q, Kp, Vp, Ko, Vo, out, lse))


@pytest.mark.parametrize("fallback", [False, True])
def test_without_clusters(sd, fallback):
    """Single tokens and own tokens joined in clusters, and by a kernel of their own."""
    prev = sd.sd_set_fallback_paths(fallback)
    try:
        for case in ((1, 2, 4, 5000, 5000, 1, 4999, None, None, 4000, 100),
                     (3, 1, 8, 700, 700, 1, 0, [699, 3, 350], None, 700, 0)):
            check_window(case, run_window(sd, *case))
        for case in ((2, 2, 4, 700, 700, 900, 900, [900, 17]), (1, 1, 1, 0, 0, 4000, 4000, None)):
            check_prefix(case, run_prefix(sd, *case))
    finally:
        sd.sd_set_fallback_paths(prev)


# ---- shared prefix -------------------------------------------------------------------------
PREFIX = [
    # B, hkv, G, p, p_cap, n, n_cap, end
    (1, 1, 1, 1, 1, 1, 1, None),
    (2, 2, 4, 100, 128, 30, 40, [30, 0]),
    (3, 1, 8, 0, 0, 50, 50, [50, 0, 7]),
    (5, 2, 2, 1000, 1001, 1, 1, None),
    (17, 4, 8, 777, 800, 333, 333, [(19 * i) % 334 for i in range(17)]),
    (64, 2, 4, 2049, 2049, 100, 128, [(7 * i) % 101 for i in range(64)]),
    (33, 1, 4, 128, 128, 5, 5, [-1] * 33),
    (130, 1, 2, 3001, 3001, 16, 16, None),
    (4, 8, 4, 20000, 20000, 700, 700, [700, 1, 0, 699]),
    (2, 1, 1, 129, 129, 5000, 5000, [5000, 4999]),
    (9, 2, 8, 500, 500, 0, 0, None),
    (3, 1, 1, 40000, 40000, 3, 3, [3, 0, 1]),
]


def run_prefix(sd, B, hkv, G, p, pcap, n, cap, end, seed=0, prep=None, ws_fill=255):
    hq = hkv * G
    q = normal((B, hq, D), seed)
    Kp, Vp = (normal((hkv, max(pcap, 1), D), seed + j) for j in (1, 2))
    Kp[:, p:], Vp[:, p:] = math.nan, math.nan
    K = V = None
    if n:
        K, V = normal((B, hkv, cap, D), seed + 3), normal((B, hkv, cap, D), seed + 4)
        for b in range(B):
            e = n if end is None else max(0, min(n, end[b]))
            K[b, :, e:], V[b, :, e:] = math.nan, math.inf
    if prep:
        prep(q, Kp, Vp, K, V)
    out = torch.full((B, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, hq), 7.0, device="cuda")
    shape = sd.make_shape(B, hq, hkv, max(n, 1), D, max(cap, 1))
    ws = torch.full((max(16, sd.sd_prefix_attend_workspace_size(shape, p)),), ws_fill,
                    dtype=torch.uint8, device="cuda")
    sd.sd_prefix_attend(shape, q, Kp if p else None, Vp if p else None, p, K, V, SCALE, out, lse,
                        ws, end=i32(end), p_cap=pcap)
    sd.sd_device_status()
    return q, Kp, Vp, K, V, out, lse


def check_prefix(case, got):
    B, hkv, G, p, pcap, n, cap, end = case
    q, Kp, Vp, K, V, out, lse = got
    for b in range(B):
        e = 0 if n == 0 else n if end is None else max(0, min(n, end[b]))
        for h in range(hkv):
            k, v = Kp[h, :p], Vp[h, :p]
            if e:
                k, v = torch.cat((k, K[b, h, :e])), torch.cat((v, V[b, h, :e]))
            rows = slice(h * G, (h + 1) * G)
            see = torch.ones((G, k.shape[0]), dtype=torch.bool, device="cuda")
            o, l, tol, ltol = attention(q[b, rows], k, v, see, SCALE)
            check(out[b, rows], o, tol, f"out of ({b}, {h})")
            check(lse[b, rows], l, ltol, f"lse of ({b}, {h})")


@pytest.mark.parametrize("case", PREFIX, ids=range(len(PREFIX)))
def test_prefix(sd, case):
    check_prefix(case, run_prefix(sd, *case))


def test_prefix_wide_scores(sd):
    """Own tokens whose scores tower over the prefix's, and the other way round."""
    def spoil(q, Kp, Vp, K, V):
        q[..., 0] = 30.0
        Kp[..., 0] = 0.0
        K[..., 0] = 0.0
        K[0, :, :, 0] = 40.0
        Kp[1, :, 0] = 40.0
    case = (3, 2, 4, 600, 600, 50, 50, None)
    check_prefix(case, run_prefix(sd, *case, prep=spoil))


def test_prefix_repeats(sd):
    case = PREFIX[8]
    a, b = run_prefix(sd, *case, ws_fill=0), run_prefix(sd, *case, ws_fill=255)
    assert torch.equal(a[5], b[5]) and torch.equal(a[6], b[6])


def test_prefix_equals_window_on_the_same_tokens(sd):
    """A batch of one: prefix and own tokens laid in one cache under the causal window."""
    B, hkv, G, p, n = 1, 2, 4, 1500, 200
    got = run_prefix(sd, B, hkv, G, p, p, n, n, None)
    q, Kp, Vp, K, V, out, lse = got
    cache = [torch.cat((a[None], b), 2).contiguous() for a, b in ((Kp, K), (Vp, V))]
    shape = sd.make_shape(B, hkv * G, hkv, p + n)
    o, l = torch.zeros_like(out).unsqueeze(2), torch.zeros_like(lse).unsqueeze(2)
    ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, 1, p + n, 0)),
                     dtype=torch.uint8, device="cuda")
    sd.sd_window_attend(shape, q.unsqueeze(2), *cache, 1, p + n, 0, SCALE, o, l, ws,
                        first=p + n - 1)
    assert (o.squeeze(2).float() - out.float()).abs().max() <= 2.0 ** -6
    assert (l.squeeze(2) - lse).abs().max() <= 1e-4


def test_prefix_graph_and_no_lse(sd):
    """A captured call follows new values in its inputs; without lse out is the same."""
    case = (6, 2, 4, 2500, 2500, 300, 300, [300, 0, 17, 299, 150, 1])
    B, hkv, G, p, pcap, n, cap, end = case
    q, Kp, Vp, K, V, out, lse = run_prefix(sd, *case)
    shape, ends = sd.make_shape(B, hkv * G, hkv, n), i32(end)
    ws = torch.empty(sd.sd_prefix_attend_workspace_size(shape, p), dtype=torch.uint8,
                     device="cuda")
    o1, o2, l2 = torch.zeros_like(out), torch.zeros_like(out), torch.zeros_like(lse)
    sd.sd_prefix_attend(shape, q, Kp, Vp, p, K, V, SCALE, o1, None, ws, end=ends)
    assert torch.equal(o1, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            sd.sd_prefix_attend(shape, q, Kp, Vp, p, K, V, SCALE, o2, l2, ws, end=ends)
            sd.sd_prefix_attend(shape, q, Kp, Vp, p, K, V, SCALE, o2, l2, ws, end=ends)
    for seed in (1, 2):
        q.copy_(normal((B, hkv * G, D), 90 + seed))
        ends.copy_(i32([(seed * 71 + 50 * b) % 301 for b in range(B)]))
        K.copy_(normal(K.shape, 95 + seed))
        V.copy_(normal(V.shape, 97 + seed))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_prefix((B, hkv, G, p, pcap, n, cap, ends.tolist()), (q, Kp, Vp, K, V, o2, l2))


FIRST = """
import torch, top_sparse_decode_gb300 as sd
bf = dict(dtype=torch.bfloat16, device="cuda")
B, hkv, G, n, m = 2, 2, 4, 3000, {m}
hq, shape = hkv * G, sd.make_shape(2, 8, 2, 3000)
x = torch.randn((B, hq + 2 * hkv, m, 128), device="cuda").bfloat16()
q, k, v = x.split([hq, hkv, hkv], dim=1)
K, V = torch.zeros((B, hkv, n, 128), **bf), torch.zeros((B, hkv, n, 128), **bf)
w, f = torch.ones(128, device="cuda"), torch.rand(64, device="cuda", dtype=torch.float64)
rope = sd.make_rope(f, w, w)
ws = torch.zeros(max(16, sd.sd_window_attend_workspace_size(shape, m, n),
                     sd.sd_prefix_attend_workspace_size(shape, n)), dtype=torch.uint8,
                 device="cuda")
qo, out = torch.zeros((B, hq, m, 128), **bf), torch.zeros((B, hq, m, 128), **bf)
q1, o1 = torch.randn((B, hq, 128), device="cuda").bfloat16(), torch.zeros((B, hq, 128), **bf)
l1 = torch.zeros((B, hq), device="cuda")
def calls():
    sd.sd_qk_norm_rope(shape, rope, q, qo, k, v, K, V, m, first=n - m)
    sd.sd_window_attend(shape, qo, K, V, m, n, 0, 0.09, out, None, ws, first=n - m)
    sd.sd_prefix_attend(shape, q1, K[0], V[0], n, K, V, 0.09, o1, l1, ws)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
a = out.clone(), o1.clone(), l1.clone(), K.clone()
for y in (out, o1, l1):
    y.zero_()
calls()
torch.cuda.synchronize()
assert all(torch.equal(s, t) for s, t in zip(a, (out, o1, l1, K))) and out.abs().max() > 0
sd.sd_device_status()
print("captured first")
"""


@pytest.mark.parametrize("m", [1, 150])
def test_first_calls_captured(sd, m):
    """The very first calls of a process are made inside a capture."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(m=m)], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def test_two_streams(sd):
    """Calls that run beside each other, each with its own workspace."""
    case = (2, 2, 4, 2500, 2500, 200, 2300, None, None, 2400, 0)
    want = run_window(sd, *case)
    B, hkv, G, n, cap, m, first = case[:7]
    shape = sd.make_shape(B, hkv * G, hkv, n)
    outs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for st in streams * 4:
        with torch.cuda.stream(st):
            out, lse = torch.zeros_like(want[3]), torch.zeros_like(want[4])
            ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, m, 2400)),
                             dtype=torch.uint8, device="cuda")
            sd.sd_window_attend(shape, *want[:3], m, 2400, 0, SCALE, out, lse, ws, first=first)
            outs.append((out, lse, ws))
    torch.cuda.synchronize()
    for out, lse, _ in outs:
        assert torch.equal(out, want[3]) and torch.equal(lse, want[4])


def test_caches_past_32_bits(sd):
    """The last sequence of caches of more than 2^31 values: written, attended by many tokens
    and by one, and as a prefix's own tokens."""
    B, hkv, G, n, m = 17, 8, 1, 131072, 40
    shape = sd.make_shape(B, hkv, hkv, n)
    K, V = (torch.zeros((B, hkv, n, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert K.numel() > 1 << 31
    K[-1, -1], V[-1, -1] = normal((n, D), 1), normal((n, D), 2)
    q, k, v = (normal((B, hkv, m, D), s) for s in (3, 4, 5))
    w, freq = torch.ones(D, device="cuda"), torch.rand(64, device="cuda", dtype=torch.float64)
    qo, first = torch.zeros_like(q), n - m
    sd.sd_qk_norm_rope(shape, sd.make_rope(freq, w, w), q, qo, k, v, K, V, m, first=first)
    r = torch.arange(first, n, device="cuda")
    ref = norm_rope(k[-1, -1], w, 1e-6, r, freq, 128, False)
    check(K[-1, -1, first:], ref, norm_rope_tol(ref, k[-1, -1], w, 1e-6, r, freq, 128, False), "K")
    assert torch.equal(V[-1, -1, first:], v[-1, -1])
    for t, window in ((m, 600), (m, n), (1, n)):
        out, lse = torch.zeros_like(q[:, :, :t]), torch.zeros((B, hkv, t), device="cuda")
        ws = torch.empty(max(16, sd.sd_window_attend_workspace_size(shape, t, window, 4)),
                         dtype=torch.uint8, device="cuda")
        x = qo[:, :, m - t:].contiguous()
        sd.sd_window_attend(shape, x, K, V, t, window, 4, SCALE, out, lse, ws, first=n - t)
        p = torch.arange(n - t, n, device="cuda")
        o, e, tol, ltol = attention(x[-1, -1], K[-1, -1], V[-1, -1],
                                    visible(p, n, window, 4, "cuda"), SCALE)
        check(out[-1, -1], o, tol, "out")
        check(lse[-1, -1], e, ltol, "lse")
    sd.sd_device_status()


# ---- together ------------------------------------------------------------------------------
def test_prompt_then_decode(sd):
    """A prompt goes through norm, rotation and window attention in chunks, then tokens one at
    a time, on a side stream; every step's result equals the 64-bit attention over the rows
    that the cache holds."""
    B, hkv, G, n, window, sink = 2, 2, 4, 420, 100, 8
    hq = hkv * G
    shape = sd.make_shape(B, hq, hkv, n)
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    w = torch.ones(D, device="cuda")
    rope = sd.make_rope(freq, w, w)
    K, V = (torch.zeros((B, hkv, n, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    need = max(sd.sd_window_attend_workspace_size(shape, m, window, sink) for m in (1, 150, 250))
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    at, steps = 0, [150, 250] + [1] * 20
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for j, m in enumerate(steps):
        with torch.cuda.stream(side):
            x = normal((B, m, hq + 2 * hkv, D), j).transpose(1, 2)
            q, k, v = x.split([hq, hkv, hkv], dim=1)
            qo, out = (torch.zeros((B, hq, m, D), dtype=torch.bfloat16, device="cuda")
                       for _ in range(2))
            lse = torch.zeros((B, hq, m), device="cuda")
            pos = i32([at, at])
            sd.sd_qk_norm_rope(shape, rope, q, qo, k, v, K, V, m, pos=pos)
            sd.sd_window_attend(shape, qo, K, V, m, window, sink, SCALE, out, lse, ws, pos=pos)
        side.synchronize()
        r = torch.arange(at, at + m, device="cuda")
        kr = norm_rope(k, w, 1e-6, r, freq, 128, False)
        check(K[:, :, at:at + m], kr, norm_rope_tol(kr, k, w, 1e-6, r, freq, 128, False), "K")
        at += m
        check_window((B, hkv, G, n, n, m, at - m, None, None, window, sink),
                     (qo, K, V, out, lse))
