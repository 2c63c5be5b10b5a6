"""The 4-bit K/V cache's plain implementation against its definition, and the refusals of
the sd_kv4_* entry points.  No GPU: every library call here is rejected on the host."""
import ctypes

import numpy as np
import pytest

import _kv4 as kv


@pytest.fixture(scope="module")
def sd():
    from top_sparse_decode_gb300 import build as b
    b.build()
    import top_sparse_decode_gb300 as sdmod
    sdmod.lib()
    return sdmod


def test_pack_follows_the_words():
    c = (np.arange(128) * 7 % 16).astype(np.uint8)
    words = kv.pack(c.reshape(2, 64)).view("<u4")
    for w in range(16):
        for i in range(8):
            assert (words[w] >> (4 * i)) & 15 == c[64 * (w % 2) + 8 * (w // 2) + i]
    assert np.array_equal(kv.unpack(kv.pack(c.reshape(2, 64))).reshape(-1), c)


def test_error_is_within_the_stated_bound():
    rng = np.random.default_rng(3)
    x = kv.tokens(rng, (4000,))
    c, s, m = kv.quantise(x)
    err = np.abs((c * s[..., None].astype(np.float64) + m[..., None]).reshape(-1, 128) -
                 kv.bf16_val(x))
    bound = np.repeat(s * (0.5 + 15 * 2.0 ** -8), 64, -1)
    assert np.all(err <= bound * (1 + 1e-6))
    assert c.min() == 0 and c.max() == 15


def test_special_groups():
    x = np.zeros((5, 128), np.float32)
    x[0, :] = 3.0                      # constant: exact
    x[1, 5] = np.nan                   # group 0 of row 1
    x[2, 100] = np.inf                 # group 1 of row 2
    x[3, 0], x[3, 1] = 3e38, -3e38     # max - m overflows
    x[4, 7] = 1e-30                    # a step below 2^-100: the minimum
    c, s, m = kv.quantise(kv.bf16_bits(x))
    assert (s[0] == 0).all() and (m[0] == 3).all() and (c[0] == 0).all()
    assert np.isnan(s[1, 0]) and s[1, 1] == 0
    assert np.isnan(s[2, 1]) and s[2, 0] == 0
    assert np.isnan(s[3, 0]) and (s[4] == 0).all() and (c[4] == 0).all()


def test_ties_go_to_even():
    # m = 0, max = 15 (s = 1): 0.5 -> 0, 1.5 -> 2, 2.5 -> 2, 14.5 -> 14
    x = np.zeros(128, np.float32)
    x[:5] = [15, 0.5, 1.5, 2.5, 14.5]
    c, s, _ = kv.quantise(kv.bf16_bits(x))
    assert s[0] == 1 and c[0, :5].tolist() == [15, 0, 2, 2, 14]


P = 1 << 20  # a fake, aligned address; never dereferenced


def test_move_refusals(sd):
    lib = sd.lib()
    cache = sd._abi.SdKv4(P, P, P)
    shp = sd.make_shape(2, 8, 2, 1000)
    S = sd._abi.SdStrides

    for fn in (lib.sd_kv4_write, lib.sd_kv4_read):
        def call(shape=shp, c=cache, K=P, ks=None, V=P, vs=None, m=10, first=0, pos=None,
                 length=None):
            return fn(ctypes.byref(shape), ctypes.byref(c) if c is not None else None, K,
                      ctypes.byref(ks) if ks is not None else None, V,
                      ctypes.byref(vs) if vs is not None else None, m, first, pos, length, None)
        bad = [dict(c=None), dict(c=sd._abi.SdKv4(P, None, P)), dict(c=sd._abi.SdKv4(P + 8, P, P)),
               dict(c=sd._abi.SdKv4(P, P, P + 2)), dict(K=None, V=None), dict(K=P + 2),
               dict(V=P + 8), dict(m=-1), dict(m=1 << 31), dict(first=-1), dict(first=1001),
               dict(pos=P + 1), dict(length=P + 2), dict(ks=S(20480, 10240, 130)),
               dict(vs=S(20480, -10240, 128)), dict(ks=S(1 << 40, 10240, 128))]
        for kw in bad:
            assert call(**kw) == sd.SD_ERR_INVALID_ARG, (fn.__name__, kw)
            assert sd.sd_last_error()
        assert call(shape=sd.make_shape(2, 8, 2, 1000, d=64)) == sd.SD_ERR_UNSUPPORTED
        assert call(m=0) == sd.SD_OK  # nothing to move, nothing launched
    # outputs whose rows overlap
    for st in (S(0, 1280, 128), S(2560, 1280, 120), S(2560, 0, 128), S(2560, 1272, 128)):
        assert lib.sd_kv4_read(ctypes.byref(shp), ctypes.byref(cache), P, ctypes.byref(st), None,
                               None, 10, 0, None, None, None) == sd.SD_ERR_INVALID_ARG


def test_attend_refusals(sd):
    lib = sd.lib()
    cache = sd._abi.SdKv4(P, P, P)
    shp = sd.make_shape(2, 8, 2, 1000)
    need = lib.sd_kv4_attend_workspace_size(ctypes.byref(shp))
    gneed = lib.sd_kv4_gather_attend_workspace_size(ctypes.byref(shp), 64)

    def att(shape=shp, q=P, c=cache, b=None, e=None, out=P, lse=P, ws=P, nb=need):
        return lib.sd_kv4_attend(ctypes.byref(shape), q, ctypes.byref(c) if c else None, b, e,
                                 0.1, out, lse, ws, nb, None)

    def gat(q=P, c=cache, idx=P, stride=64, count=P, mc=64, out=P, lse=P, ws=P, nb=gneed):
        return lib.sd_kv4_gather_attend(ctypes.byref(shp), q, ctypes.byref(c) if c else None, idx,
                                        stride, count, mc, 0.1, out, lse, ws, nb, None)

    for kw in (dict(c=None), dict(c=sd._abi.SdKv4(None, P, P)), dict(q=None), dict(out=None),
               dict(q=P + 2), dict(out=P + 4), dict(lse=P + 2), dict(ws=P + 4)):
        assert att(**kw) == sd.SD_ERR_INVALID_ARG, kw
        assert gat(**kw) == sd.SD_ERR_INVALID_ARG, kw
    assert att(b=P + 2) == att(e=P + 1) == sd.SD_ERR_INVALID_ARG
    assert att(shape=sd.make_shape(2, 6, 2, 1000)) == sd.SD_ERR_UNSUPPORTED
    for kw in (dict(idx=None), dict(count=None), dict(stride=63), dict(mc=-1), dict(idx=P + 2),
               dict(count=P + 2), dict(mc=1 << 31, stride=1 << 31)):
        assert gat(**kw) == sd.SD_ERR_INVALID_ARG, kw
    for n in (need, gneed):
        assert n > 0
    assert att(nb=need - 1) == att(ws=None) == sd.SD_ERR_WORKSPACE
    assert gat(nb=gneed - 1) == gat(ws=None) == sd.SD_ERR_WORKSPACE
    assert lib.sd_kv4_attend_workspace_size(ctypes.byref(sd.make_shape(1, 3, 1, 8))) == 0
    assert lib.sd_kv4_gather_attend_workspace_size(ctypes.byref(shp), -1) == 0


def test_binding_refusals(sd):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):  # sizes that do not match
        sd.Kv4Cache(1, 2, 64, device="cpu", k=torch.zeros((1, 2, 63, 64), dtype=torch.uint8))
    cache = sd.Kv4Cache(1, 2, 64, device="cpu")
    shp = sd.make_shape(1, 2, 2, 64)
    K = torch.zeros((1, 2, 8, 128), dtype=torch.bfloat16)
    for bad in (K[:, :1], K[:, :, :7], torch.zeros((1, 2, 8, 256))[..., ::2], K[..., :64]):
        with pytest.raises(ValueError):
            sd.sd_kv4_write(shp, cache, bad, K, 8, stream=0)
        with pytest.raises(ValueError):
            sd.sd_kv4_read(shp, cache, K, bad, 8, stream=0)


def test_binding_refuses_a_shape_beside_the_cache(sd):
    torch = pytest.importorskip("torch")
    cache = sd.Kv4Cache(2, 2, 64, device="cpu")
    K = torch.zeros((2, 2, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(64, dtype=torch.int32)
    for dims in ((3, 4, 2, 64), (2, 4, 1, 64), (2, 4, 4, 64), (2, 4, 2, 63), (2, 4, 2, 128),
                 (2, 4, 2, 64, 128, 65)):
        shp = sd.make_shape(*dims)
        rows = K.new_zeros((dims[0], dims[2], 8, 128))
        for call in (lambda: sd.sd_kv4_write(shp, cache, rows, rows, 8, stream=0),
                     lambda: sd.sd_kv4_read(shp, cache, rows, rows, 8, stream=0),
                     lambda: sd.sd_kv4_attend(shp, K, cache, 0.1, K, stream=0),
                     lambda: sd.sd_kv4_gather_attend(shp, K, cache, i, 64, i, 64, 0.1, K,
                                                     stream=0)):
            with pytest.raises(ValueError, match="do not address"):
                call()
    # fewer sequences, and fewer tokens of the same capacity, are addressed (nothing to move)
    for dims in ((1, 4, 2, 64), (2, 4, 2, 60, 128, 64)):
        shp = sd.make_shape(*dims)
        sd.sd_kv4_write(shp, cache, K[:dims[0]], K[:dims[0]], 0, stream=0)


def test_binding_refuses_wide_rows(sd):
    torch = pytest.importorskip("torch")
    cache = sd.Kv4Cache(1, 2, 64, device="cpu")
    K = torch.zeros((1, 2, 8, 128))
    for fn in (sd.sd_kv4_write, sd.sd_kv4_read):
        with pytest.raises(ValueError, match="bf16"):
            fn(sd.make_shape(1, 2, 2, 64), cache, K, K, 8, stream=0)
