"""GPU tests of the 4-bit K/V cache beyond the ordinary sizes and values: calls that are longer
than the cache."""
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
