"""What the Python binding of the 4-bit K/V cache refuses: tensors whose type or size would be
read as something else, or past their end.  No GPU: every call here is refused on the host,
or moves nothing."""
import pytest

torch = pytest.importorskip("torch")

B, H, G, N = 2, 2, 4, 64


@pytest.fixture(scope="module")
def sd():
    from top_sparse_decode_gb300 import build as b
    b.build()
    import top_sparse_decode_gb300 as sdmod
    sdmod.lib()
    return sdmod


@pytest.fixture
def cache(sd):
    return sd.Kv4Cache(B, H, N, device="cpu")


@pytest.fixture
def shp(sd):
    return sd.make_shape(B, H * G, H, N)


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("fn", ["sd_kv4_write", "sd_kv4_read"])
def test_rows(sd, cache, shp, fn):
    call, K = getattr(sd, fn), zeros(B, H, 8, 128)
    n = B * H * 8 * 128
    for bad in (K.half(), K.half().flatten(), K.float().flatten(), K.float().view(B * H, 8, 128),
                K.to(torch.int32), K.view(torch.uint8),            # other types, 256 channels
                zeros(n - 1), zeros(B * H, 7, 128), zeros(B * H, 9, 128), zeros(n + 1, 1)):
        for k, v in ((bad, K), (K, bad), (bad, None)):
            with pytest.raises(ValueError):
                call(shp, cache, k, v, 8, stream=0)
    # other ranks and bit patterns, for a call that moves nothing
    for ok in (K, K.view(torch.int16), K.flatten(), zeros(0), K.view(torch.uint8).flatten(), None):
        call(shp, cache, K, ok, 0, stream=0)


@pytest.mark.parametrize("fn", ["sd_kv4_write", "sd_kv4_read"])
@pytest.mark.parametrize("name", ["pos", "length"])
def test_positions(sd, cache, shp, fn, name):
    K = zeros(B, H, 8, 128)
    i = torch.zeros(2 * B, dtype=torch.int32)
    for bad in (i.long(), i.short(), i.float(), i[:B - 1], i[::2]):
        with pytest.raises(ValueError, match=name):
            getattr(sd, fn)(shp, cache, K, K, 0, stream=0, **{name: bad})
    getattr(sd, fn)(shp, cache, K, K, 0, stream=0, **{name: i})


def test_attend(sd, cache, shp):
    hq = H * G
    q, out, lse = zeros(B, hq, 128), zeros(B, hq, 128, dtype=torch.float32), torch.zeros(B, hq)
    i = torch.zeros(B, dtype=torch.int32)
    idx, cnt = torch.zeros((B * H, 20), dtype=torch.int32), torch.zeros(B * H, dtype=torch.int32)

    def dense(q=q, out=out, lse=lse, begin=i, end=i):
        sd.sd_kv4_attend(shp, q, cache, 0.1, out, lse, None, begin=begin, end=end, stream=0)

    def gather(q=q, out=out, lse=lse, idx=idx, count=cnt, stride=20, mc=16):
        sd.sd_kv4_gather_attend(shp, q, cache, idx, stride, count, mc, 0.1, out, lse, None,
                                stream=0)

    both = [dict(q=q.float()), dict(q=q.half()), dict(q=q[:, :-1]), dict(q=q.view(torch.int16)[1:]),
            dict(out=out.bfloat16()), dict(out=out.double()), dict(out=out[:1]),
            dict(lse=lse.half()), dict(lse=lse[:1]), dict(out=zeros(B, 128, hq, dtype=torch.float32)
                                                          .transpose(1, 2))]
    for kw in both + [dict(begin=i.long()), dict(end=i.long()), dict(begin=i[:1]), dict(end=i[:1])]:
        with pytest.raises(ValueError):
            dense(**kw)
    for kw in both + [dict(idx=idx.long()), dict(count=cnt.long()), dict(count=cnt[1:]),
                      dict(idx=idx[:-1]), dict(idx=idx, stride=22, mc=16), dict(idx=idx.short())]:
        with pytest.raises(ValueError):
            gather(**kw)
    # what is left to the library: no workspace
    for call in (dense, gather, lambda: gather(idx=idx.flatten()[:76]),
                 lambda: dense(q=q.view(torch.int16), begin=None)):
        with pytest.raises(sd.SdError) as e:
            call()
        assert e.value.code == sd.SD_ERR_WORKSPACE


def test_cache_arrays(sd):
    k, s = zeros(B, H, N, 64, dtype=torch.uint8), zeros(B, H, N, 8)
    for kw in (dict(k=k.bool()), dict(v=zeros(B, H, N, 32)), dict(v=zeros(B, H, N, 16, dtype=torch.float32)),
               dict(scale=s.half()), dict(scale=zeros(B, H, N, 4, dtype=torch.float32)),
               dict(k=zeros(B, N, H, 64, dtype=torch.uint8)), dict(scale=zeros(H, B, N, 8)[:, :, :1]),
               dict(scale=zeros(B, N, H, 8)), dict(v=k.to("meta")), dict(scale=s.to("meta"))):
        with pytest.raises(ValueError, match="Kv4Cache"):
            sd.Kv4Cache(B, H, N, device="cpu", **kw)
    sd.Kv4Cache(B, H, N, device="cpu", k=k, v=k.view(torch.int8), scale=s.view(torch.int16))
    sd.Kv4Cache(B, H, N, device="cpu", k=k.flatten(), v=k.flatten().view(torch.int32),
                scale=s.flatten().view(torch.uint8))


def test_workspace_sizes(sd):
    """One size for both calls, whatever n and max_count, and at most what the header says."""
    for b, hq, hkv in ((1, 1, 1), (2, 8, 2), (5000, 16, 2), (65535, 8, 1)):
        size = sd.sd_kv4_attend_workspace_size(sd.make_shape(b, hq, hkv, 1))
        assert 0 < size <= 11_200_000
        for n, mc in ((1, 0), (4096, 7), (2 ** 31 - 1, 2 ** 31 - 1)):
            shp = sd.make_shape(b, hq, hkv, n)
            assert sd.sd_kv4_attend_workspace_size(shp) == size
            assert sd.sd_kv4_gather_attend_workspace_size(shp, mc) == size
