"""Refusals of sd_qk_norm_rope, sd_window_attend and sd_prefix_attend: nothing here reaches
CUDA."""
import ctypes

import pytest
import torch

P = 1 << 20  # a fake, aligned address; never dereferenced


@pytest.fixture(scope="module")
def sd():
    from top_sparse_decode_gb300 import build as b
    b.build()
    import top_sparse_decode_gb300 as m
    m.lib()
    return m


def shape(sd, n=100, cap=0):
    return sd.make_shape(2, 8, 2, n, 128, cap)


def rope_call(sd, shp=None, rope="ok", q=P, qs=None, qo=P, qos=None, k=P, ks=None, v=P, vs=None,
              K=P, V=P, m=4, first=0, pos=P, length=P, rotary=P):
    shp = shp or shape(sd)
    if rope == "ok":
        rope = sd._abi.SdRope(P, P, P, 1e-6, 128, 0)
    st = [None if s is None else ctypes.byref(sd._abi.SdStrides(*s)) for s in (qs, qos, ks, vs)]
    return sd.lib().sd_qk_norm_rope(ctypes.byref(shp), None if rope is None else
                                    ctypes.byref(rope), q, st[0], qo, st[1], k, st[2], v, st[3],
                                    K, V, m, first, pos, length, rotary, None)


@pytest.mark.parametrize("kw", [
    dict(rope=None), dict(q=None), dict(qo=None), dict(k=None), dict(K=None), dict(v=None),
    dict(V=None), dict(q=None, qo=None, k=None, K=None, v=None, V=None), dict(q=P + 8),
    dict(qo=P + 2), dict(k=P + 8), dict(v=P + 4), dict(K=P + 8), dict(V=P + 1), dict(pos=P + 2),
    dict(length=P + 1), dict(rotary=P + 3), dict(m=-1), dict(m=1 << 31), dict(first=-1),
    dict(first=101), dict(qs=(4096, 512, 4)), dict(ks=(-8, 128, 128)), dict(vs=(1 << 40, 128, 128)),
    dict(qos=(4096, 512, 0)), dict(qos=(0, 512, 128)), dict(qos=(4096, 128, 128)),
])
def test_rope_refusals(sd, kw):
    assert rope_call(sd, **kw) == sd.SD_ERR_INVALID_ARG, kw
    assert sd.sd_last_error()


@pytest.mark.parametrize("rope", [
    (P, P, P, 1e-6, 8, 0), (P, P, P, 1e-6, -16, 0), (P, P, P, 1e-6, 144, 0),
    (P, P, None, 1e-6, 16, 0), (P, P, P + 4, 1e-6, 16, 0), (P + 4, P, P, 1e-6, 16, 0),
    (P, P + 8, P, 1e-6, 16, 0), (P, P, P, -1e-6, 16, 0), (P, P, P, float("nan"), 16, 0),
    (P, P, P, float("inf"), 16, 0),
])
def test_rope_record_refusals(sd, rope):
    assert rope_call(sd, rope=sd._abi.SdRope(*rope)) == sd.SD_ERR_INVALID_ARG, rope


def test_rope_nothing_to_do(sd):
    assert rope_call(sd, m=0) == sd.SD_OK


def window_call(sd, shp=None, q=P, qs=None, K=P, V=P, m=4, first=0, pos=P, length=P, window=10,
                sink=0, scale=0.1, out=P, os=None, lse=P, ws=P, ws_bytes=1 << 40):
    shp = shp or shape(sd)
    st = [None if s is None else ctypes.byref(sd._abi.SdStrides(*s)) for s in (qs, os)]
    return sd.lib().sd_window_attend(ctypes.byref(shp), q, st[0], K, V, m, first, pos, length,
                                     window, sink, scale, out, st[1], lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(K=None), dict(V=None), dict(out=None), dict(q=P + 8), dict(K=P + 8),
    dict(V=P + 2), dict(out=P + 8), dict(lse=P + 2), dict(pos=P + 1), dict(length=P + 2),
    dict(m=-1), dict(m=1 << 31), dict(first=-1), dict(first=101), dict(window=0),
    dict(window=-5), dict(sink=-1), dict(scale=-0.1), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(qs=(4096, 512, 4)), dict(os=(4096, 512, 0)),
    dict(os=(0, 512, 128)),
])
def test_window_refusals(sd, kw):
    assert window_call(sd, **kw) == sd.SD_ERR_INVALID_ARG, kw


def test_window_sizes(sd):
    assert window_call(sd, m=0) == sd.SD_OK
    assert window_call(sd, m=1 << 28) == sd.SD_ERR_UNSUPPORTED
    assert window_call(sd, shp=sd.make_shape(1, 3, 1, 10)) == sd.SD_ERR_UNSUPPORTED
    # a call that needs a workspace refuses a small or missing one
    big = sd.make_shape(1, 4, 1, 100000)
    need = sd.sd_window_attend_workspace_size(big, 100, 100000)
    if need:
        kw = dict(shp=big, m=100, window=100000)
        assert window_call(sd, ws_bytes=need - 1, **kw) == sd.SD_ERR_WORKSPACE
        assert window_call(sd, ws=None, **kw) == sd.SD_ERR_WORKSPACE
        assert window_call(sd, ws=P + 8, **kw) == sd.SD_ERR_INVALID_ARG
    assert sd.sd_window_attend_workspace_size(big, -1, 10) == 0
    assert sd.sd_window_attend_workspace_size(big, 1, 0) == 0


@pytest.mark.parametrize("scale", [2.4e38, 3.3e38])
def test_scales_without_a_finite_log2_factor(sd, scale):
    # (a workspace of 0 bytes: a call that passed the scale would be refused for that)
    big = dict(shp=sd.make_shape(1, 4, 1, 100000), m=100, window=100000, ws_bytes=0)
    assert window_call(sd, scale=2.2e38, **big) == sd.SD_ERR_WORKSPACE
    assert window_call(sd, scale=scale, **big) == sd.SD_ERR_INVALID_ARG
    assert prefix_call(sd, scale=scale, ws_bytes=0) == sd.SD_ERR_INVALID_ARG
    assert prefix_call(sd, scale=2.2e38, ws_bytes=0) == sd.SD_ERR_WORKSPACE


def prefix_call(sd, shp=None, q=P, Kp=P, Vp=P, p=50, pcap=0, K=P, V=P, end=P, scale=0.1, out=P,
                lse=P, ws=P, ws_bytes=1 << 40):
    shp = shp or shape(sd)
    return sd.lib().sd_prefix_attend(ctypes.byref(shp), q, Kp, Vp, p, pcap, K, V, end, scale, out,
                                     lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(Kp=None), dict(Vp=None), dict(K=None), dict(V=None),
    dict(q=P + 8), dict(out=P + 8), dict(Kp=P + 4), dict(Vp=P + 8), dict(K=P + 8),
    dict(V=P + 8), dict(end=P + 2), dict(lse=P + 1), dict(p=-1), dict(pcap=49),
    dict(scale=-1.0), dict(scale=float("nan")),
])
def test_prefix_refusals(sd, kw):
    assert prefix_call(sd, **kw) == sd.SD_ERR_INVALID_ARG, kw


def test_prefix_sizes(sd):
    assert prefix_call(sd, p=1 << 31) == sd.SD_ERR_UNSUPPORTED
    assert prefix_call(sd, pcap=1 << 31) == sd.SD_ERR_UNSUPPORTED
    need = sd.sd_prefix_attend_workspace_size(shape(sd), 5000)
    if need:
        assert prefix_call(sd, p=5000, ws_bytes=need - 1) == sd.SD_ERR_WORKSPACE
        assert prefix_call(sd, p=5000, ws=None) == sd.SD_ERR_WORKSPACE
        assert prefix_call(sd, p=5000, ws=P + 4) == sd.SD_ERR_INVALID_ARG
    assert sd.sd_prefix_attend_workspace_size(shape(sd), -1) == 0


def test_binding_refuses_what_would_be_misread(sd):
    """Types, ranks and sizes, before an address is taken."""
    shp = sd.make_shape(1, 4, 2, 10)
    bf = dict(dtype=torch.bfloat16)
    q, out = torch.zeros((1, 4, 2, 128), **bf), torch.zeros((1, 4, 2, 128), **bf)
    K = torch.zeros((1, 2, 10, 128), **bf)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)

    def window(**kw):
        a = dict(q=q, K=K, V=K, out=out, lse=None, pos=None, length=None)
        a.update(kw)
        sd.sd_window_attend(shp, a["q"], a["K"], a["V"], 2, 5, 0, 0.1, a["out"], a["lse"], ws,
                            pos=a["pos"], length=a["length"], stream=0)
    for kw in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[:, :, :1]), dict(K=K[:, :, :9]),
               dict(V=K.float()), dict(out=out.float()), dict(lse=torch.zeros(7)),
               dict(lse=torch.zeros(8, dtype=torch.float64)), dict(pos=torch.zeros(1)),
               dict(pos=torch.zeros(1, dtype=torch.int64)),
               dict(length=torch.zeros(0, dtype=torch.int32)),
               dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            window(**kw)
    q1 = torch.zeros((1, 4, 128), **bf)
    pre = torch.zeros((2, 6, 128), **bf)
    for kw in (dict(Kp=pre[:1]), dict(Vp=pre.half()), dict(out=torch.zeros(1, 4, 128)),
               dict(end=torch.zeros(1, dtype=torch.int64)), dict(lse=torch.zeros(3))):
        a = dict(Kp=pre, Vp=pre, out=q1, end=None, lse=None)
        a.update(kw)
        with pytest.raises(ValueError):
            sd.sd_prefix_attend(shp, q1, a["Kp"], a["Vp"], 6, K, K, 0.1, a["out"], a["lse"], ws,
                                end=a["end"], stream=0)
    w, f = torch.ones(128), torch.ones(64, dtype=torch.float64)
    for kw in (dict(inv_freq=f.float()), dict(q_weight=w[:64]), dict(k_weight=w.double()),
               dict(q_weight=torch.ones(256)[::2])):
        a = dict(inv_freq=f, q_weight=w, k_weight=w)
        a.update(kw)
        with pytest.raises(ValueError):
            sd.make_rope(a["inv_freq"], a["q_weight"], a["k_weight"])
    rope = sd.make_rope(f, w, w)
    k = torch.zeros((1, 2, 2, 128), **bf)
    for kw in (dict(q=q.half()), dict(k=k[:, :1]), dict(v=k[:, :, :1]), dict(K=K[:, :, :9]),
               dict(qo=q.float()), dict(pos=torch.zeros(1)),
               dict(rotary=torch.zeros(1, dtype=torch.int64))):
        a = dict(q=q, qo=out, k=k, v=k, K=K, pos=None, rotary=None)
        a.update(kw)
        with pytest.raises(ValueError):
            sd.sd_qk_norm_rope(shp, rope, a["q"], a["qo"], a["k"], a["v"], a["K"], K, 2,
                               pos=a["pos"], rotary=a["rotary"], stream=0)
