"""sd_device_status: a bounded wait that runs out inside a kernel is reported to
the host (SD_ERR_TIMEOUT) and cleared, instead of passing silently.  The report
is raised from the host (sd_debug_set_device_error), never by making a wait run
out on the GPU."""
import numpy as np
import pytest
import torch

import synth
from _helpers import dev, empty

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


def test_status_reports_once_and_clears(sd):
    sd.sd_device_status()  # whatever came before: read and cleared
    sd.sd_debug_set_device_error()
    with pytest.raises(sd.SdError) as e:
        sd.sd_device_status()
    assert e.value.code == sd.SD_ERR_TIMEOUT
    assert "incomplete" in str(e.value)
    sd.sd_device_status()  # cleared by the report


@pytest.mark.parametrize("scan", [False, True])
def test_status_of_the_tile_attention(sd, scan):
    """The window and prefix attention's word: reported by its own message, alone or with the
    scans', and cleared with it; the calls behind it run."""
    sd.sd_device_status()
    stream = torch.cuda.Stream()
    sd.sd_debug_set_tile_error(stream)
    if scan:
        sd.sd_debug_set_device_error()
    with pytest.raises(sd.SdError) as e:
        sd.sd_device_status()
    assert e.value.code == sd.SD_ERR_TIMEOUT
    assert "window or prefix attention" in str(e.value) and "incomplete" in str(e.value)
    assert ("so did a bit-plane scan" in str(e.value)) == scan
    sd.sd_device_status()  # both cleared
    q, K, V = (torch.ones((1, 2, 70, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    out = torch.zeros_like(q)
    sd.sd_window_attend(sd.make_shape(1, 2, 2, 70), q, K, V, 70, 70, 0, 0.0, out)
    sd.sd_device_status()
    assert (out == 1).all()


def test_status_clean_after_scans(sd):
    cfg = synth.config(2, B=1, n=8192)
    inp = synth.make_inputs(cfg, with_v=False)
    shp = sd.make_shape(cfg.B, cfg.Hq, cfg.Hkv, cfg.n)
    K, q, s2 = dev(inp.K), dev(inp.q), dev(inp.sigma2)
    planes = empty((cfg.B, cfg.Hkv, 128, 4, cfg.n // 32), np.uint32)
    scales = empty((cfg.B, cfg.Hkv, 128, cfg.n // 64), np.uint16)
    sd.sd_build_index(sd.SD_IDX_PLANES, shp, K, None, planes, scales)
    plan = empty((cfg.B, cfg.Hkv, 128), np.uint8)
    scores = empty((cfg.B * cfg.Hkv, cfg.n), np.float32)
    for fallback in (False, True):
        prev = sd.sd_set_fallback_paths(fallback)
        try:
            sd.sd_plan_score(shp, planes, scales, q, s2, sd.SD_PLAN_WATERFILL, 56, plan, scores)
            sd.sd_device_status()
        finally:
            sd.sd_set_fallback_paths(prev)
