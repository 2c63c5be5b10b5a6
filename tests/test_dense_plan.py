"""The rules that cut attention over the bf16 cache into work (sd_dense_plan.cuh), compiled
for the host: every cut covers its work, fits its workspace, and leaves no SM without a part
where there is work for it."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "top_sparse_decode_gb300", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cc", d / "plan.so"
    src.write_text('#include "sd_dense_plan.cuh"\n'
                   'extern "C" void tile(long long h, long long r, long long k, int sms, int own, '
                   'long long* o) {\n  auto p = sd::dt_plan(h, r, k, sms, own != 0);\n'
                   '  o[0] = p.dual, o[1] = p.per, o[2] = p.splits, o[3] = p.items;\n}\n'
                   'extern "C" void stream(long long r, long long t, int sms, int most, '
                   'long long* o) {\n  auto p = sd::sw_plan(r, t, sms, most);\n'
                   '  o[0] = p.parts, o[1] = p.cut, o[2] = sd::sw_cut(r, t, sms);\n}\n')
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                    f"-I{CSRC}", str(src), "-o", str(lib)], check=True)
    dll = ctypes.CDLL(str(lib))
    ll = ctypes.c_longlong
    dll.tile.argtypes = [ll, ll, ll, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ll)]
    dll.stream.argtypes = [ll, ll, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ll)]

    def call(fn, n, *args):
        out = (ll * n)()
        fn(*args, out)
        return list(out)
    return (lambda *a: call(dll.tile, 4, *a)), (lambda *a: call(dll.stream, 3, *a))


def test_early_kernels_use_ordinary_loads():
    """Kernels that are launched while their producer runs (dn_wait_prior) make no read-only
    loads: those are not ordered by the wait."""
    early = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        if "dn_wait_prior" in code:
            early.append(name)
            assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code), name
    assert {"sd_dense.cuh", "sd_dense_stream.cu", "sd_dense_tile.cu"} <= set(early)


@pytest.mark.parametrize("sms", [1, 20, 152])
@pytest.mark.parametrize("own", [0, 1])
def test_tile_cut(plan, sms, own):
    tile, _ = plan
    for heads in (1, 2, 8, 512, 65535):
        for rows in (1, 4, 128, 129, 256, 257, 5000, 131072 * 8):
            for keys in (1, 128, 129, 4300, 131072, (1 << 31) - 1):
                dual, per, splits, items = tile(heads, rows, keys, sms, own)
                assert dual == (rows <= 128)
                size = 128 if dual else 256
                assert (per - 1) * size < rows <= per * size
                assert items == heads * per * splits and 1 <= splits <= max(1, sms)
                assert splits == 1 or items <= sms
                # a split has token tiles for both softmax groups
                least = 2 if not own else 8 if dual else 4
                assert splits == 1 or splits * least <= -(-keys // 128) + 1
                # tiles times splits stay in 32 bits
                assert (-(-keys // 128) + 2) * (splits + 1) < 1 << 32


@pytest.mark.parametrize("sms", [1, 20, 152])
@pytest.mark.parametrize("most", [0, 1, 2, 4, 8])
def test_stream_cut(plan, sms, most):
    _, stream = plan
    for rows in (1, 3, 8, 64, 304, 512, 65535):
        for tokens in (0, 1, 16, 17, 1152, 4224, 131072, (1 << 31) - 1):
            parts, cut, most_parts = stream(rows, tokens, sms, most)
            assert 1 <= parts and most_parts >= 1
            if cut:  # the workspace holds what sw_cut says
                assert parts == most_parts > 1
            else:
                assert parts in (1, 2, 4, 8) and (parts == 1 or parts <= most)
            assert most_parts == 1 or rows * most_parts <= 2 * sms


def test_stream_measured_sizes(plan):
    """A GB300's 152 SMs: few rows of a window join in clusters, a long row of few in a kernel
    of its own, many rows alone or in pairs."""
    _, stream = plan
    assert stream(8, 1152, 152, 8)[:2] == [8, 0]
    assert stream(8, 32768, 152, 8)[1] == 1
    assert stream(512, 333, 152, 8)[1] == 0
