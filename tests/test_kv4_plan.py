"""The rule that picks the kernel for attention over a 4-bit K/V cache (sd_kv4_plan.cuh),
compiled for the host: what it picks on a whole GB300, and that it asks for no cluster that
the GPU cannot run."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "top_sparse_decode_gb300", "csrc")
SMS = 152


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cc", d / "plan.so"
    src.write_text('#include "sd_kv4_plan.cuh"\n'
                   'extern "C" int pick(long long rows, long long tiles, int sms, int most) {\n'
                   '  return sd::kv4_cluster_of(rows, tiles, sms, most);\n}\n')
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                    f"-I{CSRC}", str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).pick
    fn.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    fn.restype = ctypes.c_int
    return fn


def test_measured_sizes(pick):
    """The sizes whose two times the rule was set by (tokens per row -> 32-token tiles)."""
    for rows, n, cluster in ((8, 8192, True), (8, 16384, False), (128, 4096, True),
                             (128, 16384, False), (512, 128, True), (512, 2064, False)):
        assert (pick(rows, -(-n // 32), SMS, 8) > 0) == cluster, (rows, n)
    assert pick(1, 128, SMS, 8) == 8
    assert pick(512, 4, SMS, 8) == 1


@pytest.mark.parametrize("sms", [152, 76, 20, 1])
def test_no_larger_cluster_than_the_gpu_runs(pick, sms):
    for most in (0, 1, 2, 4, 8):
        for rows in (1, 2, 7, 19, 38, 76, 152, 304, 512, 65535):
            for tiles in (0, 1, 3, 16, 128, 129, 1024, 32768, 1 << 26):
                c = pick(rows, tiles, sms, most)
                assert c in (0, 1, 2, 4, 8) and c <= most, (rows, tiles, sms, most, c)
                assert c <= 1 or rows * c <= 2 * sms  # all CTAs of a joined row at once
    assert pick(1, 1, sms, 1) == 1 and pick(1, 1, sms, 0) == 0
