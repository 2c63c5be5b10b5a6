"""Rules that the 4-bit K/V cache's kernels keep and that no run shows reliably, held on their
source."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "top_sparse_decode_gb300", "csrc")


def code(path):
    """A source file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_early_kernels_use_ordinary_loads():
    """Kernels that are launched while their producer runs (griddepcontrol.wait) make no
    read-only loads: those are not ordered by the wait."""
    early = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
             if re.search(r"griddepcontrol\.wait|kv4_wait_prior", code(p))]
    assert any(p.endswith("sd_kv4_attend.cu") for p in early)
    for p in early:
        assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code(p)), p
