"""The injection of lost waits belongs to the debug flavour (CPU)."""
import os
import subprocess

import pytest

from speculative_decoding_tree_mask_gb300 import binding as G
from speculative_decoding_tree_mask_gb300 import build as B


def test_release_build_refuses_it():
    B.build()
    assert G.load().spec_debug_inject_lost_wait(None) == G.SPEC_ERR_UNSUPPORTED


@pytest.mark.parametrize("src", ["tree_attn_tc.cu"])
def test_debug_flavour_compiles(tmp_path, src):
    r = subprocess.run([B.nvcc(), *B.ARCH, *B.FLAGS, "-DSPEC_DEBUG", "-I", B.INCLUDE, "-I",
                        B.CSRC, "-c", os.path.join(B.CSRC, src), "-o", str(tmp_path / "x.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
