"""The built library holds no kernel instantiation that no call launches (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

import fft_spectral_convolution_amd as fno

HALF = ("DF16b", "DF16_")       # bfloat16 and float16 in mangled names


@pytest.mark.parametrize("kernel,mixed", [("k_gn_once_last", {2, 4, 8, 16}), ("k_gn_bwd_once_last", {2, 4, 8})])
def test_spread_group_norm_kernels(kernel, mixed):
    """Vectors a thread may hold, by (x's type, out's or grad_out's): up to 16, `mixed` for 16 bits beside float32."""
    if not os.path.exists(fno.library_path()) or not shutil.which("nm"):
        pytest.skip("needs libfno.so (run __graft_entry__.build()) and nm")
    names = subprocess.run(["nm", fno.library_path()], capture_output=True, text=True, check=True).stdout
    # <activation, vectors, [whether turned,] x's type, out's type>
    stub = r"__device_stub__%sILi\dELi(\d+)E(?:Lb\dE)?(f|DF16b|DF16_)(f|DF16b|DF16_)E" % kernel
    found = {}
    for n, x, out in re.findall(stub, names):
        found.setdefault((x, out), set()).add(int(n))
    assert found == {("f", "f"): {2, 4, 8, 16}, **{(t, t): {2, 4, 8, 16} for t in HALF},
                     **{(t, "f"): mixed for t in HALF}}
