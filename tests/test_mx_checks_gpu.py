"""The 4-bit products in the checked debug build: every block of D (and C) that
an epilogue moves is checked against their extents, and no check fires."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu

CHILD = r'''
import os, sys
sys.path.insert(0, ROOT); sys.path.insert(0, os.path.join(ROOT, "tests"))
import numpy as np
import test_mx_gemm_gpu as T
import quantized_gemm_tcgen05_gb300 as qg
import synth
assert qg.lib().gemm_checked_build() == 1
h = qg.gemm_create()
for pin in ("", "mx_bn64", "mx_bn128", "mx2_bn256"):
    os.environ["GEMM_FORCE_KERNEL"] = pin
    for fmt in T.FORMATS:
        for d, (m, n, k) in ((synth.BF16, (150, 264, 520)), (synth.F32, (33, 131, 300)), (synth.F16, (300, 512, 256))):
            T.test_shapes(h, pin, fmt, d, (m, n, k))
        T.grouped(h, [3, 0, 140], 200, 320, fmt, synth.BF16, seed=1, alpha=0.125, beta=0.5)
    T.test_strides_and_nothing_else_written(h, pin, synth.BF16, 217)
os.environ["GEMM_FORCE_KERNEL"] = ""
T.test_k_slices(h, fmt, 4, (5, 192, 2300))
print("no check fired")
'''


def test_no_check_fires():
    from quantized_gemm_tcgen05_gb300 import _build

    _build.build(checks=True)
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n{CHILD}"], env=dict(os.environ, GEMM_DEVICE_CHECKS="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "no check fired" in r.stdout
