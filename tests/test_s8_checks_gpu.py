"""The int8 products in the checked debug build: every block of D (and C) that an
epilogue moves is checked against their extents, and no check fires."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu

CHILD = r'''
import os, sys
sys.path.insert(0, ROOT); sys.path.insert(0, os.path.join(ROOT, "tests"))
import test_s8_gemm_gpu as T
import quantized_gemm_tcgen05_gb300 as qg
assert qg.lib().gemm_checked_build() == 1
h = qg.gemm_create()
for pin in T.KERNELS:
    os.environ["GEMM_FORCE_KERNEL"] = pin
    for d, (m, n, k) in (("bf16", (150, 264, 520)), ("f32", (33, 131, 300)), ("f16", (300, 512, 256)), ("bf16", (1, 77, 64))):
        T.Problem(m, n, k, d, beta=0.5).check(h)
    T.Problem(143, 200, 320, "bf16", sizes=[3, 0, 140], seed=1, beta=0.5).check(h)
    T.Problem(217, 200, 300, "bf16", lda=512, ldb=320, ldd=203, shift=1, beta=1.0).check(h)
os.environ["GEMM_FORCE_KERNEL"] = ""
T.Problem(5, 192, 2300, "f32").check(h, splitk=4)
assert qg.gemm_device_status(h, qg.current_stream()) == 0
print("no check fired")
'''


def test_no_check_fires():
    from quantized_gemm_tcgen05_gb300 import _build

    _build.build(checks=True)
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n{CHILD}"], env=dict(os.environ, GEMM_DEVICE_CHECKS="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "no check fired" in r.stdout
