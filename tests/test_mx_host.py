"""Host-side checks of the 4-bit microscaled operators that need no GPU: the
exported symbols, the struct layout, scale sizes, refusals without a handle,
and the test reference against hand values."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import mx_ref as R
import quantized_gemm_tcgen05_gb300 as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "gemm_mx.h")) as f:
        names = re.findall(r"^int\s+(gemm_\w+)\s*\(", f.read(), flags=re.M)
    assert set(names) == set(qg.MX_SYMBOLS)
    for n in names:
        assert hasattr(qg.lib(), n)


def test_struct_layout_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no host C compiler")
    cls = qg.gemm_mx_norm_t
    lines = ['printf("size %zu\\n", sizeof(gemm_mx_norm_t));']
    lines += [f'printf("{f} %zu\\n", offsetof(gemm_mx_norm_t, {f}));' for f, _ in cls._fields_]
    consts = ["GEMM_MXFP4", "GEMM_NVFP4", "GEMM_E2M1"]
    lines += [f'printf("{c} %d\\n", (int){c});' for c in consts]
    src = tmp_path / "m.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gemm_mx.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "m"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f, _ in cls._fields_:
        assert int(got[f]) == getattr(cls, f).offset, f
    for c in consts:
        assert int(got[c]) == getattr(qg, c)


@pytest.mark.parametrize("fmt", [R.MXFP4, R.NVFP4])
def test_scale_size(fmt):
    for rows, k in [(0, 5), (1, 1), (128, 64), (129, 65), (300, 4097)]:
        assert qg.gemm_mx_scale_size(fmt, rows, k) == R.tile(np.zeros((rows, R.ceil(k, R.BLOCK[fmt])), np.uint8)).size
        # any split into experts fits
        for E in (1, 3, 200):
            got = qg.gemm_mx_scale_size(fmt, rows, k, E)
            per = 512 * R.ceil(k, 4 * R.BLOCK[fmt])
            worst = min(E, rows) - 1 + R.ceil(rows - min(E, rows) + 1, 128) if rows else 0
            assert got >= worst * per
    for bad in [(fmt, -1, 4, 0), (fmt, 4, -1, 0), (fmt, 4, 4, -1), (fmt, 1 << 40, 4, 0), (0, 4, 4, 0), (3, 4, 4, 0)]:
        with pytest.raises(qg.GemmError):
            qg.gemm_mx_scale_size(*bad)


def test_null_handle_rejected():
    L, bad = qg.lib(), qg.GEMM_ERR_INVALID_ARG
    assert L.gemm_mx_quantize(None, 2, 1.0, None, None, None, None, None, 0, None, 0, None) == bad
    assert L.gemm_mx_dequantize(None, 2, 1.0, None, None, None, 0, None, None, None, 0, None) == bad
    assert L.gemm_run_mx(None, None, 2, 1.0, None, None, None, 0, None, None, None, 0, 0.0, *([None] * 5)) == bad
    assert L.gemm_run_mx_grouped(None, None, 2, 1.0, None, None, None, None, 0, None, None, None, 0, 0.0,
                                 *([None] * 5), 1, None) == bad
    assert L.gemm_mx_norm_quantize(None, *([None] * 10), 0, None) == bad
    assert L.gemm_mx_scale_size(2, 1, 1, 0, None) == bad


# ---- the reference the GPU tests compare with ------------------------------------

def test_reference_code_values_by_the_definition():
    # sign, two exponent bits (bias 1), one mantissa bit; exponent 0 is subnormal
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)
        assert R.VALUES[c] == (-v if c & 8 else v)


def test_reference_scales_against_torch():
    import torch

    b = torch.arange(128, dtype=torch.uint8)
    assert np.array_equal(R.e4m3_values(), b.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    b = torch.arange(1, 255, dtype=torch.uint8)
    assert np.array_equal(R.scale_values(b.numpy(), R.MXFP4), b.view(torch.float8_e8m0fnu).double().numpy())


def test_reference_rounding_by_hand():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.26, 7.0, 0.0, 0.5, 1, 1.5, 2, 6.0] * 2])
    code, byte = R.quantize(x, R.MXFP4)
    assert byte[0, 0] == 127  # amax 7: 2^(2 - 2)
    assert R.VALUES[code[0, :11]].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, -0.5, 6, 0]
    x[x == 7.0] = 6.0
    code, byte = R.quantize(x, R.NVFP4)
    assert byte[0].tolist() == [0x38, 0x38]


def test_reference_layout_by_hand():
    byte = np.arange(130 * 6).reshape(130, 6) % 251
    flat = R.tile(byte.astype(np.uint8))
    assert flat.size == 2 * 2 * 512
    assert flat[0] == byte[0, 0] and flat[3] == byte[0, 3] and flat[16] == byte[1, 0]
    assert flat[4] == byte[32, 0] and flat[512] == byte[0, 4] and flat[2 * 512] == byte[128, 0]
    assert flat[514] == 0 and flat[515] == 0  # blocks 6 and 7 of row 0: padding
    assert R.expert_rows([0, 3, 3, 133]).tolist()[:4] == [0, 1, 2, 128]
