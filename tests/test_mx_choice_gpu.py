"""GPU tests that a forced number of K slices is the one that runs, whatever
kernel an estimate would take, and that it gives the same sums."""
import numpy as np
import pytest

import quantized_gemm_tcgen05_gb300 as qg
import synth
import test_mx_gemm_gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [qg.GEMM_NVFP4, qg.GEMM_MXFP4])
@pytest.mark.parametrize("m", [1, 100, 128, 500])
@pytest.mark.parametrize("splits,steps,want", [(1, 16, 1), (2, 16, 2), (4, 16, 4), (8, 16, 8), (8, 5, 4), (4, 1, 1)])
def test_forced_slices(fmt, m, splits, steps, want):
    h = qg.gemm_create()
    rng = np.random.default_rng(m)
    n, k = 320, 256 * steps
    a, b = G.Operand(rng, m, k, fmt), G.Operand(rng, n, k, fmt)
    got = G.product(h, a, b, fmt, synth.F32, op=qg.gemm_op_t(splitk=splits))
    assert qg.gemm_last_choice(h).split("/")[1] == ("dp" if want == 1 else f"splitk{want}")
    G.check(got, a.values @ b.values.T, np.abs(a.values) @ np.abs(b.values).T, synth.F32)
    qg.gemm_destroy(h)
