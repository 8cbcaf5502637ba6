"""Which kernel serves an int8 product without being asked for: a build whose kernels
cannot share their registers out as they mean to would show here."""
import pytest

import quantized_gemm_tcgen05_gb300 as qg
from test_s8_gemm_gpu import Problem, h  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,want", [(1, 4096, 14336, "s8_gemv/"), (77, 11002, 4104, "s8_t32/"), (128, 4096, 4096, "s8_t128/"),
                                        (1024, 4096, 4096, "s8_pair/")])
def test_choice(h, m, n, k, want):  # noqa: F811
    p = Problem(m, n, k)
    p.run(h)
    assert qg.gemm_last_choice(h).startswith(want)


def test_choice_by_experts(h):  # noqa: F811
    for sizes, want in (([1, 0, 2, 0], "s8_grouped_gemv/"), ([20, 0, 30, 0], "s8_grouped_t")):
        Problem(sum(sizes), 96, 160, sizes=sizes).check(h)
        assert qg.gemm_last_choice(h).startswith(want)
