"""Every head width through both attention kernels, in one part and in several, against
the float64 oracle: a width is its own arrangement of channel panels."""
import pytest

from test_gpu_attention import run

pytestmark = pytest.mark.gpu

pytest.importorskip("w4a4_post_quantization_b200")

WIDTHS = list(range(8, 129, 8))


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("causal", [False, True])
def test_many_rows(D, causal):
    run(2, 140, 2, 2, D, 200, 16, [200, 77], causal, seed=D)


@pytest.mark.parametrize("D", WIDTHS)
def test_many_rows_of_grouped_heads_in_parts(D):
    run(2, 33, 6, 2, D, 1700, 32, [1700, 900], True, seed=D + 1)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("M", [1, 3, 11, 20])
def test_few_rows(D, M):
    run(2, M, 4, 2, D, 600, 16, [600, 333], True, seed=D + M)
