"""Scales that the kernels' own factor of 2^62 would take past float32 are refused on the
host (a score of 0 would come out as 0 times infinity)."""
import pytest

from test_block_abi import L, attend, cache  # noqa: F401


@pytest.mark.parametrize("scale", [2.0 ** 66, -2.0 ** 66, 1e30, -3e38, float("inf"), float("nan")])
def test_scales_past_the_range(L, scale):  # noqa: F811
    assert attend(L, cache(L), scale=scale) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 150])
def test_the_largest_scale_and_scores_of_zero(M):
    """K = 0: every score is 0, the weights are equal and the output is V's mean."""
    import torch
    kq = pytest.importorskip("w4a4_post_quantization_b200")
    cache = kq.cache_alloc(2, 16, 1, 32, device="cuda:0")
    v = torch.ones((1, 32, 1, 32), dtype=torch.bfloat16, device="cuda:0")
    v[:, 16:] = 3
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda:0")
    kq.cache_write(cache, table, torch.zeros_like(v), v)
    q = torch.randn((1, M, 1, 32), device="cuda:0").to(torch.bfloat16)
    lens = torch.tensor([32], dtype=torch.int32, device="cuda:0")
    for scale in (2.0 ** 65 * 0.99, -2.0 ** 65 * 0.99):
        assert (kq.attention_mxfp4(q, cache, table, lens, scale=scale) == 2).all()
    with pytest.raises(kq.KQError):
        kq.attention_mxfp4(q, cache, table, lens, scale=2.0 ** 66)
    with pytest.raises(kq.KQError):
        kq.attention_mxfp4(q, cache, table, lens, scale=1e300)
    assert kq.device_status() == 0
