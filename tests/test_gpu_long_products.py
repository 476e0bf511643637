"""Products so long that one lasts longer than any other wait in a kernel: the wait of
the warps that take the result out has to last with them.  Operands of ones: every
partial sum is a multiple of 64 below 2^27, exact in float32, and so is the result."""
import pytest
import torch

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"
K = 1 << 26                                                   # 262144 stages, some 50 ms


def ones(rows, k):
    return torch.full((rows, k // 2), 0x22, dtype=torch.uint8, device=DEV)


def unit(*shape):
    return torch.full(shape, 127, dtype=torch.uint8, device=DEV)


def check(c, k):
    torch.cuda.synchronize()
    assert kq.device_status() == 0
    assert bool((c == k).all())


@pytest.mark.parametrize("N", [8, 7])                         # with and without TMA's rows
def test_tiled_scales(N):
    s = unit(kq.lib().kq_scales_tiled_bytes(128, K))
    check(kq.gemm_mxfp4_tiled(ones(1, K), s, ones(N, K), s, out_dtype=torch.float32), K)


@pytest.mark.parametrize("N", [8, 7])
def test_tiled_scales_of_16(N):
    s = unit(kq.lib().kq_scales16_tiled_bytes(128, K))
    check(kq.gemm_mxfp4_16_tiled(ones(1, K), s, ones(N, K), s), K)


@pytest.mark.parametrize("k", [K, K + 32])                    # scale rows of whole words, and not
def test_scales_in_rows(k):
    check(kq.gemm_mxfp4(ones(1, k), unit(1, k // 32), ones(8, k), unit(8, k // 32)), k)


@pytest.mark.parametrize("name,value", [("KQ_GEMM_PAIR", "1"), ("KQ_GEMM_PERSISTENT", "0"), ("KQ_GEMM_BN", "128")])
def test_the_other_kernels(monkeypatch, name, value):
    monkeypatch.setenv(name, value)
    s = unit(kq.lib().kq_scales_tiled_bytes(128, K))
    check(kq.gemm_mxfp4_tiled(ones(1, K), s, ones(8, K), s, out_dtype=torch.float32), K)


@pytest.mark.parametrize("N,dt", [(2048, torch.bfloat16), (1024, torch.bfloat16), (1024, torch.float32)])
def test_the_longest_with_an_epilogue_on_every_pair(N, dt):
    """72 tiles of either width, all of whose stages share the memory's bandwidth."""
    M, k = 9 * 256, 1 << 21
    s = unit(kq.lib().kq_scales_tiled_bytes(M, k))
    check(kq.gemm_mxfp4_epilogue(ones(M, k), s, ones(N, k), s, out_dtype=dt), k)
