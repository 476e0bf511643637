"""Attention at the ends of its ranges.

K and V are multiplied in bf16 as the value times 2^-62, whose smallest step is 2^-133:
a value is exact where its block's largest magnitude is 2^-68 or more (scale byte 57,
smallest code 2^-71), and off by at most half that step, 2^-72, below.  The weights sum
to 1, so the output is off by 2^-72 more, and a score by scale sum |q| 2^-72.
"""
import numpy as np
import pytest
import torch

from oracle import kq_block as ob
from test_gpu_attention import DEV, fill, i32, make_cache, queries

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")


def bounds(q, kd, vd, lens):
    """The value, and the tolerance of test_gpu_attention with the two terms above."""
    B, M, H, D = q.shape
    L = kd.shape[1]
    ref, rl, A, logit = ob.attention(q, kd, vd, lens)
    d = (D + 8) * 2.0 ** -24 * logit + 2.0 ** -22 * (np.abs(rl) + logit)
    d = d + D ** -0.5 * np.abs(q).sum(-1).transpose(0, 2, 1) * 2.0 ** -72
    dd = np.expm1(2 * d).transpose(0, 2, 1)[..., None]
    tol = (2.0 ** -8 * (1 + 2.0 ** -8) + dd + (L + 32) * 2.0 ** -23) * A + 2.0 ** -8 * np.abs(ref)
    return ref, tol * (1 + 2.0 ** -7) + (L + 1) * 2.0 ** -126 + 2.0 ** -72 * (1 + 2.0 ** -7)


@pytest.mark.parametrize("M,L", [(1, 90), (1, 1500), (40, 90), (150, 200), (150, 1500)])
@pytest.mark.parametrize("e", [-60, -66, -70, -72, -75, -100, -126])
@pytest.mark.parametrize("D", [64, 72])
def test_small_values(M, L, e, D):
    lens = [L, L - 7]
    cache, table, k, v = make_cache(2, L, 2, D, 16, seed=L - e)
    k, v = ((x.double() * 2.0 ** p).to(torch.bfloat16) for x, p in ((k, e // 2), (v, e)))
    kd, vd = fill(cache, table, k, v, lens)
    assert np.abs(vd[0]).max() > 0                            # the cache itself holds them
    q = queries(2, M, 2, D, 5)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32(lens)).double().cpu().numpy()
    assert kq.device_status() == 0
    ref, tol = bounds(q.double().numpy(), kd, vd, lens)
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())


@pytest.mark.parametrize("M,L", [(1, 90), (40, 1500), (150, 200)])
def test_small_and_large_blocks_together(M, L):
    """Blocks of 2^-68 to 2^50 beside one another: the large ones keep every bit."""
    D, lens = 96, [L]
    cache, table, k, v = make_cache(1, L, 1, D, 16, seed=L)
    rng = np.random.default_rng(L)
    e = torch.from_numpy(rng.choice([-120, -68, -40, 0, 50], (1, L, 1, 3))).repeat_interleave(32, -1)
    v = (v.double() * 2.0 ** e).to(torch.bfloat16)
    kd, vd = fill(cache, table, k, v, lens)
    q = queries(1, M, 1, D, 6)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32(lens)).double().cpu().numpy()
    ref, tol = bounds(q.double().numpy(), kd, vd, lens)
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())


@pytest.mark.parametrize("M", [1, 40, 150])
def test_values_are_exact_from_2_to_the_minus_68(M):
    """One position: the output is V itself, the smallest code 2^-71."""
    D = 32
    cache = kq.cache_alloc(1, 16, 1, D, device=DEV)
    x = torch.tensor([0.5, 1, 1.5, 2, 3, 4, 6, 0], dtype=torch.float64).repeat(4) * 2.0 ** -70
    v = x.to(torch.bfloat16).view(1, 1, 1, D).to(DEV)
    kq.cache_write(cache, i32([[0]]), v, v)
    assert int(cache.v_scales[0, 0, 0, 0]) == 57
    q = queries(1, M, 1, D, 7).to(DEV)
    out = kq.attention_mxfp4(q, cache, i32([[0]]), i32([1]))
    assert torch.equal(out, v.expand(1, M, 1, D))
