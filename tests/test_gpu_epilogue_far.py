"""Activations of large magnitudes and of numbers that are none.  For y -> -inf every
activation goes to 0 and for y -> inf to y; y is held in float32, so by |y| = 2^7 the
rest is far below 2^-60 in absolute terms (silu: 2^7 exp(-2^7) < 2^-177).  The kernel
takes y below -43.5 (silu) and -7.6 (tanh-GELU) as that: 43.5 exp(-43.5) < 2^-57 and
7.6 / (1 + exp(2 sqrt(2 / pi) (7.6 + 0.044715 7.6^3))) < 2^-59, 2^38 times less than the
2e-6 that is promised."""
import numpy as np
import pytest
import torch

from test_gpu_epilogue import DEV, dev, kq, tiled

pytestmark = pytest.mark.gpu

ACTS = ("gelu_tanh", "gelu", "silu")
TINY = 2.0 ** -57


def operands(p, N, zero_every=5):
    """32 products a sum; rows alternate between +2^p and -2^p, some are 0."""
    M, K = 136, 32
    q = np.full((M, K // 2), 0x22, np.uint8)
    q[1::2] = 0xAA                                            # -1
    q[::zero_every] = 0
    y = np.where(np.arange(M) % 2 == 0, 1.0, -1.0) * 2.0 ** p
    y[::zero_every] = 0
    lo = (p - 5) // 2
    sa = np.full((M, 1), 127 + lo, np.uint8)
    qb, sb = np.full((N, K // 2), 0x22, np.uint8), np.full((N, 1), 127 + p - 5 - lo, np.uint8)
    return y, (q, sa, qb, sb)


@pytest.mark.parametrize("p", [7, 20, 40, 60, 64, 100, 125])
@pytest.mark.parametrize("N", [8, 7, 520])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_far_out(p, N, dt):
    y, (qa, sa, qb, sb) = operands(p, N)
    args = dev(qa), tiled(sa, 32), dev(qb), tiled(sb, 32)
    assert (kq.gemm_mxfp4_epilogue(*args, out_dtype=torch.float32).double().cpu().numpy() == y[:, None]).all()
    for act in ACTS:
        got = kq.gemm_mxfp4_epilogue(*args, activation=act, out_dtype=dt).double().cpu().numpy()
        assert (got[y > 0] == 2.0 ** p).all() and (got[y == 0] == 0).all(), act
        assert (np.abs(got[y < 0]) <= TINY).all(), (act, got[y < 0].min())


@pytest.mark.parametrize("act", ("none",) + ACTS)
@pytest.mark.parametrize("N", [8, 7, 520])
def test_a_nan_stays_in_its_own_column_and_row(act, N):
    """Scale byte 255 is NaN: one row of A, one of B."""
    y, (qa, sa, qb, sb) = operands(5, N)
    call = dict(activation=act, out_dtype=torch.float32)
    want = kq.gemm_mxfp4_epilogue(dev(qa), tiled(sa, 32), dev(qb), tiled(sb, 32), **call)
    sa, sb = sa.copy(), sb.copy()
    sa[3], sb[N // 2] = 255, 255
    got = kq.gemm_mxfp4_epilogue(dev(qa), tiled(sa, 32), dev(qb), tiled(sb, 32), **call)
    bad = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    bad[3], bad[:, N // 2] = True, True
    assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("act,limit", [("gelu_tanh", 0.0), ("gelu", 0.0), ("silu", 0.0)])
def test_sums_past_float32(act, limit):
    """A bias of -inf: the limit, 0, or not a number as in -inf times 0; never -inf."""
    y, (qa, sa, qb, sb) = operands(5, 16)
    bias = torch.zeros(16, dtype=torch.bfloat16, device=DEV)
    bias[3], bias[4] = -float("inf"), float("inf")
    got = kq.gemm_mxfp4_epilogue(dev(qa), tiled(sa, 32), dev(qb), tiled(sb, 32), bias=bias, activation=act,
                                 out_dtype=torch.float32)
    assert (((got[:, 3] - limit).abs() <= TINY) | got[:, 3].isnan()).all() and torch.isposinf(got[:, 4]).all()
    assert got[:, 5:].isfinite().all() and got[:, :3].isfinite().all()
