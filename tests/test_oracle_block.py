"""Pins of the float64 oracle of the block operators (cache, attention,
epilogue) to closed forms, so that the GPU tests compare with something that
is tied to more than itself."""
import math

import numpy as np
import pytest

from oracle import kq_block as ob
from oracle import kq_oracle as o


def test_a_row_pads_its_last_block_with_zeros():
    x = np.zeros((1, 40))
    x[0, 32:] = [6, -6, 3, 0.5, -0.25, 0.75, 1, 2]            # second block: amax 6, scale 1
    q, s = ob.quantize_rows(x)
    assert q.shape == (1, 32) and s.tolist() == [[0, 127]]
    want = [7, 15, 5, 1, 8, 2, 2, 4] + [0] * 24               # ties to the even code
    assert o.unpack_codes(q)[0, 32:].tolist() == want
    assert ob.decode_rows(q, s, 40)[0, 32:].tolist() == [6, -6, 3, 0.5, 0, 1, 1, 2]


def test_cache_places_rows_by_the_table():
    rng = np.random.default_rng(0)
    table = np.array([[3, 1], [0, 7]])                        # page 7 is not in the pool
    codes, scales = np.full((4, 2, 16, 16), 9, np.uint8), np.full((4, 2, 16, 1), 9, np.uint8)
    x = 2.0 * rng.integers(-3, 4, (2, 4, 2, 32))
    lost = ob.cache_write(codes, scales, table, x, [14, 15], [4, 3])
    assert lost == 2                                          # sequence 1, positions 16 and 17
    y = ob.cache_read(codes, scales, table, [4, 3], 5, [14, 15], 32)
    assert np.array_equal(y[0, :4], x[0]) and not y[0, 4].any()
    assert np.array_equal(y[1, 0], x[1, 0]) and not y[1, 1:].any()
    assert np.array_equal(ob.decode_rows(codes[3, :, 14], scales[3, :, 14], 32), x[0, 0])
    assert np.array_equal(ob.decode_rows(codes[1, :, 1], scales[1, :, 1], 32), x[0, 3])
    touched = np.zeros((4, 16), bool)
    touched[3, 14:], touched[1, :2], touched[0, 15] = True, True, True
    assert (codes.transpose(0, 2, 1, 3)[~touched] == 9).all()


def test_attention_closed_forms():
    q = np.zeros((1, 2, 4, 8))
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(1, 5, 2, 8)), rng.normal(size=(1, 5, 2, 8))
    out, lse, terms, _ = ob.attention(q, k, v, [3])            # equal scores: the mean of 3 rows
    assert np.allclose(out[0, 1, 3], v[0, :3, 1].mean(0)) and np.allclose(lse, math.log(3))
    assert np.allclose(terms[0, 0, 0], np.abs(v[0, :3, 0]).mean(0))
    out, lse, _, _ = ob.attention(q, k, v, [1], causal=True)   # the first query sees nothing
    assert not out[0, 0].any() and np.isneginf(lse[0, :, 0]).all()
    assert np.allclose(out[0, 1, 0], v[0, 0, 0]) and np.allclose(lse[0, :, 1], 0)
    q[0, 0, 2] = 1e3 * k[0, 4, 1]                             # one position takes all
    out, _, _, logit = ob.attention(q, k, v, [9], scale=0.5)
    assert np.allclose(out[0, 0, 2], v[0, 4, 1])
    assert logit[0, 2, 0] >= 0.5 * 1e3 * (k[0, 4, 1] ** 2).sum() * (1 - 1e-12)
    out, _, _, _ = ob.attention(q, k, v, [0])
    assert not out.any()


@pytest.mark.parametrize("name", ["none", "gelu_tanh", "gelu", "silu"])
def test_activations_far_out_and_at_zero(name):
    y = ob.activation(np.array([-40.0, 0.0, 40.0]), name)
    assert np.allclose(y, [-40.0 if name == "none" else 0.0, 0.0, 40.0], atol=1e-12)


def test_activation_values():
    assert ob.activation(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-14)
    assert ob.activation(np.array([1.0]), "silu")[0] == pytest.approx(0.7310585786300049, rel=1e-14)
    assert ob.activation(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(0.8411919906082768, rel=1e-12)


def test_epilogue_order():
    y = ob.epilogue(np.full((3, 2), 2.0), bias=[1, -2], gate=[[2, 3], [5, 7]], tokens=2,
                    residual=np.ones((3, 2)))
    assert y.tolist() == [[7, 1], [7, 1], [16, 1]]
