"""Queries with NaN or an infinity in them: every score of such a row is a NaN or an
infinity (the cache holds finite values), so its softmax is not a number.  Its
output and log-sum-exp are NaN however the positions are cut, a row that sees
nothing has 0 and -inf whatever its queries are, and the other rows keep their bits."""
import numpy as np
import pytest
import torch

from test_gpu_attention import DEV, fill, i32, make_cache, queries

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")

NAN, INF = float("nan"), float("inf")


def attend(q, cache, table, lens, causal=False, **kw):
    B, M, H, _ = q.shape
    lse = torch.empty((B, H, M), dtype=torch.float32, device=DEV)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32(lens), causal=causal, lse=lse, **kw)
    assert kq.device_status() == 0
    return out.cpu(), lse.transpose(1, 2).cpu()


# Few rows and many; lengths in one part (also one with a ragged last tile) and in several.
@pytest.mark.parametrize("M,L", [(1, 40), (1, 3000), (12, 40), (12, 3000), (40, 130), (40, 3000), (150, 128),
                                 (150, 200), (150, 3000), (300, 6000)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["nan", "inf", "-inf", "one nan"])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_that_are_not_numbers(M, L, D, kind, causal):
    B, H = 2, 2
    lens = [L, L // 2]
    cache, table, k, v = make_cache(B, L, 1, D, 16, seed=M + L + D)
    fill(cache, table, k, v, lens)
    q = queries(B, M, H, D, 3)
    want, want_lse = attend(q, cache, table, lens, causal)
    bad = torch.zeros((B, M, H), dtype=torch.bool)
    bad[0, 0, 1] = bad[1, M // 2, 0] = bad[0, M - 1, 1] = True
    poison = torch.tensor({"nan": NAN, "inf": INF, "-inf": -INF, "one nan": NAN}[kind], dtype=torch.bfloat16)
    q[bad, :] = torch.where(torch.arange(D) == (D - 1 if kind == "one nan" else 0), poison, q[bad, :])
    if kind == "nan":
        q[bad, :] = poison
    got, lse = attend(q, cache, table, lens, causal)
    blind = torch.isneginf(want_lse)                          # causal: more queries than positions
    assert torch.equal(got[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    assert got[bad & ~blind].isnan().all() and lse[bad & ~blind].isnan().all()
    assert (got[bad & blind] == 0).all() and torch.isneginf(lse[bad & blind]).all()
    assert (bad & ~blind).any()


@pytest.mark.parametrize("M,L", [(1, 40), (1, 3000), (40, 3000), (150, 128), (150, 200), (150, 3000)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_scores_of_one_sign(M, L, sign):
    """All scores of the row +inf, or all -inf: neither is a softmax."""
    B, H, D = 1, 1, 64
    cache, table, k, v = make_cache(B, L, H, D, 16, seed=M + L)
    k = k.clone()
    k[..., 0] = 30.0                                          # positive, and the largest of its block
    fill(cache, table, k, v, [L])
    q = queries(B, M, H, D, 4)
    want, want_lse = attend(q, cache, table, [L])
    q[0, M // 2, 0, 0] = sign * INF
    got, lse = attend(q, cache, table, [L])
    others = torch.arange(M) != M // 2
    assert got[0, M // 2].isnan().all() and lse[0, M // 2].isnan().all()
    assert torch.equal(got[0, others], want[0, others]) and torch.equal(lse[0, others], want_lse[0, others])


@pytest.mark.parametrize("M", [1, 40, 150])
@pytest.mark.parametrize("L", [100, 3000])
def test_nothing_seen_is_zero_whatever_the_query(M, L):
    """An empty sequence, and one without any page in the pool."""
    B, H, D = 2, 2, 72
    cache, table, k, v = make_cache(B, L, H, D, 16, seed=M)
    fill(cache, table, k, v, [L, L])
    q = torch.full((B, M, H, D), NAN, dtype=torch.bfloat16)
    q[1] = -INF
    table = table.clone()
    table[1] = cache.pages
    lse = torch.empty((B, H, M), dtype=torch.float32, device=DEV)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([0, L]), lse=lse)
    assert kq.device_status() == 8
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_numbers_beside_missing_pages():
    """A row of NaN that sees one page only, in a later part than the first."""
    for M in (1, 40, 150):
        L, D = 3000, 64
        cache, table, k, v = make_cache(1, L, 1, D, 16, seed=M)
        fill(cache, table, k, v, [L])
        table = table.clone()
        table[0, :140] = -1
        table[0, 141:] = -1
        q = queries(1, M, 1, D, 5)
        q[0, 0] = NAN
        lse = torch.empty((1, 1, M), dtype=torch.float32, device=DEV)
        out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([L]), lse=lse)
        assert kq.device_status() == 8
        assert out[0, 0].isnan().all() and lse[0, 0, 0].isnan()
        assert out[0, 1:].isfinite().all() and lse[0, 0, 1:].isfinite().all()
