"""Attention over the MXFP4 cache against the float64 oracle.

Tolerance, from the arithmetic (u = 2^-24, A = sum_p softmax_p |V[p]|):
* a score is a float32 sum of D exact products (bf16 times a decoded value),
  scaled once and taken through ex2: |d score| <= (D + 8) u * (scale sum |q||k|)
  + 2^-22 |score|, and a change d of every score changes each normalized weight
  by at most a factor exp(2 d);
* a weight is rounded to bf16, by at most 2^-8 of itself; ex2 and the float32
  sums over the L positions add (L + 32) 2^-23 (rescalings among them);
* the result is rounded to bf16 once: 2^-8 |out|.
So |d out| <= (2^-8 (1 + 2^-8) + expm1(2 d) + (L + 32) 2^-23) A + 2^-8 |out|
(times 1 + 2^-7 for the product of the two roundings) + (L + 1) 2^-126: float32
and bf16 have no normal number below 2^-126, so each of the L products, and the
result, may lose that much absolutely where the weights are that small.  And
|d lse| <= d + (L + 32) 2^-23 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import kq_block as ob

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"
CACHE_INDEX = 8


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make_cache(B, L, H, D, page, seed, kv_scale=1.0, spare=1, garbage=True):
    """A filled cache with scattered pages, its table, and the decoded K and V.
    Slots behind each sequence hold garbage bytes, NaN scales among them."""
    rng = np.random.default_rng(seed)
    per_seq = max(1, -(-L // page))
    pages = B * per_seq + spare
    table = rng.permutation(pages)[: B * per_seq].reshape(B, per_seq).astype(np.int32)
    cache = kq.cache_alloc(pages, page, H, D, device=DEV)
    if garbage:
        for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
        cache.k_scales[..., 0] = 255
        cache.v_scales[..., 0] = 255
    if L == 0:
        z = np.zeros((B, 0, H, D))
        return cache, i32(table), z, z
    k = torch.from_numpy(rng.normal(size=(B, L, H, D))).to(torch.bfloat16)
    v = torch.from_numpy(rng.normal(size=(B, L, H, D)) * kv_scale).to(torch.bfloat16)
    v[..., :1] *= 20                                         # an outlier channel
    return cache, i32(table), k, v


def fill(cache, table, k, v, lens):
    kq.cache_write(cache, table, k.to(DEV), v.to(DEV), lens=i32(lens))
    gk, gv = kq.cache_read(cache, table, None, k.shape[1])
    return gk.double().cpu().numpy(), gv.double().cpu().numpy()


def check(out, lse, q, kd, vd, lens, causal, scale=None, seen=None):
    D, L = q.shape[-1], kd.shape[1]
    ref, rl, A, logit = ob.attention(q, kd, vd, lens, causal, scale, seen)
    with np.errstate(invalid="ignore"):
        d = (D + 8) * 2.0 ** -24 * logit + 2.0 ** -22 * np.where(np.isinf(rl), 0, np.abs(rl) + logit)
    dd = np.expm1(2 * d).transpose(0, 2, 1)[..., None]
    tol = (2.0 ** -8 * (1 + 2.0 ** -8) + dd + (L + 32) * 2.0 ** -23) * A + 2.0 ** -8 * np.abs(ref)
    tol = tol * (1 + 2.0 ** -7) + (L + 1) * 2.0 ** -126
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))
    if lse is not None:
        gl = lse.double().cpu().numpy()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty)
        ltol = d + (L + 32) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(empty, 0, rl))
        assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl)) <= ltol).all()


def queries(B, M, H, D, seed, gain=1.0):
    rng = np.random.default_rng(seed + 77)
    return torch.from_numpy(rng.normal(size=(B, M, H, D)) * gain).to(torch.bfloat16)


def run(B, M, H, Hkv, D, L, page, lens, causal, seed=0, gain=1.0, scale=None, **kw):
    cache, table, k, v = make_cache(B, L, Hkv, D, page, seed)
    kd, vd = fill(cache, table, k, v, lens)
    q = queries(B, M, H, D, seed, gain)
    lse = torch.empty((B, H, M), dtype=torch.float32, device=DEV)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32(lens), causal=causal, scale=scale, lse=lse,
                             **kw)
    assert kq.device_status() == 0
    check(out, lse, q.double().numpy(), kd, vd, lens, causal, scale)
    return out


@pytest.mark.parametrize("D", [8, 32, 40, 64, 72, 96, 104, 112, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_head_dims(D, causal):
    run(2, 3, 4, 2, D, 77, 16, [77, 50], causal, seed=D)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 300, 513])
@pytest.mark.parametrize("M", [1, 5])
def test_lengths(L, M):
    run(2, M, 4, 2, 64, L, 16, [L, L // 2], True, seed=L)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 8), (8, 1), (12, 4), (20, 20), (40, 2)])
@pytest.mark.parametrize("M", [1, 2, 7])
def test_head_layouts(H, Hkv, M):
    run(2, M, H, Hkv, 72, 90, 32, [90, 41], False, seed=H + M)


@pytest.mark.parametrize("M", [16, 17, 33, 64, 100, 127, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_query_counts(M, causal):
    """Row tiles that end inside, with more queries than positions among them:
    the first rows of a causal call see nothing."""
    run(2, M, 2, 2, 72, 140, 64, [140, 61], causal, seed=M)


@pytest.mark.parametrize("M,G", [(1, 1), (1, 4), (40, 4), (130, 1), (64, 3)])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_long_lengths_are_joined(M, G, D):
    """Long enough to be cut along the positions, with sequences that end in
    the first part, at an edge and nowhere."""
    run(4, M, G, 1, D, 2600, 16, [2600, 512, 3, 0], True, seed=M + D)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
def test_page_sizes(page):
    run(2, 9, 4, 2, 128, 333, page, [333, 200], True, seed=page)
    run(2, 150, 4, 2, 128, 333, page, [333, 200], True, seed=page)


@pytest.mark.parametrize("M", [1, 20, 140])
def test_rows_that_see_nothing(M):
    out = run(3, M, 2, 2, 64, 30, 16, [0, 30, 1], False, seed=M)
    assert not out[0].any()


@pytest.mark.parametrize("M", [1, 160])
def test_no_positions_at_all(M):
    cache, table, _, _ = make_cache(1, 0, 2, 64, 16, 3)
    lse = torch.zeros((1, 2, M), dtype=torch.float32, device=DEV)
    out = kq.attention_mxfp4(queries(1, M, 2, 64, 1).to(DEV), cache, table, i32([0]), lse=lse)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("M", [1, 130])
@pytest.mark.parametrize("gain,scale", [(40.0, None), (1.0, 3.0), (1.0, 0.0), (1.0, -0.5)])
def test_peaked_flat_and_negative_scores(M, gain, scale):
    run(1, M, 2, 2, 64, 200, 16, [200], False, seed=5, gain=gain, scale=scale)


@pytest.mark.parametrize("M", [1, 150])
def test_growing_scores(M):
    """Scores that rise along the positions: the running maximum grows in
    every tile, by far more than any slack."""
    B, L, H, D = 1, 700, 1, 64
    cache, table, k, v = make_cache(B, L, H, D, 64, 9)
    ramp = torch.linspace(0, 60, L)[None, :, None, None]
    k = (torch.ones_like(k).float() * ramp).to(torch.bfloat16)
    kd, vd = fill(cache, table, k, v, [L])
    q = torch.ones((B, M, H, D), dtype=torch.bfloat16) * 0.25
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([L]))
    check(out, None, q.double().numpy(), kd, vd, [L], False)


@pytest.mark.parametrize("M", [1, 150])
def test_wide_value_ranges(M):
    """Blocks of K and V many binades apart, tiny and large."""
    B, L, H, D = 1, 150, 2, 96
    cache, table, k, v = make_cache(B, L, H, D, 32, 10)
    rng = np.random.default_rng(4)
    e = torch.from_numpy(rng.integers(-40, 40, (B, L, H, 3))).repeat_interleave(32, -1)
    v = (v.double() * 2.0 ** e).to(torch.bfloat16)
    k = (k.double() * 2.0 ** e.clamp(max=0)).to(torch.bfloat16)
    kd, vd = fill(cache, table, k, v, [L])
    q = queries(B, M, H, D, 6)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([L]))
    check(out, None, q.double().numpy(), kd, vd, [L], False)


@pytest.mark.parametrize("M,Hkv,D,causal", [(140, 2, 64, False), (100, 4, 128, True)])
@pytest.mark.parametrize("empty", [0, 1, 2, 5])
def test_many_sequences_with_empty_ones_among_them(M, Hkv, D, causal, empty):
    """Several times as much work as a GPU holds at once, so that a block takes
    sequences of every length one after another; ``empty`` of six have none."""
    B = 130
    lens = [0 if b % 6 < empty else 1 + (37 * b) % 150 for b in range(B)]
    run(B, M, Hkv, Hkv, D, 150, 32, lens, causal, seed=empty)


def test_very_long_sequences_one_after_another():
    """More tiles of rows than a GPU holds at once, so that a block takes a second
    one after 4 million positions of the first.  Flat weights and values of 1: every
    sum is a whole number below 2^24, and the result exactly 1."""
    L, M, page = 1 << 22, 128 * 300, 1024
    cache = kq.cache_alloc(L // page, page, 1, 16, device=DEV)
    rng = np.random.default_rng(3)
    cache.k_codes.copy_(torch.from_numpy(rng.integers(0, 256, tuple(cache.k_codes.shape), dtype=np.uint8)))
    cache.k_scales.fill_(127)
    cache.v_codes.fill_(0x22)                                # 1.0 and 1.0
    cache.v_scales.fill_(127)
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).view(1, -1)
    q = torch.zeros((1, M, 1, 16), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, float("nan"))
    kq.attention_mxfp4(q, cache, table, i32([L]), out=out)
    assert kq.device_status() == 0
    assert bool((out == 1).all())


@pytest.mark.parametrize("M", [1, 140])
def test_max_len_bounds_lens(M):
    """Lengths above max_len count as max_len, negative ones as 0."""
    cache, table, k, v = make_cache(2, 64, 2, 64, 16, 11)
    kd, vd = fill(cache, table, k, v, [64, 64])
    q = queries(2, M, 2, 64, 7)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([1 << 30, -5]), max_len=37)
    check(out, None, q.double().numpy(), kd, vd, [37, 0], False)


@pytest.mark.parametrize("M", [1, 20, 140])
def test_strided_queries_and_output(M):
    B, H, D, L = 2, 4, 72, 60
    cache, table, k, v = make_cache(B, L, H, D, 16, 12)
    kd, vd = fill(cache, table, k, v, [L, 30])
    fused = queries(B, M, 3 * H, D, 8).to(DEV)
    q = fused[:, :, H:2 * H]
    want = kq.attention_mxfp4(q.contiguous(), cache, table, i32([L, 30]))
    buf = torch.full((B, H, M + 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
    got = kq.attention_mxfp4(q, cache, table, i32([L, 30]), out=buf.transpose(1, 2)[:, 1:-1])
    assert torch.equal(got, want)
    assert (buf[:, :, 0] == 7).all() and (buf[:, :, -1] == 7).all()
    check(want, None, q.double().cpu().numpy(), kd, vd, [L, 30], False)


@pytest.mark.parametrize("M", [1, 24, 140])
def test_pages_outside_the_pool_are_not_seen(M):
    B, L, H, D, page = 1, 96, 2, 64, 16
    cache, table, k, v = make_cache(B, L, H, D, page, 13)
    kd, vd = fill(cache, table, k, v, [L])
    bad = table.clone()
    bad[0, 2], bad[0, 5] = -1, cache.pages
    q = queries(B, M, H, D, 9)
    out = kq.attention_mxfp4(q.to(DEV), cache, bad, i32([L]))
    assert kq.device_status() == CACHE_INDEX
    seen = np.ones((B, L), bool)
    seen[0, 32:48] = seen[0, 80:96] = False
    check(out, None, q.double().numpy(), kd, vd, [L], False, seen=seen)
    bad[:] = 1 << 30
    out = kq.attention_mxfp4(q.to(DEV), cache, bad, i32([L]))
    assert kq.device_status() == CACHE_INDEX and not out.any()


@pytest.mark.parametrize("M", [1, 140])
def test_shared_pages(M):
    """Two sequences that read the same pages."""
    cache, table, k, v = make_cache(1, 80, 2, 64, 16, 14)
    kd, vd = fill(cache, table, k, v, [80])
    q = queries(2, M, 2, 64, 10)
    out = kq.attention_mxfp4(q.to(DEV), cache, table.expand(2, -1).contiguous(), i32([80, 33]))
    check(out, None, q.double().numpy(), np.repeat(kd, 2, 0), np.repeat(vd, 2, 0), [80, 33], False)


@pytest.mark.parametrize("M,L", [(1, 3000), (150, 200), (40, 3000)])
def test_runs_repeat_bit_for_bit_and_replay(M, L):
    B, H, D = 2, 4, 128
    cache, table, k, v = make_cache(B, L, 2, D, 64, 15)
    lens = i32([L, L // 3])
    kq.cache_write(cache, table, k.to(DEV), v.to(DEV), lens=lens)
    q = queries(B, M, H, D, 11).to(DEV)
    want = kq.attention_mxfp4(q, cache, table, lens, causal=True)
    for _ in range(3):
        assert torch.equal(kq.attention_mxfp4(q, cache, table, lens, causal=True), want)
    need = kq.attention_workspace_bytes(B, M, H, 2, D, table.shape[1] * 64)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device=DEV)      # NaN everywhere
    out = torch.empty_like(q)
    kq.attention_mxfp4(q, cache, table, lens, causal=True, out=out, workspace=ws)
    assert torch.equal(out, want)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            kq.attention_mxfp4(q, cache, table, lens, causal=True, out=out, workspace=ws)
    # The sequences shrink and the queries change; the graph stays.
    q.copy_(queries(B, M, H, D, 12))
    lens.copy_(i32([L // 2, 7]))
    ws.fill_(0xFF)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, kq.attention_mxfp4(q, cache, table, lens, causal=True))
    assert kq.device_status() == 0
    del g


def test_two_streams_at_once():
    cache, table, k, v = make_cache(2, 2000, 2, 64, 64, 16)
    lens = i32([2000, 900])
    kq.cache_write(cache, table, k.to(DEV), v.to(DEV), lens=lens)
    qs = [queries(2, m, 4, 64, 20 + m).to(DEV) for m in (1, 3, 150)]
    want = [kq.attention_mxfp4(q, cache, table, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in qs]
    got = [None] * len(qs)
    for _ in range(5):
        for i, (s, q) in enumerate(zip(streams, qs)):
            with torch.cuda.stream(s):
                got[i] = kq.attention_mxfp4(q, cache, table, lens)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M", [1, 140])
def test_offsets_past_32_bits(M):
    page, H, D, L = 1024, 8, 128, 50
    pages = (1 << 32) // (page * H * D // 2) + 2
    cache = kq.cache_alloc(pages, page, H, D, device=DEV)
    table = i32([[pages - 1]])
    rng = np.random.default_rng(17)
    k, v = (torch.from_numpy(rng.normal(size=(1, L, H, D))).to(torch.bfloat16) for _ in range(2))
    kd, vd = fill(cache, table, k, v, [L])
    q = queries(1, M, H, D, 18)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([L]))
    check(out, None, q.double().numpy(), kd, vd, [L], False)


def test_refusals():
    cache, table, k, v = make_cache(2, 32, 2, 64, 16, 19)
    q = queries(2, 3, 4, 64, 21).to(DEV)
    lens = i32([32, 32])
    call = kq.attention_mxfp4
    for bad in (lambda: call(q.float(), cache, table, lens), lambda: call(q[..., :32], cache, table, lens),
                lambda: call(q[:, :, :3].contiguous(), cache, table, lens),
                lambda: call(q, cache, table[:1], lens), lambda: call(q, cache, table.long(), lens),
                lambda: call(q, cache, table, lens[:1]), lambda: call(q, cache, table, None),
                lambda: call(q, cache, table, lens, max_len=33), lambda: call(q, cache, table, lens, max_len=0),
                lambda: call(q, cache, table, lens, out=torch.empty_like(q)[:, :2]),
                lambda: call(q, cache, table, lens, out=q[:, :, :1].expand(-1, -1, 4, -1)),
                lambda: call(q, cache, table, lens, lse=torch.empty((2, 3, 4), device=DEV)),
                lambda: call(q.cpu(), cache, table, lens), lambda: call(q[0], cache, table, lens),
                lambda: call(q.transpose(2, 3), cache, table, lens)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kq.KQError):
        call(q, cache, table, lens, scale=float("nan"))
    empty = call(q[:, :0], cache, table, lens)
    assert empty.shape == (2, 0, 4, 64)


def test_output_over_the_queries_is_refused():
    cache, table, k, v = make_cache(2, 32, 2, 64, 16, 19)
    both = torch.zeros((3, 2, 3, 4, 64), dtype=torch.bfloat16, device=DEV)
    q, lens = both[0], i32([32, 32])
    for out in (q, both.flatten()[64 : 64 + q.numel()].view(q.shape)):
        with pytest.raises(ValueError):
            kq.attention_mxfp4(q, cache, table, lens, out=out)
    kq.attention_mxfp4(q, cache, table, lens, out=both[1])
    fused = torch.zeros((2, 3, 2, 4, 64), dtype=torch.bfloat16, device=DEV)
    kq.attention_mxfp4(fused[:, :, 0], cache, table, lens, out=fused[:, :, 1])
    torch.cuda.synchronize()
