"""The MXFP4 K/V cache against its float64 oracle.  Quantizing bf16 values to
MXFP4 and decoding them are exact operations (powers of two, comparisons), so
codes, scale bytes and values are compared for equality."""
import numpy as np
import pytest
import torch

from oracle import kq_block as ob
from oracle import kq_oracle as o

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"
CACHE_INDEX = 8


def draw(shape, seed):
    """bf16 values over many binades, with zeros, zero rows and ties."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape) * 2.0 ** rng.integers(-30, 30, shape[:-1] + (1,))
    x[rng.random(shape) < 0.05] = 0
    x[rng.random(shape[:-1]) < 0.05] = 0
    ties = rng.random(shape[:-1]) < 0.2
    x[ties] = (rng.integers(-12, 13, shape) / 4)[ties]        # E2M1 midpoints at amax in [2, 4)
    return torch.from_numpy(x).to(torch.bfloat16)


def f64(t):
    return t.double().numpy()


def pool(pages, page_size, H, D, fill=0xA5):
    cache = kq.cache_alloc(pages, page_size, H, D, device=DEV)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(fill)
    return cache


def arrays(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def table_of(B, per_seq, pages, seed):
    t = np.random.default_rng(seed).permutation(pages)[: B * per_seq].reshape(B, per_seq)
    return t.astype(np.int32)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


SHAPES = [(1, 1, 1, 8, 16), (2, 300, 16, 72, 64), (3, 17, 5, 128, 16), (2, 33, 3, 64, 32),
          (1, 70, 20, 112, 128), (4, 1, 8, 128, 64), (2, 129, 2, 104, 16), (1, 40, 1, 32, 1024),
          (5, 3, 7, 40, 16)]


@pytest.mark.parametrize("B,T,H,D,page", SHAPES)
@pytest.mark.parametrize("offset", [0, 13])
def test_write_and_read_match_the_oracle(B, T, H, D, page, offset):
    per_seq = -(-(T + offset) // page)
    cache = pool(B * per_seq + 2, page, H, D)
    table = table_of(B, per_seq, B * per_seq + 2, seed=T + D)
    k, v = draw((B, T, H, D), seed=T * 7 + D), draw((B, T, H, D), seed=T * 7 + D + 1)
    lens = [max(0, T - 3 * b) for b in range(B)]
    start = [offset] * B
    want = arrays(cache)
    for i, x in ((0, k), (2, v)):
        assert ob.cache_write(want[i], want[i + 1], table, f64(x), start, lens) == 0
    kq.cache_write(cache, i32(table), k.to(DEV), v.to(DEV), start=i32(start), lens=i32(lens))
    for got, w in zip(arrays(cache), want):                   # untouched slots keep their bytes
        assert np.array_equal(got, w)
    for dt in (torch.bfloat16, torch.float32):
        gk, gv = kq.cache_read(cache, i32(table), i32(lens), T, start=i32(start), out_dtype=dt)
        for got, i in ((gk, 0), (gv, 2)):
            assert np.array_equal(f64(got.cpu()),
                                  ob.cache_read(want[i], want[i + 1], table, lens, T, start, D))
    assert kq.device_status() == 0


def test_defaults_and_the_format_of_the_quantizer():
    """No start and no lens: every row, from position 0.  With head_dim a
    multiple of 32 a page array is what kq.dequantize decodes."""
    B, T, H, D, page = 2, 48, 4, 64, 16
    cache = pool(6, page, H, D)
    table = i32([[0, 1, 2], [5, 4, 3]])
    k, v = draw((B, T, H, D), 3).to(DEV), draw((B, T, H, D), 4).to(DEV)
    kq.cache_write(cache, table, k, v)
    gk, gv = kq.cache_read(cache, table, None, T)
    y = kq.dequantize(cache.k_codes.view(-1, D // 2), cache.k_scales.view(-1, D // 32))
    y = y.view(6, H, page, D)[[0, 1, 2, 5, 4, 3]].view(2, 3, H, page, D).transpose(2, 3)
    assert torch.equal(gk.float(), y.reshape(B, T, H, D))
    q, s = kq.quantize_smooth(k.view(-1, D), torch.ones(D, device=DEV))
    assert torch.equal(kq.dequantize(q, s).view(B, T, H, D), gk.float())
    kq.cache_write(cache, table, gk, gv)                      # a decoded row quantizes to itself
    assert all(torch.equal(a, b) for a, b in zip((gk, gv), kq.cache_read(cache, table, None, T)))


def test_strided_and_broadcast_rows():
    """K and V as slices of one projection's output, heads before rows, and a
    row shared by every sequence."""
    B, T, H, D = 3, 21, 6, 80
    table = i32(np.arange(6).reshape(3, 2))
    fused = draw((B, T, 3 * H, D), 5).to(DEV)
    heads_first = draw((B, H, T, D), 6).to(DEV).transpose(1, 2)
    shared = draw((1, T, H, D), 7).to(DEV).expand(B, T, H, D)
    for k, v in ((fused[:, :, H:2 * H], fused[:, :, 2 * H:]), (heads_first, shared)):
        a, b = pool(6, 16, H, D), pool(6, 16, H, D)
        kq.cache_write(a, table, k, v)
        kq.cache_write(b, table, k.contiguous(), v.contiguous())
        assert all(np.array_equal(x, y) for x, y in zip(arrays(a), arrays(b)))
    out = torch.full((B, H, T, D), -1.0, dtype=torch.bfloat16, device=DEV)
    kq.cache_read(a, table, None, T, k=out.transpose(1, 2), v=torch.empty_like(fused[:, :, :H]))
    assert torch.equal(out.transpose(1, 2), kq.cache_read(a, table, None, T)[0])


def test_rows_without_a_page_are_left_out():
    """A page id outside the pool, a negative one, a negative start and a start
    past the table: those rows are skipped and reported, the rest is written."""
    H, D, T = 2, 32, 20
    cache = pool(3, 16, H, D)
    table = np.array([[0, 3], [-1, 1], [2, 2], [2, 2]], dtype=np.int32)
    start = [0, 0, -2, 1 << 30]
    lens = [T, T, 4, T]
    k, v = draw((4, T, H, D), 8), draw((4, T, H, D), 9)
    want = arrays(cache)
    lost = [ob.cache_write(want[i], want[i + 1], table, f64(x), start, lens)
            for i, x in ((0, k), (2, v))]
    assert lost == [4 + 16 + 2 + T] * 2
    kq.cache_write(cache, i32(table), k.to(DEV), v.to(DEV), start=i32(start), lens=i32(lens))
    assert kq.device_status() == CACHE_INDEX
    for got, w in zip(arrays(cache), want):
        assert np.array_equal(got, w)
    gk, _ = kq.cache_read(cache, i32(table), i32(lens), T, start=i32(start))
    assert kq.device_status() == CACHE_INDEX
    assert np.array_equal(f64(gk.cpu()), ob.cache_read(want[0], want[1], table, lens, T, start, D))
    assert kq.device_status() == 0


def test_lengths_outside_the_rows():
    """Negative lengths write nothing, longer ones every row."""
    H, D, T = 1, 32, 5
    cache = pool(2, 16, H, D)
    table = i32([[0], [1]])
    k = draw((2, T, H, D), 10)
    before = arrays(cache)
    kq.cache_write(cache, table, k.to(DEV), k.to(DEV), lens=i32([-3, 0]))
    assert all(np.array_equal(x, y) for x, y in zip(before, arrays(cache)))
    gk, gv = kq.cache_read(cache, table, i32([-1, 0]), T)
    assert not gk.any() and not gv.any()
    kq.cache_write(cache, table, k.to(DEV), k.to(DEV), lens=i32([T + 9, T]))
    want = f64(k)
    q, s = ob.quantize_rows(want)
    gk, _ = kq.cache_read(cache, table, i32([1 << 30, T]), T)
    assert np.array_equal(f64(gk.cpu()), ob.decode_rows(q, s, D))
    assert kq.device_status() == 0


def test_empty_calls():
    cache = pool(1, 16, 2, 32)
    empty = torch.empty((1, 0, 2, 32), dtype=torch.bfloat16, device=DEV)
    kq.cache_write(cache, i32([[0]]), empty, empty)
    gk, gv = kq.cache_read(cache, i32([[0]]), None, 0)
    assert gk.shape == gv.shape == (1, 0, 2, 32)


def test_offsets_past_32_bits():
    """A pool whose code arrays pass 2^32 bytes: rows land at the far end."""
    page, H, D = 1024, 8, 128
    pages = (1 << 32) // (page * H * D // 2) + 2
    cache = kq.cache_alloc(pages, page, H, D, device=DEV)
    table = i32([[pages - 1, 0]])
    k = draw((1, 40, H, D), 11)
    start = i32([page - 8])
    kq.cache_write(cache, table, k.to(DEV), k.to(DEV), start=start)
    gk, gv = kq.cache_read(cache, table, None, 40, start=start)
    q, s = ob.quantize_rows(f64(k))
    assert np.array_equal(f64(gk.cpu()), ob.decode_rows(q, s, D)) and torch.equal(gk, gv)
    assert cache.k_codes[pages - 1, :, page - 8:].any() and cache.k_codes[0, :, :32].any()
    assert not cache.k_codes[1:pages - 1].any()


def test_special_scales_decode():
    """Scale byte 0 (2^-127), 254 and 255 (NaN) read back as kq.dequantize has
    them, as far as bf16 goes."""
    cache = pool(1, 16, 1, 32, fill=0)
    cache.k_codes[0, 0, :4] = torch.arange(16, dtype=torch.uint8, device=DEV) * 17
    cache.k_scales[0, 0, :4, 0] = torch.tensor([0, 1, 254, 255], dtype=torch.uint8, device=DEV)
    gk, _ = kq.cache_read(cache, i32([[0]]), None, 4, out_dtype=torch.float32)
    y = kq.dequantize(cache.k_codes.view(-1, 16), cache.k_scales.view(-1, 1))[:4]
    assert torch.equal(gk[0, :3, 0], y[:3]) and gk[0, 3].isnan().all()
    g16, _ = kq.cache_read(cache, i32([[0]]), None, 4)
    assert torch.equal(g16[0, :3, 0], y[:3].to(torch.bfloat16))


def test_graph_replay_and_another_stream():
    B, T, H, D = 2, 1, 4, 128
    cache = pool(4, 16, H, D)
    table = i32([[0, 1], [2, 3]])
    k, v = draw((B, T, H, D), 12).to(DEV), draw((B, T, H, D), 13).to(DEV)
    start = i32([0, 5])
    out = [torch.empty((B, T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kq.cache_write(cache, table, k, v, start=start)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kq.cache_write(cache, table, k, v, start=start)
            kq.cache_read(cache, table, None, T, start=start, k=out[0], v=out[1])
    k.copy_(draw((B, T, H, D), 14))
    start.copy_(i32([17, 3]))                                  # the step moves on; the graph stays
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    q, s = ob.quantize_rows(f64(k.cpu()))
    assert np.array_equal(f64(out[0].cpu()), ob.decode_rows(q, s, D))
    page = o.unpack_codes(cache.k_codes[1, :, 1].cpu().numpy())
    assert np.array_equal(page, o.unpack_codes(q[0, 0]))
    del g


def test_refusals():
    cache = pool(4, 16, 2, 64)
    table = i32([[0, 1], [2, 3]])
    k = draw((2, 20, 2, 64), 15).to(DEV)
    lens = i32([20, 20])
    odd = torch.zeros((2, 20, 2, 68), dtype=torch.bfloat16, device=DEV)[..., 4:]
    for bad in (lambda: kq.cache_write(cache, table, k.float(), k), lambda: kq.cache_write(cache, table, k, k[:, :19]),
                lambda: kq.cache_write(cache, table, k[:, :, :1], k[:, :, :1]),
                lambda: kq.cache_write(cache, table[:1], k, k), lambda: kq.cache_write(cache, table.long(), k, k),
                lambda: kq.cache_write(cache, table, k, k, lens=lens[:1]),
                lambda: kq.cache_write(cache, table, k, k, start=lens.long()),
                lambda: kq.cache_write(cache, table, odd, k), lambda: kq.cache_write(cache, table, k, k.cpu()),
                lambda: kq.cache_write(cache, table, k.transpose(2, 3), k),
                lambda: kq.cache_write(cache, table.t(), k, k),
                lambda: kq.cache_read(cache, table, lens, -1), lambda: kq.cache_read(cache, table, lens[:1], 4),
                lambda: kq.cache_read(cache, table, lens, 20, out_dtype=torch.float16),
                lambda: kq.cache_read(cache, table, lens, 20, k=k[:, :19]),
                lambda: kq.cache_read(cache, table, lens, 20, k=k.float()),
                lambda: kq.cache_read(cache, table, lens, 20, k=k[:, :1].expand(-1, 20, -1, -1)),
                lambda: kq.cache_read(cache, table, lens, "20"), lambda: kq.cache_read(cache, table, lens, 20, k=k, v=k),
                lambda: kq.KVCache(cache.k_codes, cache.k_scales, cache.v_codes[:2], cache.v_scales, 64),
                lambda: kq.KVCache(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, 96),
                lambda: kq.cache_alloc(4, 24, 2, 64, device=DEV)):
        with pytest.raises(ValueError):
            bad()
    assert kq.device_status() == 0
