"""Block operators at the ends of what their calls allow: the largest batches, heads,
pages and tables, calls at once, and first calls inside a capture."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import kq_block as ob
from test_gpu_attention import check, fill, make_cache, queries

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rows(shape, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def round_trip(x):
    return ob.decode_rows(*ob.quantize_rows(x.double().cpu().numpy()), x.shape[-1])


def test_the_largest_batch():
    """65535 sequences of one position, on 16 pages in turn of a pool shared by all."""
    B, H, D = 65535, 1, 16
    cache = kq.cache_alloc(4096, 16, H, D, device=DEV)
    table = (torch.arange(B, device=DEV, dtype=torch.int32) // 16).view(B, 1)
    start = torch.arange(B, device=DEV, dtype=torch.int32) % 16
    k, v = rows((B, 1, H, D), 1), rows((B, 1, H, D), 2)
    kq.cache_write(cache, table, k, v, start=start)
    gk, gv = kq.cache_read(cache, table, None, 1, start=start)
    assert np.array_equal(gk.double().cpu().numpy(), round_trip(k))
    assert np.array_equal(gv.double().cpu().numpy(), round_trip(v))
    q = rows((B, 1, H, D), 3)
    lens = start + 1
    out = kq.attention_mxfp4(q, cache, table, lens)
    pick = [0, 1, 15, 16, 40000, B - 1]
    kd, vd = (x.double().cpu().numpy() for x in kq.cache_read(cache, table[pick], None, 16))
    check(out[pick], None, q[pick].double().cpu().numpy(), kd, vd, lens[pick].tolist(), False)
    assert kq.device_status() == 0


def test_the_most_heads():
    """65535 heads: one row of all of them, and of a few more query heads."""
    H, D, T = 65535, 8, 3
    cache = kq.cache_alloc(1, 16, H, D, device=DEV)
    k, v = rows((1, T, H, D), 1), rows((1, T, H, D), 2)
    kq.cache_write(cache, i32([[0]]), k, v)
    gk, gv = kq.cache_read(cache, i32([[0]]), None, T)
    assert np.array_equal(gk.double().cpu().numpy(), round_trip(k))
    q = rows((1, 2, 2 * H, D), 3)
    out = kq.attention_mxfp4(q, cache, i32([[0]]), i32([T]), causal=True)
    heads = [0, 1, 2 * 40000, 2 * H - 1]
    kv = [h // 2 for h in heads]
    check(out[:, :, heads], None, *(x[:, :, j].double().cpu().numpy() for x, j in ((q, heads), (gk, kv), (gv, kv))),
          [T], True)
    assert kq.device_status() == 0


@pytest.mark.parametrize("M", [1, 40, 100])
def test_the_largest_pages_and_table(M):
    """Pages of 65536 positions and a table for 2^30: everything a block works out from
    the table's size stays inside 31 bits."""
    L, D, page = 70000, 8, 65536
    cache = kq.cache_alloc(2, page, 1, D, device=DEV)
    wide = torch.full((1, (1 << 30) // page), -1, dtype=torch.int32, device=DEV)
    wide[0, :2] = i32([1, 0])
    k, v = rows((1, L, 1, D), 1), rows((1, L, 1, D), 2)
    kq.cache_write(cache, wide, k, v)
    q = rows((1, M, 1, D), 3)
    lse = torch.empty((1, 1, M), device=DEV)
    out = kq.attention_mxfp4(q, cache, wide, i32([L]), lse=lse)
    gk, gv = kq.cache_read(cache, wide, None, L)
    check(out[:, -1:], lse[:, :, -1:], q[:, -1:].double().cpu().numpy(), gk.double().cpu().numpy(),
          gv.double().cpu().numpy(), [L], False)
    assert kq.device_status() == 0
    # Nothing behind the second page: every position there is left out and reported.
    assert not kq.attention_mxfp4(q, cache, wide[:, 2:].contiguous(), i32([100])).any()
    assert kq.device_status() == 8


def test_wide_groups():
    """4096 query heads on one K/V head."""
    H, D, L = 4096, 64, 50
    cache, table, k, v = make_cache(1, L, 1, D, 16, seed=1)
    kd, vd = fill(cache, table, k, v, [L])
    q = queries(1, 1, H, D, 2)
    out = kq.attention_mxfp4(q.to(DEV), cache, table, i32([L]))
    check(out, None, q.double().numpy(), kd, vd, [L], False)


def test_calls_at_once():
    """Four threads with streams, caches and workspaces of their own."""
    def work(n, result):
        torch.cuda.set_device(0)
        stream = torch.cuda.Stream(DEV)
        with torch.cuda.stream(stream):
            B, M, H, D, L = 2, 5 + 45 * n, 4, 64 + 8 * n, 700
            cache = kq.cache_alloc(2 * 44, 16, 2, D, device=DEV)
            table = torch.arange(88, dtype=torch.int32, device=DEV).view(2, 44)
            k, v, q = rows((B, L, 2, D), n), rows((B, L, 2, D), n + 9), rows((B, M, H, D), n + 18)
            lens = torch.tensor([L, L // 2], dtype=torch.int32, device=DEV)
            outs = []
            for _ in range(30):
                kq.cache_write(cache, table, k, v, lens=lens)
                outs.append(kq.attention_mxfp4(q, cache, table, lens, causal=True))
                outs.append(kq.cache_read(cache, table, lens, L)[0])
            stream.synchronize()
        result[n] = outs
    alone, together = {}, {}
    for n in range(4):
        work(n, alone)
    threads = [threading.Thread(target=work, args=(n, together)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for n in range(4):
        assert all(torch.equal(a, b) for a, b in zip(alone[n], together[n]))
    assert kq.device_status() == 0


FIRST = """
import sys, torch
import w4a4_post_quantization_b200 as kq
what = sys.argv[1]
dev = "cuda:0"
cache = kq.cache_alloc(40, 16, 2, 64, device=dev)
table = torch.arange(40, dtype=torch.int32, device=dev).view(1, 40)
lens = torch.tensor([600], dtype=torch.int32, device=dev)
x = torch.randn((1, 600, 2, 64), device=dev).to(torch.bfloat16)
codes = torch.randint(0, 256, (256, 64), dtype=torch.uint8, device=dev)
scales = torch.full((1024,), 127, dtype=torch.uint8, device=dev)
calls = dict(write=lambda: kq.cache_write(cache, table, x, x).v_codes, read=lambda: kq.cache_read(cache, table, lens, 600)[0],
             few=lambda: kq.attention_mxfp4(x[:, :1], cache, table, lens),
             many=lambda: kq.attention_mxfp4(x, cache, table, lens),
             product=lambda: kq.gemm_mxfp4_epilogue(codes, scales, codes, scales, activation="gelu"),
             narrow=lambda: kq.gemm_mxfp4_epilogue(codes, scales, codes, scales, out_dtype=torch.float32))
f = calls[what]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = f()
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, f()) and kq.device_status() == 0
print("ok")
"""


@pytest.mark.parametrize("what", ["write", "read", "few", "many", "product", "narrow"])
def test_the_first_call_of_a_process_can_be_captured(what):
    run = subprocess.run([sys.executable, "-c", FIRST, what], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stderr[-2000:]


def test_float32_rows_read_into_strided_outputs():
    B, T, H, D = 2, 37, 3, 40
    cache = kq.cache_alloc(6, 16, H, D, device=DEV)
    table = i32([[0, 1, 2], [5, 4, 3]])
    k, v = rows((B, T, H, D), 1), rows((B, T, H, D), 2)
    kq.cache_write(cache, table, k, v)
    fused = torch.full((B, H, T + 2, 2 * D), 7.0, device=DEV)
    a, b = (fused[:, :, 1:-1, i * D:(i + 1) * D].transpose(1, 2) for i in range(2))
    gk, gv = kq.cache_read(cache, table, i32([T, 20]), T, out_dtype=torch.float32, k=a, v=b)
    want = round_trip(k)
    want[1, 20:] = 0
    assert gk.data_ptr() == a.data_ptr() and np.array_equal(a.double().cpu().numpy(), want)
    want = round_trip(v)
    want[1, 20:] = 0
    assert np.array_equal(b.double().cpu().numpy(), want)
    assert (fused[:, :, 0] == 7).all() and (fused[:, :, -1] == 7).all()


@pytest.mark.parametrize("M", [1, 30, 100])
@pytest.mark.parametrize("max_len", [1, 15, 17, 129])
def test_short_bounds_and_a_query_shared_by_the_batch(M, max_len):
    B, H, D, L = 3, 4, 56, 140
    cache, table, k, v = make_cache(B, L, 2, D, 16, seed=M)
    kd, vd = fill(cache, table, k, v, [L] * B)
    q = queries(1, M, H, D, 4).expand(B, M, H, D)
    lens = [L, 16, 0]
    lse = torch.empty((B, H, M), device=DEV)
    out = kq.attention_mxfp4(q.to(DEV)[:1].expand(B, M, H, D), cache, table, i32(lens), causal=True, max_len=max_len, lse=lse)
    assert kq.device_status() == 0
    check(out, lse, q.double().numpy(), kd, vd, [min(n, max_len) for n in lens], True)
