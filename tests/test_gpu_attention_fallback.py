"""Many query rows where the decoded tiles would pass 4 GiB, or there are 32768 K/V heads
and more: the kernel for few rows takes them, 32 at a time."""
import numpy as np
import pytest
import torch

from test_gpu_attention import DEV, check, fill, i32, make_cache, queries

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")


@pytest.mark.parametrize("M,H,causal", [(300, 8, False), (300, 8, True), (90, 32, True), (513, 8, False)])
def test_a_table_of_more_than_4_gib(M, H, causal):
    """33 short sequences with tables for 32768 positions.  A max_len of what they
    hold takes the other kernel; both are right."""
    B, Hkv, D, L, page = 33, 8, 128, 150, 64
    lens = [max(0, L - 7 * b) for b in range(B)]              # empty ones at the end
    cache, table, k, v = make_cache(B, L, Hkv, D, page, seed=M)
    kd, vd = fill(cache, table, k, v, lens)
    wide = torch.zeros((B, 32768 // page), dtype=torch.int32, device=DEV)
    wide[:, : table.shape[1]] = table
    assert kq.attention_workspace_bytes(B, M, H, Hkv, D, 32768) < 1 << 30 < \
        kq.attention_workspace_bytes(B - 1, M, H, Hkv, D, 32768)
    q = queries(B, M, H, D, 2)
    lse = torch.empty((B, H, M), dtype=torch.float32, device=DEV)
    out = kq.attention_mxfp4(q.to(DEV), cache, wide, i32(lens), causal=causal, lse=lse)
    other = kq.attention_mxfp4(q.to(DEV), cache, wide, i32(lens), causal=causal, max_len=L)
    assert kq.device_status() == 0
    heads = np.arange(0, H, H // 4)                           # the oracle is slow
    kv = heads // (H // Hkv)
    for b in (0, 5, B - 1):
        s = slice(b, b + 1)
        for o, x in ((out, lse[s, heads]), (other, None)):
            check(o[s][:, :, heads], x, q[s][:, :, heads].double().numpy(), kd[s][:, :, kv], vd[s][:, :, kv],
                  [lens[b]], causal)


def test_more_heads_than_a_grid_takes_twice():
    B, M, H, D, L = 1, 300, 32768, 8, 40
    cache = kq.cache_alloc(4, 16, H, D, device=DEV)
    table = i32([[2, 0, 3]])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    k, v, q = (torch.randn((B, n, H, D), generator=gen, device=DEV).to(torch.bfloat16) for n in (L, L, M))
    kq.cache_write(cache, table, k, v)
    kd, vd = kq.cache_read(cache, table, None, L)
    out = kq.attention_mxfp4(q, cache, table, i32([L]), causal=True)
    assert kq.device_status() == 0
    heads = [0, 1, 777, 16384, H - 1]
    check(out[:, :, heads], None, *(x[:, :, heads].double().cpu().numpy() for x in (q, kd, vd)), [L], True)
