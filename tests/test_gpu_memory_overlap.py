"""Outputs that share memory with one another or with an input are refused; slices of one
buffer that lie between each other are not."""
import itertools

import numpy as np
import pytest
import torch

from test_gpu_attention import DEV, i32, queries

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")


def view(buf, offset, shape, strides):
    return torch.as_strided(buf, shape, strides, offset)


def elements(t):
    at = t.storage_offset()
    for n, s in zip(t.shape, t.stride()):
        at = np.add.outer(at, np.arange(n) * s)
    return set(np.asarray(at).ravel().tolist())


def layouts(rng):
    """Nested strides of [batch, rows, heads, 8]: the dimensions in any order, with
    space between them now and then."""
    shape = [int(rng.integers(1, 4)) for _ in range(3)] + [8]
    strides, step = [0, 0, 0, 1], 8
    for i in rng.permutation(3):
        step += 8 * int(rng.integers(0, 3))
        strides[i] = step
        step *= shape[i] if shape[i] > 1 else 1
    return shape, strides, step


def cases():
    rng = np.random.default_rng(5)
    for _ in range(400):
        shape, strides, step = layouts(rng)
        yield shape, strides, 8 * int(rng.integers(0, step // 8 + 2))


def test_read_into_slices_of_one_buffer():
    cache = kq.cache_alloc(4, 16, 3, 8, device=DEV)
    x = queries(3, 16, 3, 8, 1).to(DEV)
    table3 = i32([[0], [1], [2]])
    seen = {True: 0, False: 0}
    buf = torch.zeros(1 << 16, dtype=torch.bfloat16, device=DEV)
    for shape, strides, d in cases():
        B, T, H, D = shape
        if H != 3:
            continue
        k, v = view(buf, 0, shape, strides), view(buf, d, shape, strides)
        shared = bool(elements(k) & elements(v))
        seen[shared] += 1
        kq.cache_write(cache, table3[:B], x[:B, :T].contiguous(), (-x[:B, :T]).contiguous())
        for a, b in ((k, v), (v, k)):
            if shared:
                with pytest.raises(ValueError, match="k and v"):
                    kq.cache_read(cache, table3[:B], None, T, k=a, v=b)
            else:
                kq.cache_read(cache, table3[:B], None, T, k=a, v=b)
                want = kq.cache_read(cache, table3[:B], None, T)
                assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert min(seen.values()) > 10 and kq.device_status() == 0


def test_output_and_queries_in_one_buffer():
    cache = kq.cache_alloc(4, 16, 1, 8, device=DEV)
    x = queries(3, 16, 1, 8, 1).to(DEV)
    table = i32([[0], [1], [2]])
    kq.cache_write(cache, table, x, x)
    seen = {True: 0, False: 0}
    buf = torch.randn(1 << 16, device=DEV).to(torch.bfloat16)
    for shape, strides, d in cases():
        B = shape[0]
        q, out = view(buf, 0, shape, strides), view(buf, d, shape, strides)
        shared = bool(elements(q) & elements(out))
        seen[shared] += 1
        lens = i32([16] * B)
        if shared:
            with pytest.raises(ValueError, match="out and q"):
                kq.attention_mxfp4(q, cache, table[:B], lens, out=out)
        else:
            want = kq.attention_mxfp4(q.clone(), cache, table[:B], lens)
            assert kq.attention_mxfp4(q, cache, table[:B], lens, out=out) is out
            assert torch.equal(out, want)
    assert min(seen.values()) > 10 and kq.device_status() == 0


def test_other_layouts_lse_and_workspace():
    B, M, H, D, L = 2, 70, 2, 64, 64
    cache = kq.cache_alloc(8, 16, 2, D, device=DEV)
    table, lens = i32(np.arange(8).reshape(2, 4)), i32([L, L])
    need = kq.attention_workspace_bytes(B, M, H, 2, D, L)
    n = B * M * H * D
    buf = torch.zeros(8 * n + need + 512, dtype=torch.uint8, device=DEV)
    q = buf[:2 * n].view(torch.bfloat16).view(B, M, H, D)
    out = buf[2 * n:4 * n].view(torch.bfloat16).view(B, M, H, D)
    lse = buf[4 * n:4 * n + 4 * B * M * H].view(torch.float32).view(B, H, M)
    ws = buf[-need - 256:]
    ws = ws[-ws.data_ptr() % 256:][:need]
    f = lambda **kw: kq.attention_mxfp4(q, cache, table, lens, **kw)  # noqa: E731
    want = f()
    assert torch.equal(f(out=out, lse=lse, workspace=ws), want)
    over = buf[2 * n - 64:4 * n - 64].view(torch.bfloat16).view(B, M, H, D)
    turned = buf[2 * n - 64:4 * n - 64].view(torch.bfloat16).view(B, H, M, D).transpose(1, 2)
    at = lambda b: buf[b:b + 4 * B * M * H].view(torch.float32).view(B, H, M)  # noqa: E731
    for bad in (dict(out=over), dict(out=turned), dict(lse=at(0)), dict(out=out, lse=at(2 * n)),
                dict(workspace=buf[:need]), dict(out=out, workspace=buf[4 * n - 256:][:need]),
                dict(lse=lse, workspace=buf[4 * n:][:need])):
        with pytest.raises(ValueError, match="memory"):
            f(**bad)
    expanded = q[:, :1].expand(B, M, H, D)
    assert torch.equal(kq.attention_mxfp4(expanded, cache, table, lens, out=out),
                       kq.attention_mxfp4(expanded.contiguous(), cache, table, lens))
    with pytest.raises(ValueError, match="out and q"):
        kq.attention_mxfp4(expanded, cache, table, lens, out=q)
    assert kq.device_status() == 0


def test_what_the_cases_cover():
    """The brute-force sets above meet in every way the exact test distinguishes."""
    kinds = set()
    for shape, strides, d in itertools.islice(cases(), 400):
        buf = torch.zeros(1 << 16, dtype=torch.bfloat16)
        a, b = elements(view(buf, 0, shape, strides)), elements(view(buf, d, shape, strides))
        kinds.add((bool(a & b), max(a) < min(b)))
    assert kinds == {(True, False), (False, False), (False, True)}
