"""The cache and attention entry points reject bad arguments on the host,
before any CUDA call, and their binding refuses tensors it cannot pass."""
import ctypes

import pytest
import torch

FAKE = 0x10000          # 16-byte aligned, never dereferenced: checks fail first


@pytest.fixture(scope="module")
def L():
    from w4a4_post_quantization_b200 import build
    build.build()
    from w4a4_post_quantization_b200 import _lib
    return _lib


def cache(L, **kw):
    f = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, pages=4, page_size=16, heads=2,
             head_dim=64)
    f.update(kw)
    return L._CacheStruct(**f)


BAD_CACHES = [dict(k_codes=None), dict(v_scales=None), dict(k_codes=FAKE + 8), dict(v_scales=FAKE + 1),
              dict(pages=0), dict(pages=1 << 31), dict(page_size=8), dict(page_size=48),
              dict(page_size=131072), dict(heads=0), dict(heads=65536), dict(head_dim=0),
              dict(head_dim=36), dict(head_dim=136)]


def write(L, c, table=FAKE, batch=2, pages=3, k=FAKE, ks=(256, 128, 64), v=FAKE, vs=(256, 128, 64),
          tokens=2, start=None, lens=None):
    return L.lib().kq_cache_write(ctypes.byref(c), table, batch, pages, k, *ks, v, *vs, tokens, start,
                                  lens, None)


def read(L, c, table=FAKE, batch=2, pages=3, k=FAKE, ks=(256, 128, 64), v=FAKE, vs=(256, 128, 64),
         tokens=2, start=None, lens=None, dtype=1):
    return L.lib().kq_cache_read(ctypes.byref(c), table, batch, pages, tokens, start, lens, k, *ks, v,
                                 *vs, dtype, None)


def attend(L, c, q=FAKE, qs=(256, 128, 64), batch=2, M=2, heads=2, table=FAKE, pages=3, lens=FAKE,
           max_len=48, scale=0.1, causal=0, out=FAKE, os_=(256, 128, 64), lse=None, ws=None, nbytes=0):
    return L.lib().kq_attention_mxfp4(q, *qs, batch, M, heads, ctypes.byref(c), table, pages, lens,
                                      max_len, scale, causal, out, *os_, lse, ws, nbytes, None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(L, bad):
    c = cache(L, **bad)
    for f in (write, read, attend):
        assert f(L, c) == 1


@pytest.mark.parametrize("bad", [dict(table=None), dict(table=FAKE + 2), dict(batch=-1), dict(batch=65536),
                                 dict(pages=0), dict(pages=1 << 31), dict(pages=1 << 28), dict(k=None),
                                 dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ks=(256, 4, 64)),
                                 dict(vs=(-8, 128, 64)), dict(tokens=-1), dict(tokens=1 << 31),
                                 dict(start=FAKE + 1), dict(lens=FAKE + 2)], ids=str)
def test_bad_rows(L, bad):
    assert write(L, cache(L), **bad) == 1
    assert read(L, cache(L), **bad) == 1


def test_bad_read_type(L):
    assert read(L, cache(L), dtype=2) == 1
    assert read(L, cache(L), dtype=0, ks=(256, 128, 66)) == 1


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=FAKE + 8), dict(qs=(256, 128, 60)), dict(batch=-1),
                                 dict(M=-1), dict(heads=3), dict(heads=0), dict(table=None),
                                 dict(lens=None), dict(lens=FAKE + 2), dict(max_len=0),
                                 dict(max_len=49), dict(scale=float("nan")), dict(pages=1 << 27, max_len=(1 << 30) + 1), dict(scale=float("inf")),
                                 dict(out=None), dict(out=FAKE + 4), dict(os_=(256, 128, -64)),
                                 dict(lse=FAKE + 2), dict(M=1 << 31)], ids=str)
def test_bad_attention(L, bad):
    assert attend(L, cache(L), **bad) == 1


def test_workspace_is_checked(L):
    size = L.lib().kq_attention_workspace_bytes
    need = size(1, 1, 32, 8, 128, 65536)
    assert need > 0
    c = cache(L, heads=8, head_dim=128, page_size=64)
    kw = dict(batch=1, M=1, heads=32, pages=1024, max_len=65536, qs=(4096, 4096, 128),
              os_=(4096, 4096, 128))
    assert attend(L, c, **kw) == 1                               # none given
    assert attend(L, c, ws=FAKE, nbytes=need - 1, **kw) == 1
    assert attend(L, c, ws=FAKE + 64, nbytes=need, **kw) == 1
    for bad in ((0, 1, 8, 8, 64, 10), (1, 0, 8, 8, 64, 10), (1, 1, 6, 4, 64, 10), (1, 1, 8, 8, 60, 10),
                (1, 1, 8, 8, 64, 0)):
        assert size(*bad) == 0


def test_empty_calls_need_no_device(L):
    c = cache(L)
    assert write(L, c, tokens=0) == 0 and write(L, c, batch=0) == 0
    assert read(L, c, tokens=0) == 0 and read(L, c, batch=0) == 0
    assert attend(L, c, M=0) == 0 and attend(L, c, batch=0) == 0


def test_binding_refuses_host_tensors(L):
    t = torch.zeros((2, 2, 16, 32), dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.KVCache(t, t[..., :2].contiguous(), t, t[..., :2].contiguous(), 64)
    with pytest.raises(ValueError):
        L.KVCache(t, t, t, t, 60)
    u8 = torch.zeros((16, 32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="qa must be a CUDA tensor"):
        L.gemm_mxfp4_epilogue(u8, u8, u8, u8)
    with pytest.raises(ValueError, match="qa must be a CUDA tensor"):
        L.gemm_mxfp4_epilogue(None, u8, u8, u8)
    with pytest.raises(ValueError, match="activation"):
        L.gemm_mxfp4_epilogue(u8, u8, u8, u8, activation="relu")


def epilogue(L, qa=FAKE, sa=FAKE, qb=FAKE, sb=FAKE, M=4, N=8, K=64, bias=None, act=0, gate=None, tokens=0,
             residual=None, c=FAKE, dtype=1):
    return L.lib().kq_gemm_mxfp4_epilogue(qa, sa, qb, sb, M, N, K, bias, act, gate, tokens, residual, c,
                                          dtype, None)


@pytest.mark.parametrize("bad", [dict(qa=None), dict(qa=FAKE + 8), dict(sa=FAKE + 4), dict(qb=FAKE + 1),
                                 dict(sb=None), dict(M=-1), dict(N=-1), dict(K=0), dict(K=48),
                                 dict(M=(1 << 31) - 1), dict(M=1 << 30, N=1 << 30), dict(bias=FAKE + 2),
                                 dict(act=-1), dict(act=4), dict(gate=FAKE, tokens=0),
                                 dict(gate=FAKE + 2, tokens=4), dict(residual=FAKE + 4), dict(c=None),
                                 dict(c=FAKE + 8), dict(dtype=2)], ids=str)
def test_bad_epilogue(L, bad):
    assert epilogue(L, **bad) == 1


def test_empty_epilogue_needs_no_device(L):
    assert epilogue(L, M=0, qa=None, c=None) == 0 and epilogue(L, N=0, qb=None, c=None) == 0


def test_epilogue_bound_of_k(L):
    assert epilogue(L, K=(1 << 21) + 32) == 1
