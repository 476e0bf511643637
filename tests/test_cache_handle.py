"""A KVCache names its tensors' memory once, when it is made: what it holds cannot be
exchanged behind its back."""
import pytest
import torch

FIELDS = ["k_codes", "k_scales", "v_codes", "v_scales", "pages", "page_size", "heads", "head_dim", "device"]


@pytest.fixture(scope="module")
def L():
    from w4a4_post_quantization_b200 import build
    build.build()
    from w4a4_post_quantization_b200 import _lib
    return _lib


def host_cache(L, D=64):
    """A KVCache over host tensors, which its constructor refuses: for the checks in
    front of a call, none of which reads the memory."""
    nb = -(-D // 32)
    c = object.__new__(L.KVCache)
    c._tensors = tuple(torch.zeros((4, 2, 16, n), dtype=torch.uint8) for n in (16 * nb, nb, 16 * nb, nb))
    c._c = L._CacheStruct(*(t.data_ptr() for t in c._tensors), 4, 16, 2, D)
    c._ptr, c._index = L.ctypes.addressof(c._c), 0
    return c


@pytest.mark.parametrize("name", FIELDS)
def test_fields_cannot_be_assigned(L, name):
    c = host_cache(L)
    value = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, value)
    assert getattr(c, name) is value or getattr(c, name) == value


def calls(L, c):
    t = torch.zeros((1, 1), dtype=torch.int32)
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    return (lambda: L.cache_write(c, t, x, x), lambda: L.cache_read(c, t, None, 1),
            lambda: L.attention_mxfp4(x, c, t, t[0]))


MOVES = {"storage": lambda t: t.untyped_storage().resize_(0), "data": lambda t: setattr(t, "data", torch.zeros_like(t)),
         "set": lambda t: t.set_(torch.zeros(t.numel(), dtype=torch.uint8)),
         "grown": lambda t: t.resize_(1 << 20),
         "half": lambda t: t.untyped_storage().resize_(t.numel() // 2)}


@pytest.mark.parametrize("move", MOVES)
@pytest.mark.parametrize("which", range(4))
def test_other_memory_is_refused(L, move, which):
    c = host_cache(L)
    for f in calls(L, c):                                     # so far it is the memory that is refused
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    MOVES[move](c._tensors[which])
    for f in calls(L, c):
        with pytest.raises(ValueError, match="KVCache"):
            f()


@pytest.mark.gpu
def test_a_grown_pool_is_another_cache():
    import w4a4_post_quantization_b200 as kq
    cache = kq.cache_alloc(2, 16, 2, 64, device="cuda:0")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda:0")
    k = torch.randn((1, 32, 2, 64), device="cuda:0").to(torch.bfloat16)
    kq.cache_write(cache, table, k, k)
    want = kq.cache_read(cache, table, None, 32)
    bigger = [torch.cat((t, torch.zeros_like(t))) for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    with pytest.raises(AttributeError):
        cache.k_codes = bigger[0]
    grown = kq.KVCache(*bigger, 64)
    assert (grown.pages, cache.pages) == (4, 2)
    assert all(torch.equal(a, b) for a, b in zip(kq.cache_read(grown, table, None, 32), want))
    cache.k_codes.data = bigger[0]
    for f in (lambda: kq.cache_write(cache, table, k, k), lambda: kq.cache_read(cache, table, None, 32),
              lambda: kq.attention_mxfp4(k, cache, table, table[0, 1:])):
        with pytest.raises(ValueError, match="KVCache"):
            f()
    assert kq.device_status() == 0
