"""The block operators together, as a W4A4 transformer block uses them: the
prompt's K and V projected and cached once, then per step the queries projected,
the cross attention, the output projection onto the residual stream, and the
gated MLP.  Every stage is checked against the float64 oracle on the inputs that
the stage before it gave, and the whole step replays from a graph while the
prompt's cache stays."""
import numpy as np
import pytest
import torch

import workloads as w
from oracle import kq_block as ob
from test_gpu_attention import check as check_attention
from test_gpu_epilogue import check as check_linear
from test_gpu_epilogue import expect

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"


class Linear:
    """A W4A4 layer: folded, quantized weight, the activation transform, bias."""

    def __init__(self, n, d, seed):
        rng = np.random.default_rng([seed, 1])
        p = np.stack([rng.uniform(-1, 1, (d // 32, 5)), 2.0 ** rng.uniform(-1, 1, (d // 32, 5)),
                      rng.uniform(-1, 1, (d // 32, 5))], -1)
        self.params = torch.from_numpy(p.astype(np.float32)).to(DEV)
        self.weight = w.draw_weight(n, d, seed).to(DEV)
        self.q, self.s = kq.quantize_weight_tiled(self.weight, self.params)
        self.row_s = kq.quantize_weight(self.weight, self.params)[1]
        self.bias = torch.from_numpy(rng.normal(size=n) * 0.2).to(torch.bfloat16).to(DEV)

    def operands(self, x):
        return kq.quantize_tiled(x, self.params)

    def __call__(self, x, **kw):
        return kq.gemm_mxfp4_epilogue(*self.operands(x), self.q, self.s, bias=self.bias, **kw)

    def verify(self, got, x, act="none", gate=None, tokens=1, residual=None):
        """The product's epilogue on the codes that the quantizers gave."""
        qa, sa = kq.quantize(x, self.params)
        ops = [t.cpu().numpy() for t in (qa, sa, self.q, self.row_s)]
        want, tol = expect(ops, x.shape[1], self.bias, act, gate, tokens, residual)
        check_linear(got, want, tol, got.dtype)


def test_a_block_over_a_cached_prompt():
    B, T, L, H, D, F = 2, 150, 40, 4, 72, 640
    d = H * D                                                  # 288
    rng = np.random.default_rng(1)

    def bf16(*shape, gain=1.0):
        return torch.from_numpy(rng.normal(size=shape) * gain).to(torch.bfloat16).to(DEV)

    to_kv, to_q, to_out = Linear(2 * d, 320, 2), Linear(d, d, 3), Linear(d, d, 4)
    up, down = Linear(F, d, 5), Linear(d, F, 6)
    text, x0 = bf16(B * L, 320), bf16(B * T, d)
    shift, scale, gate = bf16(B, d, gain=0.3), bf16(B, d, gain=0.3), bf16(B, d)
    lens = torch.tensor([L, 23], dtype=torch.int32, device=DEV)
    cache = kq.cache_alloc(2 * B + 1, 32, H, D, device=DEV)
    table = torch.tensor([[4, 0], [3, 1]], dtype=torch.int32, device=DEV)

    # The prompt, once.
    kv = to_kv(text)
    to_kv.verify(kv, text)
    rows = kv.view(B, L, 2 * H, D)
    kq.cache_write(cache, table, rows[:, :, :H], rows[:, :, H:], lens=lens)
    kd, vd = (t.double().cpu().numpy() for t in kq.cache_read(cache, table, lens, L))
    for got, part in ((kd, rows[:, :, :H]), (vd, rows[:, :, H:])):
        q, s = ob.quantize_rows(part.double().cpu().numpy())
        want = ob.decode_rows(q, s, D)
        want[1, 23:] = 0
        assert np.array_equal(got, want)

    def step(x, keep=None):
        q = to_q(x)
        o = kq.attention_mxfp4(q.view(B, T, H, D), cache, table, lens)
        x1 = to_out(o.view(B * T, d), residual=x)
        a, sa = kq.quantize_adaln_tiled(x1, shift, scale, T, up.params)
        h = kq.gemm_mxfp4_epilogue(a, sa, up.q, up.s, bias=up.bias, activation="gelu_tanh")
        x2 = down(h, gate=gate, tokens_per_sample=T, residual=x1)
        if keep is not None:
            keep.update(q=q, o=o, x1=x1, h=h)
        return x2

    st = {}
    x2 = step(x0, st)
    torch.cuda.synchronize()
    to_q.verify(st["q"], x0)
    check_attention(st["o"], None, st["q"].view(B, T, H, D).double().cpu().numpy(), kd, vd, [L, 23], False)
    to_out.verify(st["x1"], st["o"].view(B * T, d), residual=x0)
    qa, sa = kq.quantize_adaln(st["x1"], shift, scale, T, up.params)
    want, tol = expect([t.cpu().numpy() for t in (qa, sa, up.q, up.row_s)], d, up.bias, "gelu_tanh", None, 1, None)
    check_linear(st["h"], want, tol, torch.bfloat16)
    down.verify(x2, st["h"], gate=gate, tokens=T, residual=st["x1"])

    # The step as a graph, on another input and a shorter prompt.
    x = x0.clone()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(x)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            y = step(x)
    x.copy_(bf16(B * T, d))
    lens.copy_(torch.tensor([7, 0], dtype=torch.int32))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, step(x))
    assert kq.device_status() == 0
    del g


def test_decoding_token_by_token_matches_the_prompt_at_once():
    """A causal prompt in one call, and the same positions one by one, the cache
    growing: the same attention."""
    B, T, H, Hkv, D = 2, 70, 8, 2, 64
    rng = np.random.default_rng(3)
    q, k, v = (torch.from_numpy(rng.normal(size=(B, T, h, D))).to(torch.bfloat16).to(DEV) for h in (H, Hkv, Hkv))
    table = torch.arange(2 * 5, dtype=torch.int32, device=DEV).view(2, 5)
    whole, grown = (kq.cache_alloc(10, 16, Hkv, D, device=DEV) for _ in range(2))
    kq.cache_write(whole, table, k, v)
    full = torch.full((B,), T, dtype=torch.int32, device=DEV)
    at_once = kq.attention_mxfp4(q, whole, table, full, causal=True)
    kd, vd = (t.double().cpu().numpy() for t in kq.cache_read(whole, table, None, T))
    check_attention(at_once, None, q.double().cpu().numpy(), kd, vd, [T, T], True)
    for t in range(T):
        start = torch.full((B,), t, dtype=torch.int32, device=DEV)
        kq.cache_write(grown, table, k[:, t:t + 1], v[:, t:t + 1], start=start)
        one = kq.attention_mxfp4(q[:, t:t + 1], grown, table, start + 1, causal=True)
        check_attention(one, None, q[:, t:t + 1].double().cpu().numpy(), kd, vd, [t + 1] * B, True)
    assert torch.equal(whole.k_codes, grown.k_codes) and torch.equal(whole.v_scales, grown.v_scales)
    assert kq.device_status() == 0
