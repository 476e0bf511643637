"""The W4A4 product with its epilogue against the float64 oracle.

Tolerance, from the arithmetic: the product is within (K/64 + 1) 2^-22 of its
terms' magnitudes (test_gpu_gemm.py); adding the bias rounds once, 2^-24; an
activation's slope is below 1.2 and its own error 2e-6 max(|y|, 1); the gate's
product and the residual's sum round once each, 2^-24 of their values; bf16
rounds once more, 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import kq_block as ob
from oracle import kq_oracle as o

pytestmark = pytest.mark.gpu

kq = pytest.importorskip("w4a4_post_quantization_b200")
DEV = "cuda:0"


def operands(M, N, K, seed):
    """Random codes; scales that give outputs of a few units, both signs."""
    rng = np.random.default_rng([seed, 5])
    qa = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
    qb = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    sa = rng.integers(124, 127, (M, K // 32), dtype=np.uint8)
    sb = rng.integers(121, 125, (N, K // 32), dtype=np.uint8)
    return qa, sa, qb, sb


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def tiled(s, K):
    return kq.scales_to_tiled(dev(s), K)


def bf16(shape, seed, gain=1.0):
    x = np.random.default_rng([seed, 9]).normal(size=shape) * gain
    return torch.from_numpy(x).to(torch.bfloat16)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def expect(ops, K, bias, act, gate, tokens, residual):
    """(value, tolerance of the float32 result)."""
    y, mag = o.mxfp4_gemm(*ops), o.abs_mxfp4_gemm(*ops)
    d = (K / 64 + 1) * 2.0 ** -22 * mag
    if bias is not None:
        y = y + f64(bias)
        d = d + 2.0 ** -24 * np.abs(y)
    if act != "none":
        d = 1.2 * d + 2e-6 * np.maximum(1, np.abs(y))
        y = ob.activation(y, act)
    if gate is not None:
        g = f64(gate)[np.arange(y.shape[0]) // tokens]
        y, d = y * g, d * np.abs(g) + 2.0 ** -24 * np.abs(y * g)
    if residual is not None:
        y = y + f64(residual)
        d = d + 2.0 ** -24 * np.abs(y)
    return y, d * (1 + 2.0 ** -10) + 2.0 ** -126


def check(got, want, tol, dt):
    if dt == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    g = f64(got)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(),
                           [(float(g[tuple(i)]), float(want[tuple(i)])) for i in np.argwhere(bad)[:5]])


def run(M, N, K, act="none", bias=True, gate=True, residual=True, tokens=None, dt=torch.bfloat16, seed=0):
    ops = operands(M, N, K, seed + M + N + K)
    tokens = tokens or max(1, M // 3)
    b = bf16((N,), seed + 1) if bias else None
    g = bf16((-(-M // tokens), N), seed + 2) if gate else None
    r = bf16((M, N), seed + 3, 3.0).to(dt) if residual else None
    if r is not None and dt == torch.float32:
        r = r + torch.from_numpy(np.random.default_rng(seed).normal(size=(M, N))).float() * 1e-3
    want, tol = expect(ops, K, b, act, g, tokens, r)
    call = dict(bias=None if b is None else b.to(DEV), activation=act, gate=None if g is None else g.to(DEV),
                tokens_per_sample=tokens if gate else None, out_dtype=dt)
    args = dev(ops[0]), tiled(ops[1], K), dev(ops[2]), tiled(ops[3], K)
    got = kq.gemm_mxfp4_epilogue(*args, residual=None if r is None else r.to(DEV), **call)
    check(got, want, tol, dt)
    if r is not None:                                          # in place, the same bits
        x = r.to(DEV)
        assert kq.gemm_mxfp4_epilogue(*args, residual=x, out=x, **call) is x
        assert torch.equal(x, got)
    assert kq.device_status() == 0
    return got


SHAPES = [(1, 1, 32), (1, 8, 64), (3, 200, 96), (128, 128, 256), (130, 264, 544), (257, 520, 1152),
          (300, 77, 160), (64, 129, 2240), (255, 1000, 320), (511, 250, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_everything_at_once(M, N, K, dt):
    run(M, N, K, act="gelu_tanh", dt=dt)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu", "silu"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [136, 131])
def test_activations(act, dt, N):
    run(200, N, 192, act=act, dt=dt, seed=3)
    run(200, N, 192, act=act, dt=dt, bias=False, gate=False, residual=False, seed=4)


@pytest.mark.parametrize("bias,gate,residual", [(b, g, r) for b in (0, 1) for g in (0, 1) for r in (0, 1)])
@pytest.mark.parametrize("N", [264, 90])
def test_each_part_alone_and_together(bias, gate, residual, N):
    for dt in (torch.bfloat16, torch.float32):
        run(150, N, 128, act="silu", bias=bias, gate=gate, residual=residual, dt=dt, seed=7)


@pytest.mark.parametrize("tokens", [1, 7, 32, 100, 149, 150, 100000])
def test_samples_change_inside_a_tile(tokens):
    run(150, 72, 64, tokens=tokens, seed=tokens)


@pytest.mark.parametrize("M,N,K", [(2500, 3832, 96), (2560, 3840, 544), (2500, 3830, 64), (5000, 4608, 32)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_many_tiles(M, N, K, dt):
    """Several tiles a CTA pair, and both tile widths."""
    run(M, N, K, dt=dt, seed=11)


@pytest.mark.parametrize("M,N,K", [(300, 520, 544), (2560, 3840, 1152), (1, 64, 12320), (130, 77, 96)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_nothing_added_is_the_product_itself(M, N, K, dt):
    """Without an epilogue the same MMAs give gemm_mxfp4_tiled's bits."""
    ops = operands(M, N, K, 13)
    args = dev(ops[0]), tiled(ops[1], K), dev(ops[2]), tiled(ops[3], K)
    assert torch.equal(kq.gemm_mxfp4_epilogue(*args, out_dtype=dt), kq.gemm_mxfp4_tiled(*args, out_dtype=dt))


def test_activations_far_out():
    """Accumulators of +-2^20 and 0: the activations saturate, with no NaN."""
    K, M = 32, 128
    q = np.full((M, K // 2), 0x22, np.uint8)
    q[1::2] = 0xAA                                              # -1
    q[2::4] = 0
    sa = np.full((M, 1), 127 + 15, np.uint8)
    qb, sb = np.full((8, K // 2), 0x22, np.uint8), np.full((8, 1), 127, np.uint8)
    args = dev(q), tiled(sa, K), dev(qb), tiled(sb, K)
    for act in ("gelu_tanh", "gelu", "silu"):
        y = f64(kq.gemm_mxfp4_epilogue(*args, activation=act, out_dtype=torch.float32))
        assert (y[0::4] == 2.0 ** 20).all() and (y[2::4] == 0).all()
        assert (np.abs(y[1::2]) <= 2.0 ** -38).all()


def test_the_gate_of_zero_and_a_residual_alone():
    M, N, K = 140, 96, 64
    ops = operands(M, N, K, 17)
    r = bf16((M, N), 18).to(DEV)
    args = dev(ops[0]), tiled(ops[1], K), dev(ops[2]), tiled(ops[3], K)
    zero = torch.zeros((1, N), dtype=torch.bfloat16, device=DEV)
    assert torch.equal(kq.gemm_mxfp4_epilogue(*args, gate=zero, tokens_per_sample=M, residual=r), r)


def test_a_whole_output_stays_inside_its_rows():
    """Rows and columns around the output keep their bytes, with and without
    TMA's boxes."""
    for M, N in ((100, 200), (100, 203)):
        ops = operands(M, N, 64, 19)
        args = dev(ops[0]), tiled(ops[1], 64), dev(ops[2]), tiled(ops[3], 64)
        buf = torch.full((M * N + 128,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = buf[64:64 + M * N].view(M, N)
        kq.gemm_mxfp4_epilogue(*args, out=out)
        assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
        assert torch.equal(out, kq.gemm_mxfp4_epilogue(*args))


def test_the_longest_product():
    """2^21 products of ones a sum: exact in float32.  One more block is refused."""
    M, N, K = 4, 8, 1 << 21
    s = torch.full((128 * (K // 32) + 512,), 127, dtype=torch.uint8, device=DEV)   # one tile of 128 rows
    qa, qb = (torch.full((r, K // 2), 0x22, dtype=torch.uint8, device=DEV) for r in (M, N))
    out = kq.gemm_mxfp4_epilogue(qa, s[:-512], qb, s[:-512], out_dtype=torch.float32)
    assert kq.device_status() == 0
    assert bool((out == K).all())
    longer = [torch.full((r, K // 2 + 16), 0x22, dtype=torch.uint8, device=DEV) for r in (M, N)]
    with pytest.raises((ValueError, kq.KQError)):
        kq.gemm_mxfp4_epilogue(longer[0], s, longer[1], s)


def test_empty_and_refusals():
    e = torch.empty((0, 32), dtype=torch.uint8, device=DEV)
    s0 = torch.empty((0,), dtype=torch.uint8, device=DEV)
    ops = operands(16, 24, 64, 23)
    args = dev(ops[0]), tiled(ops[1], 64), dev(ops[2]), tiled(ops[3], 64)
    assert kq.gemm_mxfp4_epilogue(e, s0, args[2], args[3]).shape == (0, 24)
    b = torch.zeros(24, dtype=torch.bfloat16, device=DEV)
    g, r = b.view(1, 24), torch.zeros((16, 24), dtype=torch.bfloat16, device=DEV)
    two = torch.zeros((40, 24), dtype=torch.bfloat16, device=DEV)
    f = kq.gemm_mxfp4_epilogue
    for bad in (lambda: f(*args, bias=b.float()), lambda: f(*args, bias=b[:23]), lambda: f(*args, gate=g),
                lambda: f(*args, gate=g, tokens_per_sample=0), lambda: f(*args, gate=g, tokens_per_sample=8),
                lambda: f(*args, residual=r.float()), lambda: f(*args, residual=r[:8]),
                lambda: f(*args, residual=r, out_dtype=torch.float32), lambda: f(*args, activation="relu"),
                lambda: f(*args, out_dtype=torch.float16), lambda: f(args[0], args[1][:100], *args[2:]),
                lambda: f(*args, residual=two[:16], out=two[8:24]), lambda: f(args[0].cpu(), *args[1:])):
        with pytest.raises(ValueError):
            bad()


def test_replays_from_a_graph():
    M, N, K = 300, 264, 320
    ops = operands(M, N, K, 29)
    args = dev(ops[0]), tiled(ops[1], K), dev(ops[2]), tiled(ops[3], K)
    b, r = bf16((N,), 30).to(DEV), bf16((M, N), 31).to(DEV)
    want = kq.gemm_mxfp4_epilogue(*args, bias=b, activation="gelu", residual=r)
    x = torch.empty_like(r)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        kq.gemm_mxfp4_epilogue(*args, bias=b, activation="gelu", residual=x, out=x)
    for _ in range(3):
        x.copy_(r)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    assert kq.device_status() == 0
    del g
