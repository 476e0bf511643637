"""Cases of the W4A4 transformer-block operators: the MXFP4 product with its
epilogue, the MXFP4 K/V cache (written and read back) and the attention that
reads it.

A case is measured in two forms: elementary torch operations in float32, and
(where ``own`` is true) the library's calls.  ``exact`` gives the same values
in float64, from the definitions.
"""
import math

import torch

own = False

DEV = "cuda:0"

# Nearest E2M1 magnitudes and the midpoints between them; a tie goes to the
# even code, so every second midpoint belongs to the upper code.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # AdaLN modulation of a two-image batch: all six shifts, scales and
        # gates from the timestep embedding.  Few rows: latency and weights.
        dict(name="linear modulation 2", op="linear", M=2, N=6912, K=1152, act="none", bias=True,
             gate=False, residual=False, tokens=2, out="f32"),
        # MLP up projection of the image tokens, GELU.
        dict(name="linear mlp up", op="linear", M=8192, N=4608, K=1152, act="gelu_tanh", bias=True,
             gate=False, residual=False, tokens=4096, out="bf16"),
        # MLP down projection, gated by AdaLN, added to the residual stream.
        dict(name="linear mlp down", op="linear", M=8192, N=1152, K=4608, act="none", bias=True,
             gate=True, residual=True, tokens=4096, out="bf16"),
        # A ragged token count and an odd width, SiLU, a float32 residual stream.
        dict(name="linear odd silu f32", op="linear", M=3993, N=2241, K=2240, act="silu", bias=True,
             gate=False, residual=True, tokens=1331, out="f32"),
        # The prompt's K and V, written once per image and read back.
        dict(name="cache text", op="cache", B=2, T=300, H=16, D=72, page=64, start=0, ragged=True),
        # One new token for each of 64 sequences.
        dict(name="cache one token", op="cache", B=64, T=1, H=8, D=128, page=64, start=1000,
             ragged=False),
        # A batch of long prompts.
        dict(name="cache prompts", op="cache", B=16, T=4096, H=8, D=128, page=64, start=0,
             ragged=True),
        # Long contexts read back as bf16.
        dict(name="cache read", op="read", B=8, T=8000, H=8, D=128, page=128, start=17, ragged=True),
        dict(name="attention one short", op="attention", B=1, M=1, H=16, Hkv=16, D=72, len=300,
             page=64, causal=False, ragged=False, empty=False),
        # Single-token step of a batch over long contexts, four query heads a K/V head.
        dict(name="attention one long", op="attention", B=8, M=1, H=32, Hkv=8, D=128, len=32768,
             page=64, causal=True, ragged=True, empty=False),
        # Image tokens to the prompt: cross attention of the denoiser.
        dict(name="attention cross", op="attention", B=2, M=4096, H=16, Hkv=16, D=72, len=300,
             page=64, causal=False, ragged=True, empty=False),
        # A prompt chunk against what came before it.
        dict(name="attention chunk", op="attention", B=1, M=2048, H=32, Hkv=8, D=128, len=8192,
             page=64, causal=True, ragged=False, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "cache", "read", "attention", "attention", "attention"])
    if op == "linear":
        while True:
            M, N = _log(rng, 1, 8192), _log(rng, 64, 8192)
            if rng.random() < 0.5:
                N = max(64, N // 32 * 32)
            K = 32 * _log(rng, 2, 256)
            if M * N * K <= 8192 * 4608 * 1152:
                break
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "gelu_tanh", "gelu", "silu"]),
                    bias=rng.random() < 0.8, gate=rng.random() < 0.5, residual=rng.random() < 0.5,
                    tokens=rng.randint(1, M), out=rng.choice(["bf16", "bf16", "f32"]))
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 72, 80, 96, 104, 112, 128])
    if op in ("cache", "read"):
        while True:
            B, T, H = _log(rng, 1, 64), _log(rng, 1, 8192), rng.choice([1, 4, 8, 16, 20])
            if B * T * H * D <= 16 * 4096 * 8 * 128:
                break
        return dict(op=op, B=B, T=T, H=H, D=D, page=page, start=rng.choice([0, rng.randint(1, 3000)]),
                    ragged=rng.random() < 0.7)
    while True:
        Hkv, G = rng.choice([1, 2, 4, 8, 16, 20]), rng.choice([1, 1, 2, 4, 8])
        B, L = _log(rng, 1, 16), _log(rng, 1, 32768)
        M = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        if B * L * Hkv * D <= 8 * 32768 * 8 * 128 and B * M * L * Hkv * G * D <= 2048 * 8192 * 32 * 128 \
                and B * M * Hkv * G * D <= 2 * 4096 * 32 * 128:
            break
    return dict(op=op, B=B, M=M, H=Hkv * G, Hkv=Hkv, D=D, len=L, page=page, causal=rng.random() < 0.5,
                ragged=rng.random() < 0.7, empty=B > 1 and rng.random() < 0.3)


def _lens(c):
    """Rows of each sequence: the longest first, falling to about half of it."""
    B, n = c["B"], c.get("T", c.get("len"))
    lens = [max(1, n - (b * n) // (2 * B)) if c["ragged"] else n for b in range(B)]
    if c.get("empty"):
        lens[-1] = 0
    return lens


# ------------------------------------------------------------------ inputs
def _values(shape, gen, outliers=0.01, gain=8.0):
    """Standard normal values with a share of amplified channels (last axis)."""
    x = torch.randn(shape, generator=gen, device=DEV)
    hot = torch.rand(shape[-1], generator=gen, device=DEV) < outliers
    return torch.where(hot, x * gain, x).to(torch.bfloat16)


def _power(e):
    """2^e in float32, exactly, from the fields of a float64."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _quantize(x):
    """MXFP4 of the last axis in blocks of 32 (padded with zeros): codes two a
    byte, scale bytes.  Float32 throughout; every step is exact."""
    d = x.shape[-1]
    pad = -d % 32
    x = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    a = x.abs() * _power(-e)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code |= torch.signbit(x).to(torch.uint8) << 3
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _tiled(scales):
    """Scale bytes [rows, n] in the product's layout: 128-row x 4-scale tiles."""
    rows, n = scales.shape
    s = torch.nn.functional.pad(scales, (0, -n % 4, 0, -rows % 128))
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4)     # tile, r1, r0, column, i
    return s.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _table(B, pages, gen):
    """Every sequence's pages, scattered over the pool."""
    return torch.randperm(B * pages, generator=gen, device=DEV).to(torch.int32).view(B, pages)


def _pool(total, H, page, D):
    nb = (D + 31) // 32
    return (torch.zeros((total, H, page, 16 * nb), dtype=torch.uint8, device=DEV),
            torch.zeros((total, H, page, nb), dtype=torch.uint8, device=DEV))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        s["qa"], s["sa"] = _quantize(_values((M, K), gen))
        s["qb"], s["sb"] = _quantize((torch.randn((N, K), generator=gen, device=DEV) / K ** 0.5)
                                     .to(torch.bfloat16))
        s["sa_tiled"], s["sb_tiled"] = _tiled(s["sa"]), _tiled(s["sb"])
        dt = torch.float32 if c["out"] == "f32" else torch.bfloat16
        groups = -(-M // c["tokens"])
        s["bias"] = torch.randn(N, generator=gen, device=DEV).to(torch.bfloat16) if c["bias"] else None
        s["gate"] = torch.randn((groups, N), generator=gen, device=DEV).to(torch.bfloat16) \
            if c["gate"] else None
        s["residual"] = torch.randn((M, N), generator=gen, device=DEV).to(dt) if c["residual"] else None
        s["dtype"] = dt
        return s
    B, D, page, lens = c["B"], c["D"], c["page"], _lens(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    H = c["Hkv"] if c["op"] == "attention" else c["H"]
    last = c["len"] if c["op"] == "attention" else c["start"] + c["T"]
    pages = -(-last // page)
    s["table"] = _table(B, pages, gen)
    s["k_codes"], s["k_scales"] = _pool(B * pages, H, page, D)
    s["v_codes"], s["v_scales"] = _pool(B * pages, H, page, D)
    if c["op"] != "attention":
        s["start"] = torch.full((B,), c["start"], dtype=torch.int32, device=DEV)
    if c["op"] == "cache":
        # K and V as the two halves of one projection's output.
        kv = _values((B, c["T"], 2 * H, D), gen)
        s["k"], s["v"] = kv[:, :, :H], kv[:, :, H:]
        return s
    for b in range(B):                                            # one sequence at a time: memory
        at = s["table"][b].long()
        for codes, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])):
            q, sc = _quantize(_values((pages, H, page, D), gen))
            codes[at], scales[at] = q, sc
    if c["op"] == "attention":
        s["q"] = torch.randn((B, c["M"], c["H"], D), generator=gen, device=DEV).to(torch.bfloat16)
    return s


# -------------------------------------------------------------- plain form
def _lut():
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    return torch.stack((v.repeat(16), v.repeat_interleave(16)), -1)      # byte -> (low, high)


def _decode(codes, scales):
    x = _lut()[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    power = _power(torch.arange(-127, 129, device=DEV))
    return (x * power[scales.int()].unsqueeze(-1)).flatten(-2)


def _act(x, act):
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _plain_linear(s):
    c = s["case"]
    y = _decode(s["qa"], s["sa"]) @ _decode(s["qb"], s["sb"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if s["gate"] is not None:
        y = y * s["gate"].float().repeat_interleave(c["tokens"], 0)[: c["M"]]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["dtype"])


def _places(s, T):
    """Page and slot of row t of each sequence, and which rows there are."""
    t = torch.arange(T, device=DEV)
    pos = s["start"][:, None] + t
    page = torch.gather(s["table"], 1, (pos // s["case"]["page"]).long())
    return page.long(), (pos % s["case"]["page"]).long(), t < s["lens"][:, None]


def _plain_read(s):
    c = s["case"]
    page, slot, there = _places(s, c["T"])
    got = []
    for codes, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])):
        x = _decode(codes[page, :, slot], scales[page, :, slot])[..., : c["D"]]
        got.append(torch.where(there[..., None, None], x, 0.0).to(torch.bfloat16))
    return got


def _plain_cache(s):
    page, slot, there = _places(s, s["case"]["T"])
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]),
                             (s["v"], s["v_codes"], s["v_scales"])):
        q, sc = _quantize(x)
        codes[page[there], :, slot[there]] = q[there]
        scales[page[there], :, slot[there]] = sc[there]
    return _plain_read(s)


def _plain_attention(s):
    c = s["case"]
    B, M, H, Hkv, D, L = c["B"], c["M"], c["H"], c["Hkv"], c["D"], c["len"]
    at = s["table"].long()
    k, v = (_decode(s[n + "_codes"][at], s[n + "_scales"][at])[..., :D].transpose(1, 2)
            .flatten(2, 3)[:, :, :L] for n in "kv")                     # [B, Hkv, L, D]
    q = s["q"].float().unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    p = (q @ k.transpose(2, 3)) * D ** -0.5                               # [B, Hkv, G M, L]
    pos = torch.arange(L, device=DEV)
    see = (pos < s["lens"][:, None])[:, None, None, :]
    if c["causal"]:
        last = s["lens"][:, None] - M + torch.arange(M, device=DEV)       # [B, M]
        see = see & (pos <= last[:, None, :, None].repeat(1, 1, H // Hkv, 1))
    p = p.masked_fill(~see, -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))
    o = p @ v / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.unflatten(2, (H // Hkv, M)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)


# ----------------------------------------------------------- library calls
def _own(s):
    import w4a4_post_quantization_b200 as kq
    c = s["case"]
    if c["op"] == "linear":
        return kq.gemm_mxfp4_epilogue(s["qa"], s["sa_tiled"], s["qb"], s["sb_tiled"], bias=s["bias"],
                                      activation=c["act"], gate=s["gate"],
                                      tokens_per_sample=c["tokens"], residual=s["residual"],
                                      out_dtype=s["dtype"])
    cache = s.get("cache")
    if cache is None:
        cache = s["cache"] = kq.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                        c["D"])
    if c["op"] == "attention":
        return kq.attention_mxfp4(s["q"], cache, s["table"], s["lens"], causal=c["causal"])
    if c["op"] == "cache":
        kq.cache_write(cache, s["table"], s["k"], s["v"], start=s["start"], lens=s["lens"])
    return list(kq.cache_read(cache, s["table"], s["lens"], c["T"], start=s["start"]))


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "cache": _plain_cache, "read": _plain_read,
            "attention": _plain_attention}[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        e = 4 if c["out"] == "f32" else 2
        groups = -(-M // c["tokens"])
        return {"bytes": (M + N) * (K // 2 + K // 32) + M * N * e * (1 + c["residual"]) +
                2 * N * (c["bias"] + groups * c["gate"]), "flops": 2 * M * N * K}
    lens, D = _lens(c), c["D"]
    row = D // 2 + (D + 31) // 32                                        # a head's row in the cache
    if c["op"] == "cache":
        rows = 2 * sum(lens) * c["H"]
        return {"bytes": rows * (2 * D + 2 * row) + 2 * c["B"] * c["T"] * c["H"] * 2 * D,
                "flops": 4 * rows * D}
    if c["op"] == "read":
        rows = 2 * sum(lens) * c["H"]
        return {"bytes": rows * row + 2 * c["B"] * c["T"] * c["H"] * 2 * D, "flops": rows * D}
    M = c["M"]
    seen = sum(sum(max(0, n - M + i + 1) for i in range(M)) if c["causal"] else n * M for n in lens)
    return {"bytes": 2 * sum(lens) * c["Hkv"] * row + 4 * c["B"] * M * c["H"] * D,
            "flops": 4 * seen * c["H"] * D}


# ------------------------------------------------------- float64 reference
def _values64(codes, scales):
    """E2M1 by its fields: (-1)^s 2^(e-1) (1 + m/2), or m/2 where e = 0."""
    power = torch.tensor([math.ldexp(1.0, e - 127) for e in range(256)], dtype=torch.float64,
                         device=DEV)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    e, m = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(e > 0, power[126 + e.int()] * (1 + m / 2), m / 2)
    val = torch.where(c >= 8, -mag, mag).unflatten(-1, (-1, 32))
    return (val * power[scales.int()].unsqueeze(-1)).flatten(-2)


def _round_trip64(x):
    """The value nearest to x on its block's scaled E2M1 grid, by rounding
    to the step of its binade (ties to even)."""
    d = x.shape[-1]
    x = torch.nn.functional.pad(x.double(), (0, -d % 32)).unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    edges = torch.tensor([math.ldexp(1.0, e) for e in range(-126, 129)], dtype=torch.float64,
                         device=DEV)                     # binades of the block maximum
    scale = edges[torch.bucketize(amax, edges, right=True).clamp(3, 254) - 3]
    scale = torch.where(amax < edges[2], math.ldexp(1.0, -127), scale)
    a = x.abs() / scale
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = (torch.round(a / step) * step).clamp(max=6.0) * scale
    return torch.where(x < 0, -r, r).flatten(-2)[..., :d]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "linear":
        y = _values64(s["qa"], s["sa"]).matmul(_values64(s["qb"], s["sb"]).mT)
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "gelu_tanh":
            # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
            y = y / (1 + torch.exp(-2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
        elif c["act"] == "gelu":
            y = y * 0.5 * torch.erfc(-y / 2 ** 0.5)
        elif c["act"] == "silu":
            y = y * torch.sigmoid(y)
        if c["gate"]:
            y *= s["gate"].double()[torch.arange(c["M"], device=DEV) // c["tokens"]]
        return y + s["residual"].double() if c["residual"] else y
    lens = _lens(c)
    if c["op"] == "cache":
        got = []
        for x in (s["k"], s["v"]):
            y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
            for b, n in enumerate(lens):
                y[b, :n] = _round_trip64(x[b, :n])
            got.append(y)
        return got
    D, page = c["D"], c["page"]
    if c["op"] == "read":
        got = []
        for n in "kv":
            y = torch.zeros((c["B"], c["T"], c["H"], D), dtype=torch.float64, device=DEV)
            for b, rows in enumerate(lens):
                pages = s["table"][b].long()
                x = _values64(s[n + "_codes"][pages], s[n + "_scales"][pages])[..., :D]
                y[b, :rows] = x.transpose(1, 2).reshape(-1, c["H"], D)[c["start"]: c["start"] + rows]
            got.append(y)
        return got
    B, M, H, Hkv, L = c["B"], c["M"], c["H"], c["Hkv"], c["len"]
    out = torch.zeros((B, M, H, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        pages = s["table"][b].long()
        for h in range(Hkv):
            if n == 0:
                continue
            k, v = (_values64(s[x + "_codes"][pages, h], s[x + "_scales"][pages, h])
                    .reshape(-1, s[x + "_codes"].shape[-1] * 2)[:n, :D] for x in "kv")
            for g in range(H // Hkv):
                head = h * (H // Hkv) + g
                logit = s["q"][b, :, head].double().matmul(k.mT) / D ** 0.5
                if c["causal"]:
                    row = torch.arange(M, device=DEV)[:, None]
                    logit[torch.arange(n, device=DEV)[None] > n - M + row] = -math.inf
                w = torch.nan_to_num(torch.softmax(logit, -1), nan=0.0)
                out[b, :, head] = w.matmul(v)
    return out
