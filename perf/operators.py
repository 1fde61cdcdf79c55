"""The fp8 operators' measured cases: inputs, one pass each, and its value in 64 bits.

Three operators, used one after the other by a layer whose experts are held in
8-bit floating point (e4m3) with one fp32 scale per block of 128:

  quantize  values -> e4m3 codes and scales; a scale per 1 x 128 (activations)
            or per 128 x 128 block (weights), the smallest power of two that
            brings the block into e4m3's range, so that dividing by it is exact;
  matmul    out = A B^T, A with 1 x 128 scales, B with 128 x 128 scales;
  experts   the expert half of the layer for given routing: quantised x,
            SwiGLU experts, quantised h, down, weighted sum, shared expert.

`run` computes them with elementary torch operations, or, where `own` is true,
with the calls of sparse_moe_routing_gb300.
"""
import math

import torch

own = False

BLK = 128
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
LEAST = -126  # exponent of the smallest scale, the smallest normal fp32

# (d_model, experts, top-k, expert width, shared width) of the layers this
# repository configures: the 256-, 128-, 160-, 64- and 60-expert shapes, the
# 8-expert wide one and the tiny one
SHAPES = {
    "e256": (2048, 256, 8, 512, 512),
    "e128": (2048, 128, 8, 512, 512),
    "e160": (2048, 160, 6, 512, 512),
    "e64": (2048, 64, 6, 1408, 1408),
    "e60": (2048, 60, 4, 1408, 5632),
    "e8": (4096, 8, 2, 14336, 0),
    "tiny": (256, 16, 4, 64, 64),
}


def listed():
    return [
        # activations of a decode batch, the smallest call
        {"name": "quantize_decode", "op": "quantize", "rows": 8, "cols": 2048, "dtype": "bf16", "block_rows": 1},
        # activations of a prefill batch in fp32, an odd number of rows
        {"name": "quantize_prefill", "op": "quantize", "rows": 4097, "cols": 4096, "dtype": "f32", "block_rows": 1},
        # one expert's gate matrix of the 8-expert shape, quantised when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "rows": 14336, "cols": 4096, "dtype": "bf16", "block_rows": 128},
        # one token through a wide shared expert's projection
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 5632, "K": 2048, "out": "bf16"},
        # a decode batch through a down projection
        {"name": "matmul_decode", "op": "matmul", "M": 64, "N": 4096, "K": 14336, "out": "bf16"},
        # ragged in every direction, fp32 result (a residual-stream projection)
        {"name": "matmul_ragged", "op": "matmul", "M": 333, "N": 1001, "K": 1400, "out": "f32"},
        # a long prefill through an up projection, the largest product
        {"name": "matmul_prefill", "op": "matmul", "M": 8192, "N": 14336, "K": 4096, "out": "bf16"},
        # one token through the 256-expert layer: latency
        {"name": "experts_token", "op": "experts", "shape": "e256", "T": 1, "skew": 0.0, "residual": False},
        # small and usual decode batches: the expert weights' bytes
        {"name": "experts_decode8", "op": "experts", "shape": "e256", "T": 8, "skew": 0.0, "residual": True},
        {"name": "experts_decode64", "op": "experts", "shape": "e256", "T": 64, "skew": 0.0, "residual": False},
        # prefill with an uneven load of the experts
        {"name": "experts_prefill", "op": "experts", "shape": "e256", "T": 4096, "skew": 1.5, "residual": False},
        # few wide experts: bound by the products
        {"name": "experts_wide", "op": "experts", "shape": "e8", "T": 2048, "skew": 0.0, "residual": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range: odd, or a multiple of 16 or 128."""
    n = _log_int(rng, lo, hi)
    step = rng.choice((1, 16, 128))
    n = max(lo, n // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(("quantize", "matmul", "matmul", "experts", "experts"))
    if op == "quantize":
        rows, cols = _size(rng, 1, 16384), _size(rng, 64, 14336)
        rows = min(rows, 14336 * 4096 // cols)
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "f32")),
                "block_rows": rng.choice((1, 128))}
    if op == "matmul":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 14336), "K": _size(rng, 64, 4096),
                "out": rng.choice(("bf16", "f32"))}
    shape = rng.choice(sorted(SHAPES))
    return {"op": op, "shape": shape, "T": _log_int(rng, 1, 2048 if shape in ("e8", "e60") else 4096),
            "skew": rng.choice((0.0, 1.5)), "residual": rng.choice((False, True))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(n):
    return -(-n // BLK)


def _amax(x, block_rows):
    """Largest magnitude of each block of x [..., rows, cols]."""
    rows, cols = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -cols % BLK, 0, -rows % block_rows))
    return x.unflatten(-1, (-1, BLK)).unflatten(-3, (-1, block_rows)).abs().amax(dim=(-1, -3))


def _scales_of(x, block_rows):
    """fp32 scales of x (fp32): the smallest power of two, 2^-126 at least, that is amax / 448 or more; NaN where
    the block holds a value that is not finite."""
    amax = _amax(x, block_rows)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    n = torch.where(m > 0.875, e - 8, e - 9).clamp(min=LEAST)
    s = ((n + 127) << 23).to(torch.int32).view(torch.float32)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, math.nan))


def _spread(s, rows, cols, block_rows):
    """Scales [..., row blocks, column blocks] at every value's place [..., rows, cols]."""
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return s.repeat_interleave(BLK, dim=-1)[..., :cols]


def _quantize(x, block_rows):
    """(e4m3 codes, fp32 scales) of x in fp32; the division by a power of two is exact."""
    s = _scales_of(x, block_rows)
    return (x / _spread(s, x.shape[-2], x.shape[-1], block_rows)).to(F8), s


def _pitched(codes):
    """Codes with rows 16 bytes apart or a multiple, as the framework's products take them."""
    cols = codes.shape[-1]
    if cols % 16 == 0:
        return codes.contiguous()
    room = torch.zeros(codes.shape[:-1] + (-(-cols // 16) * 16,), dtype=torch.uint8, device=codes.device)
    room[..., :cols] = codes.view(torch.uint8)
    return room.view(F8)[..., :cols]


def _weights(g, *shape):
    """Codes and scales of weights N(0, 0.02), with scales amax / 448 of no special form, as a checkpoint brings
    them; quantised matrix by matrix where there are many."""
    parts = []
    flat = shape if len(shape) == 3 else (1,) + shape
    for i in range(flat[0]):
        w = torch.randn(flat[1:], generator=g, device="cuda") * 0.02
        s = _amax(w, BLK) / F8_MAX
        parts.append(((w / _spread(s, *flat[1:], BLK)).clamp(-F8_MAX, F8_MAX).to(F8), s))
    codes = torch.stack([p[0].view(torch.uint8) for p in parts]).view(F8)
    scales = torch.stack([p[1] for p in parts])
    return (codes, scales) if len(shape) == 3 else (_pitched(codes[0]), scales[0])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "quantize":
        # rows of very different size, as activations have
        x = torch.randn(case["rows"], case["cols"], generator=g, device="cuda")
        x = x * torch.exp(1.5 * torch.randn(case["rows"], 1, generator=g, device="cuda"))
        x = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s |= {"x": x, "block_rows": case["block_rows"]}
        if own:
            import sparse_moe_routing_gb300 as smr
            s["codes"], s["scales"] = smr.fp8_empty(case["rows"], case["cols"], case["block_rows"])
            s["smr"] = smr
        return s
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        a, a_scale = _quantize(torch.randn(M, K, generator=g, device="cuda"), 1)
        b, b_scale = _weights(g, N, K)
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s |= {"a": _pitched(a), "a_scale": a_scale, "b": b, "b_scale": b_scale, "dtype": dt}
        if own:
            import sparse_moe_routing_gb300 as smr
            s["out"] = torch.empty(M, N, dtype=dt, device="cuda")
            s["ws"] = smr.fp8_matmul_workspace(M, N, K)
            s["smr"] = smr
        return s
    d, E, k, width, shared = SHAPES[case["shape"]]
    T = case["T"]
    x = torch.randn(T, d, generator=g, device="cuda")
    x = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    # routing of the layer's softmax rule for random logits, uneven where skewed
    z = torch.randn(T, E, generator=g, device="cuda") + case["skew"] * torch.randn(E, generator=g, device="cuda")
    p, ids = torch.softmax(z, -1).topk(k, dim=-1)
    s |= {"x": x, "ids": ids.to(torch.int32), "alpha": (p / p.sum(-1, keepdim=True)).contiguous(),
          "w": {"W_gate": _weights(g, E, width, d), "W_up": _weights(g, E, width, d),
                "W_down": _weights(g, E, d, width)},
          "gate": None, "residual": None, "rows": int(torch.bincount(ids.reshape(-1), minlength=E).max())}
    if shared:
        s["w"] |= {"Ws_gate": _weights(g, shared, d), "Ws_up": _weights(g, shared, d),
                   "Ws_down": _weights(g, d, shared)}
        s["gate"] = torch.sigmoid(torch.randn(T, generator=g, device="cuda"))
    if case["residual"]:
        s["residual"] = torch.randn(T, d, generator=g, device="cuda")
    if own:
        import sparse_moe_routing_gb300 as smr
        cfg = smr.MoEConfig(T=T, d_model=d, n_experts=E, top_k=k, d_ff=width, d_ff_shared=shared,
                            expert_dtype=smr.F8_E4M3_B128)
        s["experts"] = smr.Fp8Experts(cfg, s["w"])
        s["out"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _dequantize(codes, scales, block_rows):
    return codes.float() * _spread(scales, codes.shape[-2], codes.shape[-1], block_rows)


def _requantized(x):
    """x rounded to e4m3 with 1 x 128 scales, as values."""
    return _dequantize(*_quantize(x, 1), 1)


def _mlp(x, gate, up, down):
    """SwiGLU expert of quantised rows x [..., n, d]; weights as (codes, scales)."""
    g = x @ _dequantize(*gate, BLK).transpose(-1, -2)
    u = x @ _dequantize(*up, BLK).transpose(-1, -2)
    h = _requantized(g / (1 + torch.exp(-g)) * u)
    return h @ _dequantize(*down, BLK).transpose(-1, -2)


def _experts(s):
    x = _requantized(s["x"].float())
    ids, alpha, w = s["ids"].long(), s["alpha"], s["w"]
    T, k = ids.shape
    bank = [w["W_gate"], w["W_up"], w["W_down"]]
    E, rows = bank[0][0].shape[0], s["rows"]
    if T * k < E:  # the chosen experts' matrices, pair by pair
        at = ids.reshape(-1)
        picked = [(c.view(torch.uint8)[at].view(F8), sc[at]) for c, sc in bank]
        y = _mlp(x.repeat_interleave(k, 0).unsqueeze(1), *picked).squeeze(1)
    else:  # every expert's pairs, padded to the largest group
        order = torch.argsort(ids.reshape(-1), stable=True)
        expert = ids.reshape(-1)[order]
        first = torch.searchsorted(expert, torch.arange(E, device=expert.device))
        slot = torch.arange(T * k, device=expert.device) - first[expert]
        padded = torch.zeros(E, rows, x.shape[1], device=x.device)
        padded[expert, slot] = x[order // k]
        y = torch.empty(T * k, x.shape[1], device=x.device)
        y[order] = _mlp(padded, *bank)[expert, slot]
    y = (y.view(T, k, -1) * alpha.unsqueeze(-1)).sum(1)
    if s["gate"] is not None:
        y = y + s["gate"].unsqueeze(-1) * _mlp(x, w["Ws_gate"], w["Ws_up"], w["Ws_down"])
    if s["residual"] is not None:
        y = s["residual"] + y
    return y.to(torch.bfloat16)


def run(state):
    s = state
    if s["op"] == "quantize":
        if own:
            s["smr"].fp8_quantize(s["x"], s["codes"], s["scales"], block_rows=s["block_rows"])
            return {"codes": s["codes"], "scales": s["scales"]}
        codes, scales = _quantize(s["x"].float(), s["block_rows"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "matmul":
        if own:
            s["smr"].fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], s["ws"])
            return s["out"]
        return (_dequantize(s["a"], s["a_scale"], 1) @ _dequantize(s["b"], s["b_scale"], BLK).T).to(s["dtype"])
    if own:
        s["experts"].forward(s["x"], s["ids"], s["alpha"], s_shared=s["gate"], r_attn=s["residual"], out=s["out"])
        return s["out"]
    return _experts(s)


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * _blocks(case["cols"])
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * blocks, "flops": 3 * n}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": M * K + N * K + 4 * M * _blocks(K) + 4 * _blocks(N) * _blocks(K) + out * M * N,
                "flops": 2 * M * N * K}
    d, E, k, width, shared = SHAPES[case["shape"]]
    T = case["T"]
    active = E * (1 - (1 - k / E) ** T)  # experts with a token, on average over even loads
    one = 3 * width * d + 12 * _blocks(width) * _blocks(d)
    sh = 3 * shared * d + 12 * _blocks(shared) * _blocks(d) if shared else 0
    io = T * d * (2 + 2 + (4 if case["residual"] else 0)) + T * k * 8 + (4 * T if shared else 0)
    return {"bytes": active * one + sh + io, "flops": 2 * T * 3 * d * (k * width + shared)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3(v):
    """fp64 values rounded to the nearest e4m3 number, ties to even."""
    mag = v.abs().clamp(min=2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(mag)).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _codes64(x, tall):
    """(code values, scales) of a matrix in fp64, block by block of `tall` rows x 128."""
    R, C = x.shape
    nr, nc = -(-R // tall), _blocks(C)
    full = x.new_zeros(nr * tall, nc * BLK)
    full[:R, :C] = x
    cut = full.view(nr, tall, nc, BLK)
    amax = cut.abs().amax((1, 3))
    near = torch.exp2(torch.ceil(torch.log2(amax / F8_MAX)).clamp(min=LEAST + 1, max=127))
    # the logarithm may be off by its last bit at a power of two
    scale = torch.where(near / 2 * F8_MAX >= amax, near / 2, torch.where(near * F8_MAX >= amax, near, near * 2))
    codes = _e4m3(cut / scale[:, None, :, None])
    return codes.reshape(nr * tall, nc * BLK)[:R, :C], scale


def _values64(codes, scale, tall):
    """What codes [R, C] with scales stand for, in fp64."""
    R, C = codes.shape
    i = torch.arange(R, device=codes.device) // tall
    j = torch.arange(C, device=codes.device) // BLK
    return codes.to(torch.float64) * scale.to(torch.float64)[i][:, j]


def _rounded64(x):
    codes, scale = _codes64(x, 1)
    return _values64(codes, scale, 1)


def _expert64(x, gate, up, down):
    g = x @ _values64(*gate, BLK).T
    h = _rounded64(g * torch.sigmoid(g) * (x @ _values64(*up, BLK).T))
    return h @ _values64(*down, BLK).T


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        codes, scales = _codes64(s["x"].double(), s["block_rows"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "matmul":
        return _values64(s["a"], s["a_scale"], 1) @ _values64(s["b"], s["b_scale"], BLK).T
    w, ids = s["w"], s["ids"].long()
    x = _rounded64(s["x"].double())
    out = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    for e in range(w["W_gate"][0].shape[0]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            y = _expert64(x[token], *((w[n][0][e], w[n][1][e]) for n in ("W_gate", "W_up", "W_down")))
            out.index_add_(0, token, s["alpha"][token, slot].double()[:, None] * y)
    if s["gate"] is not None:
        out += s["gate"].double()[:, None] * _expert64(x, w["Ws_gate"], w["Ws_up"], w["Ws_down"])
    return out
