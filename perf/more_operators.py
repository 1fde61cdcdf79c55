"""Measured cases of the norm in front of a layer and of the 8-bit integer products: inputs, one pass each, and its
value in 64 bits.

Four operators, used one after the other by a decoder layer whose dense projections are held in 8-bit integers:

  norm      s = x + residual; out = s * gain / sqrt(mean(s^2) + eps); also the updated residual s and out in 8 bits:
            integers with a scale per row, or e4m3 with a scale per 1 x 128 block;
  quantize  values -> integers in [-127, 127] and a scale per row (a token's activations, or an output channel's weights);
  matmul    out = (A B^T) * a_scale * b_scale, integer codes, a scale per row of A and per row of B;
  gated     out = SiLU(x gate^T) * (x up^T), both products as above.

The 8-bit codes of a row t (for norm t = s * gain, whose factor 1 / sqrt(..) goes into the scale) are
round(t * f) with f = 127 / m, m = max(max |t|, 127 * 2^-126), and stand for code * (m / 127); every step is rounded to
32 bits. e4m3 codes are e4m3(t / p), p the smallest power of two, 2^-126 at least, with max |t| / p <= 448.

`run` computes them with elementary torch operations, or, where `own` is true, with the calls of
sparse_moe_routing_gb300.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token in front of an expert layer: values for the router, integers for the dense projections; latency
        {"name": "norm_token", "op": "norm", "T": 1, "d": 2048, "x": "bf16", "residual": "f32", "gain": True,
         "out": "bf16", "codes": "int8"},
        # a decode batch in front of the layer in 8-bit floating point
        {"name": "norm_decode", "op": "norm", "T": 64, "d": 4096, "x": "bf16", "residual": "bf16", "gain": True,
         "out": "bf16", "codes": "e4m3"},
        # a ragged batch, values only
        {"name": "norm_ragged", "op": "norm", "T": 333, "d": 1001, "x": "f32", "residual": "f32", "gain": False,
         "out": "f32", "codes": ""},
        # a long prefill, integers only
        {"name": "norm_prefill", "op": "norm", "T": 8192, "d": 4096, "x": "bf16", "residual": "f32", "gain": True,
         "out": "", "codes": "int8"},
        # the hidden values of a decode batch in front of a down projection
        {"name": "quantize_decode", "op": "quantize", "rows": 64, "cols": 14336, "x": "bf16"},
        # a projection's weights, quantised when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "rows": 14336, "cols": 4096, "x": "bf16"},
        # one token through a wide projection
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 5632, "K": 2048, "out": "bf16"},
        # a decode batch through a down projection: the weights' bytes
        {"name": "matmul_decode", "op": "matmul", "M": 64, "N": 4096, "K": 14336, "out": "bf16"},
        # ragged in every direction, fp32 result
        {"name": "matmul_ragged", "op": "matmul", "M": 333, "N": 1001, "K": 1400, "out": "f32"},
        # a long prefill through an up projection, the largest product
        {"name": "matmul_prefill", "op": "matmul", "M": 8192, "N": 14336, "K": 4096, "out": "bf16"},
        # a small decode batch through a dense layer's gate and up projections
        {"name": "gated_decode", "op": "gated", "M": 8, "N": 14336, "K": 4096, "out": "bf16"},
        # a prefill through the same
        {"name": "gated_prefill", "op": "gated", "M": 2048, "N": 14336, "K": 4096, "out": "bf16"},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of the range: odd, or a multiple of 16 or 128."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 16, 128))
    return max(lo, n // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm", "quantize", "matmul", "matmul", "gated"))
    kind = lambda: rng.choice(("bf16", "f32"))  # noqa: E731
    if op == "norm":
        d = _size(rng, 64, 14336)
        out, codes = rng.choice((("bf16", "int8"), ("", "int8"), ("bf16", "e4m3"), ("", "e4m3"), ("bf16", ""),
                                 ("f32", "")))
        return {"op": op, "T": min(_size(rng, 1, 8192), 8192 * 4096 // d), "d": d, "x": kind(),
                "residual": rng.choice(("", "bf16", "f32")), "gain": rng.choice((False, True)), "out": out,
                "codes": codes}
    if op == "quantize":
        cols = _size(rng, 64, 14336)
        return {"op": op, "rows": min(_size(rng, 1, 14336), 14336 * 4096 // cols), "cols": cols, "x": kind()}
    n = 1 if op == "matmul" else 2
    N, K = _size(rng, 64, 14336), _size(rng, 64, 14336)
    return {"op": op, "M": min(_size(rng, 1, 8192), 8192 * 14336 * 4096 // (n * N * K)), "N": N, "K": K, "out": kind()}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _int8(t):
    """(int8 codes, fp32 scales) of the rows of t in fp32; full() tensors, since a division by or of a plain number
    would go through a reciprocal."""
    m = t.abs().amax(-1).clamp(min=127.0 * 2.0 ** -126)
    c = torch.full_like(m, 127.0)
    return torch.round(t * (c / m)[:, None]).to(torch.int8), m / c


def _e4m3(t):
    """(e4m3 codes, fp32 power-of-two scales) of the 1 x 128 blocks of t in fp32; dividing by the scale is exact."""
    T, d = t.shape
    nb = -(-d // 128)
    amax = torch.nn.functional.pad(t, (0, -d % 128)).view(T, nb, 128).abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    n = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    p = ((n + 127) << 23).to(torch.int32).view(torch.float32)
    return (t / p.repeat_interleave(128, -1)[:, :d]).to(F8), p


def _pitched(codes):
    """Codes with rows 16 bytes apart or a multiple, as the framework's products take them."""
    rows, cols = codes.shape
    if cols % 16 == 0:
        return codes
    room = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.int8, device=codes.device)
    room[:, :cols] = codes
    return room[:, :cols]


def _rows(g, rows, cols):
    """Rows of very different size with a few large columns, as activations have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x[:, :: 97] *= 8.0
    return x * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))


def _weights(g, N, K):
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    q, s = _int8(w)
    return _pitched(q), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if own:
        import sparse_moe_routing_gb300 as smr
        s["smr"] = smr
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        s["x"] = _rows(g, T, d).to(DT[case["x"]])
        s["residual"] = 3 * torch.randn(T, d, generator=g, device="cuda").to(DT[case["residual"]]) if case["residual"] else None
        s["gain"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["gain"] else None
        if own:
            s["sum"] = torch.empty_like(s["residual"]) if case["residual"] else None
            s["values"] = torch.empty(T, d, dtype=DT[case["out"]], device="cuda") if case["out"] else None
            s["q"] = smr.int8_empty(T, d) if case["codes"] == "int8" else smr.fp8_empty(T, d) if case["codes"] else (None, None)
    elif case["op"] == "quantize":
        s["x"] = _rows(g, case["rows"], case["cols"]).to(DT[case["x"]])
        if own:
            s["q"] = smr.int8_empty(case["rows"], case["cols"])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        a, s["a_scale"] = _int8(_rows(g, M, K))
        s["a"] = _pitched(a)
        s["b"] = _weights(g, N, K)
        s["up"] = _weights(g, N, K) if case["op"] == "gated" else None
        if own:
            s["y"] = torch.empty(M, N, dtype=DT[case["out"]], device="cuda")
            s["ws"] = smr.int8_matmul_workspace(M, N, K, gated=case["op"] == "gated")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _norm(s):
    t = s["x"].float()
    found = {}
    if s["residual"] is not None:
        t = t + s["residual"].float()
        found["sum"] = t.to(s["residual"].dtype)
    inv = 1 / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS)
    if s["gain"] is not None:
        t = t * s["gain"].float()
    if s["out"]:
        found["values"] = (t * inv).to(DT[s["out"]])
    if s["codes"]:
        codes, scales = _int8(t) if s["codes"] == "int8" else _e4m3(t)
        found |= {"codes": codes, "scales": scales * (inv[:, 0] if s["codes"] == "int8" else inv)}
    return found


def _product(s, b):
    return (s["a"].float() @ b[0].float().T) * s["a_scale"][:, None] * b[1]


def run(state):
    s = state
    if own:
        smr = s["smr"]
        if s["op"] == "norm":
            codes, scales = s["q"]
            smr.add_rmsnorm(s["x"], residual=s["residual"], gain=s["gain"], eps=EPS, out=s["values"], sum_out=s["sum"],
                            codes=codes, scales=scales)
            found = {"sum": s["sum"], "values": s["values"], "codes": codes, "scales": scales}
            return {k: v for k, v in found.items() if v is not None}
        if s["op"] == "quantize":
            smr.int8_quantize(s["x"], *s["q"])
            return {"codes": s["q"][0], "scales": s["q"][1]}
        if s["op"] == "matmul":
            smr.int8_matmul(s["a"], s["a_scale"], *s["b"], s["y"], s["ws"])
        else:
            smr.int8_gated_matmul(s["a"], s["a_scale"], *s["b"], *s["up"], s["y"], s["ws"])
        return s["y"]
    if s["op"] == "norm":
        return _norm(s)
    if s["op"] == "quantize":
        codes, scales = _int8(s["x"].float())
        return {"codes": codes, "scales": scales}
    y = _product(s, s["b"])
    if s["op"] == "gated":
        y = y / (1 + torch.exp(-y)) * _product(s, s["up"])
    return y.to(DT[s["out"]])


def work(case):
    size = {"bf16": 2, "f32": 4, "": 0}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        per = size[case["x"]] + 2 * size[case["residual"]] + size[case["out"]] + (1 if case["codes"] else 0)
        scales = {"int8": 1, "e4m3": -(-d // 128), "": 0}[case["codes"]]
        return {"bytes": T * d * per + 4 * T * scales + (2 * d if case["gain"] else 0), "flops": 8 * T * d}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + 1) + 4 * case["rows"], "flops": 3 * n}
    M, N, K = case["M"], case["N"], case["K"]
    n = 1 if case["op"] == "matmul" else 2
    return {"bytes": M * K + n * N * K + 4 * (M + n * N) + size[case["out"]] * M * N, "flops": 2 * n * M * N * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _r32(v):
    """fp64 values rounded to 32 bits, as the definition of the codes does at each step."""
    return v.to(torch.float32).to(torch.float64)


def _int8_64(t):
    """(codes, scales in fp64) of rows t that are fp32 numbers: the codes by the definition's steps, a row's largest
    value by the scale unrounded."""
    m = t.abs().max(dim=-1, keepdim=True).values.clamp(min=127 * 2.0 ** -126)
    return torch.round(_r32(t * _r32(127.0 / m))).to(torch.int8), (m / 127).squeeze(-1)


def _e4m3_64(t):
    """(code values, scales) of 1 x 128 blocks in fp64."""
    T, d = t.shape
    codes = torch.empty_like(t)
    scales = t.new_empty(T, -(-d // 128))
    for j in range(scales.shape[1]):
        block = t[:, 128 * j:128 * (j + 1)]
        amax = block.abs().max(dim=-1).values
        p = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448)))
        p = torch.where(p / 2 * 448 >= amax, p / 2, torch.where(p * 448 >= amax, p, p * 2)).clamp(min=2.0 ** -126)
        v = block / p[:, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
        codes[:, 128 * j:128 * (j + 1)] = torch.round(v / step) * step
        scales[:, j] = p
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        codes, scales = _int8_64(s["x"].double())
        return {"codes": codes, "scales": scales}
    if s["op"] == "norm":
        x, found = s["x"].double(), {}
        if s["residual"] is not None:
            x = x + s["residual"].double()
            found["sum"] = x
        gain = s["gain"].double() if s["gain"] is not None else 1.0
        root = torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
        if s["out"]:
            found["values"] = x / root * gain
        if s["codes"]:
            t = _r32(_r32(x) * gain)
            codes, scales = _int8_64(t) if s["codes"] == "int8" else _e4m3_64(t)
            found |= {"codes": codes, "scales": scales / (root[:, 0] if s["codes"] == "int8" else root)}
        return found
    y = torch.mm(s["a"].double(), s["b"][0].double().T) * torch.outer(s["a_scale"].double(), s["b"][1].double())
    if s["op"] == "gated":
        u = torch.mm(s["a"].double(), s["up"][0].double().T) * torch.outer(s["a_scale"].double(), s["up"][1].double())
        y = y * torch.sigmoid(y) * u
    return y
