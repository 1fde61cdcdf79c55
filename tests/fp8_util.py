"""Plain 64-bit forms of the 8-bit operators, for the tests: e4m3 codes with
one scale per block of 128, the product, and the expert half of the layer."""
import math

import torch

F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def round_e4m3(v):
    """Nearest e4m3 number (ties to even, magnitudes above 448 to 448), fp64."""
    v = v.double()
    _, e = torch.frexp(v)                       # |v| = m 2^e, m in [0.5, 1)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def block_scale(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448 (a Python float)."""
    if not math.isfinite(amax):
        return math.nan
    s = 2.0 ** -126
    while amax / s > 448.0:
        s *= 2.0
    return s


def quantize_ref(x, block_rows):
    """(code values fp64, scales fp32) of a matrix on the CPU, block by block."""
    x = x.double().cpu()
    R, C = x.shape
    codes = torch.empty_like(x)
    scales = torch.empty(-(-R // block_rows), blocks(C), dtype=torch.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            b = x[at]
            s = block_scale(float(b.abs().max()) if bool(torch.isfinite(b).all()) else math.nan)
            scales[i, j] = s
            codes[at] = round_e4m3(b / s) if math.isfinite(s) else math.nan
    return codes, scales


def quantize64(x):
    """x [n, K] (fp64) rounded to e4m3 with 1 x 128 power-of-two scales, as values."""
    n, K = x.shape
    p = torch.zeros(n, blocks(K) * 128, dtype=torch.float64, device=x.device)
    p[:, :K] = x
    p = p.view(n, -1, 128)
    amax = p.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    s = torch.exp2(torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126).double())
    s = torch.where(torch.isfinite(amax), s, torch.full_like(s, math.nan))
    return (round_e4m3(p / s) * s).view(n, -1)[:, :K]


def values(codes, scales, block_rows):
    """fp64 values of codes [R, C] with their scales."""
    R, C = codes.shape
    s = scales.double().repeat_interleave(block_rows, 0)[:R].repeat_interleave(128, 1)[:, :C]
    return codes.to(torch.float64) * s


def pitched(codes):
    """The same codes with rows a multiple of 16 bytes apart; the bytes between hold NaN codes."""
    R, C = codes.shape
    room = torch.full((R, -(-C // 16) * 16), 0x7F, dtype=torch.uint8, device=codes.device)
    room[:, :C] = codes.view(torch.uint8)
    return room.view(F8)[:, :C]


def random_matrix(g, R, C, block_rows, spread=1.0, pow2=False):
    """Random codes and scales of no special form; the pitch's padding holds NaN codes."""
    v = torch.randn(R, C, generator=g, device="cuda") * 60.0
    codes = v.clamp(-448, 448).to(F8)
    s = torch.exp(spread * torch.randn(-(-R // block_rows), blocks(C), generator=g, device="cuda")) * 0.01
    return pitched(codes), s


def bank(g, E, N, K):
    """(codes [E, N, K], scales) of weights N(0, 0.02) with scales amax / 448."""
    w = torch.randn(E, N, K, generator=g, device="cuda") * 0.02
    p = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    s = p.view(E, -1, 128, blocks(K), 128).abs().amax((2, 4)) / 448.0
    at = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return (w / at).clamp(-448, 448).to(F8).contiguous(), s.contiguous()


def mlp64(x, gate, up, down):
    g = x @ values(*gate, 128).T
    h = g * torch.sigmoid(g) * (x @ values(*up, 128).T)
    return quantize64(h) @ values(*down, 128).T


def experts_ref(x, ids, alpha, w, gate=None, residual=None):
    """out of the expert half in fp64. w: dict of (codes, scales) banks."""
    xq = quantize64(x.double())
    y = torch.zeros_like(xq)
    for e in range(w["W_gate"][0].shape[0]):
        t, s = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            one = [(w[n][0][e], w[n][1][e]) for n in ("W_gate", "W_up", "W_down")]
            y.index_add_(0, t, alpha[t, s].double()[:, None] * mlp64(xq[t], *one))
    if "Ws_gate" in w:
        sh = [(w[n][0][0], w[n][1][0]) for n in ("Ws_gate", "Ws_up", "Ws_down")]
        y += gate.double()[:, None] * mlp64(xq, *sh)
    return y if residual is None else residual.double() + y
