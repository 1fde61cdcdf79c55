"""A layer held in 8-bit floating point, from a bf16 layer's weights.

Quantises the expert banks of a bf16 layer (e4m3 codes, one scale per 128 x 128
block), routes and runs a batch of tokens through it, adds the residual, and
multiplies the result by an 8-bit projection, as the next block of a model
would. Prints how far the result is from the bf16 layer's and what a step
takes.

    python examples/fp8_layer.py [--tokens 8] [--shape qwen36_decode]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import moe_inputs as mi  # noqa: E402
import sparse_moe_routing_gb300 as smr  # noqa: E402


def bf16_weights(shape, g):
    """Random bf16 weights of a layer's shape on the GPU, as smr.MoELayer takes them."""
    def w(*size):
        return (torch.randn(*size, generator=g, device="cuda") * 0.02).to(torch.bfloat16)

    d, E, width, shared = shape.d_model, shape.n_experts, shape.d_ff, shape.d_ff_shared
    out = {"W_router": w(E, d), "W_gate": w(E, width, d), "W_up": w(E, width, d), "W_down": w(E, d, width)}
    if shared:
        out.update(Ws_gate=w(shared, d), Ws_up=w(shared, d), Ws_down=w(d, shared), w_shared=w(d))
    return out


def run(shape, tokens, steps=20):
    """(relative error against the bf16 layer, of the projection against fp32, us per step)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    weights = bf16_weights(shape, g)
    base = dict(T=tokens, d_model=shape.d_model, n_experts=shape.n_experts, top_k=shape.top_k,
                d_ff=shape.d_ff, d_ff_shared=shape.d_ff_shared)
    layer16 = smr.MoELayer(smr.MoEConfig(**base), weights)
    layer8 = smr.Fp8Experts.from_bf16(smr.MoEConfig(expert_dtype=smr.F8_E4M3_B128, **base), weights)
    proj = (torch.randn(shape.d_ff, shape.d_model, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    linear = smr.Fp8Linear(proj, tokens)

    x = torch.randn(tokens, shape.d_model, generator=g, device="cuda")
    x = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
    zero = torch.zeros(tokens, shape.d_model, device="cuda")
    ids = torch.empty(tokens, shape.top_k, dtype=torch.int32, device="cuda")
    alpha = torch.empty(tokens, shape.top_k, device="cuda")
    out = torch.empty_like(zero)
    y = torch.empty(tokens, shape.d_ff, dtype=torch.bfloat16, device="cuda")

    def step():
        layer8.layer(x, ids, alpha, r_attn=zero, out=out)
        return linear(out, y)

    step()
    want, _, _ = layer16.forward(x, zero)
    off = float((out - want).norm() / want.norm())
    ref = out @ proj.float().T
    off_y = float((y.float() - ref).norm() / ref.norm())
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        step()
    stop.record()
    torch.cuda.synchronize()
    status, word = layer8.device_status()
    if status != 0:
        raise RuntimeError("device status %d (word 0x%x)" % (status, word))
    return off, off_y, start.elapsed_time(stop) / steps * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--shape", default="qwen36_decode",
                    choices=sorted(n for n, s in mi.PRESETS.items() if s.expert_dtype == "bf16"))
    a = ap.parse_args()
    off, off_y, us = run(mi.PRESETS[a.shape], a.tokens)
    print("%s, %d tokens: layer %.1f %% from the bf16 layer, projection %.1f %% from fp32, %.1f us per step"
          % (a.shape, a.tokens, 100 * off, 100 * off_y, us))


if __name__ == "__main__":
    main()
