"""What the 8-bit layer's binding refuses on the host, by the name of the
tensor at fault. Nothing here launches a kernel."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


@pytest.mark.parametrize("scales,good", [
    ((4, 2, 3), True), ((2, 3), False), ((1, 2, 3), False), ((4, 2, 2), False), ((8, 3), False), ((4, 6), False)])
def test_bank_scales_have_one_matrix_per_expert(scales, good):
    """Scales without the experts' dimension are too short for more than one expert."""
    b = (codes(4, 200, 300), torch.zeros(scales))
    with pytest.raises(ValueError, match="CUDA" if good else "scales"):  # (a good bank: only not on a GPU)
        smr._bank8(b, (4, 200, 300))


@pytest.mark.parametrize("shape,scales,good", [
    ((200, 300), (2, 3), True), ((1, 200, 300), (1, 2, 3), True), ((200, 300), (1, 2, 3), True),
    ((1, 200, 300), (2, 3), True), ((200, 300), (2, 2), False), ((200, 300), (3, 2), False)])
def test_bank_of_one_matrix_may_leave_its_dimension_out(shape, scales, good):
    with pytest.raises(ValueError, match="CUDA" if good else "scales"):
        smr._bank8((codes(*shape), torch.zeros(scales)), (1, 200, 300))


def routing(**kw):
    a = dict(W_router=torch.zeros(16, 256, dtype=torch.bfloat16), expert_bias=torch.zeros(16),
             w_shared=torch.zeros(256, dtype=torch.bfloat16))
    a.update(kw)
    return a


BAD = [("W_router", torch.zeros(15, 256, dtype=torch.bfloat16)), ("W_router", torch.zeros(16, 256)),
       ("W_router", torch.zeros(16, 128, dtype=torch.bfloat16)), ("expert_bias", torch.zeros(15)),
       ("expert_bias", torch.zeros(16, dtype=torch.bfloat16)), 
       ("w_shared", torch.zeros(255, dtype=torch.bfloat16)), ("w_shared", torch.zeros(256))]
BAD_IDS = ["%s-%s-%s" % (n, "x".join(map(str, t.shape)), str(t.dtype)[6:]) for n, t in BAD]


@pytest.mark.parametrize("name,bad", BAD, ids=BAD_IDS)
def test_routing_tensors_of_the_layer(name, bad):
    """The router's matrix, its bias and the shared gate's vector: types and
    shapes, in the calls and in Fp8Experts."""
    cfg = smr.MoEConfig(T=4, d_model=256, n_experts=16, top_k=4, d_ff=64, d_ff_shared=64,
                        expert_dtype=smr.F8_E4M3_B128)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    ids, alpha, out = torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4), torch.zeros(4, 256)
    ws = torch.zeros(8, dtype=torch.uint8)

    def layer(t):
        smr.fp8_layer_forward(cfg, ws, x, t["W_router"], None, None, None, out, ids, alpha,
                              expert_bias=t["expert_bias"], w_shared=t["w_shared"])

    with pytest.raises(ValueError, match="CUDA"):
        layer(routing())
    with pytest.raises(ValueError, match="^" + name):
        layer(routing(**{name: bad}))
    with pytest.raises(ValueError, match="^" + name):
        smr.Fp8Experts(cfg, routing(**{name: bad}))
    if name == "w_shared":
        with pytest.raises(ValueError, match="^" + name):
            smr.fp8_experts_forward(cfg, ws, x, ids, alpha, None, None, None, out, w_shared=bad)
