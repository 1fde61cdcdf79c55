"""The 8-bit operators on the GPU where their form or their state matters:
precision of fp32 results, many slots, streams, workspaces, timeouts, large
grids, the layer's own shapes and its other routing rule."""
import gc
import math

import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import sparse_moe_routing_gb300 as smr  # noqa: E402
from fp8_util import (F8, bank, blocks, experts_ref, pitched, quantize64, random_matrix,  # noqa: E402
                      round_e4m3, values)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_routing_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def disarmed():
    yield
    smr.inject_stall(None, 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# (d, E, k, width, shared width)
SHAPES = {"tiny": (256, 16, 4, 64, 64), "ragged": (272, 5, 2, 144, 80), "wide": (512, 8, 2, 896, 0),
          "apart": (384, 12, 4, 128, 512), "slots": (256, 40, 32, 64, 64), "e256": (2048, 256, 8, 512, 512)}


def config(shape, T, path=smr.PATH_AUTO, **kw):
    d, E, k, width, shared = SHAPES[shape]
    return smr.MoEConfig(**(dict(T=T, d_model=d, n_experts=E, top_k=k, d_ff=width, d_ff_shared=shared,
                                 expert_dtype=smr.F8_E4M3_B128, path=path) | kw))


# ---------------------------------------------------------------------------
# a layer whose h has exact codes
# ---------------------------------------------------------------------------
def exact_bank(g, E, N, K, gate):
    """Codes 64, 128 or 256 (gate), or 1 to 15 with either sign (up); scales 2^-3."""
    if gate:
        v = torch.exp2(torch.randint(6, 9, (E, N, K), generator=g, device="cuda").float())
    else:
        v = torch.randint(1, 16, (E, N, K), generator=g, device="cuda").float()
        v = v * (1 - 2 * torch.randint(0, 2, (E, N, K), generator=g, device="cuda").float())
    return v.to(F8), torch.full((E, blocks(N), blocks(K)), 2.0 ** -3, device="cuda")


def make_exact(shape, T, k=None, seed=0):
    """Inputs for which every code of h is beyond doubt. x has one value, 8, a
    row: a gate sum is 64, 128 or 256, whose SiLU is itself to 1e-27, an up sum a
    whole number of magnitude 1 to 15; their product has four significant bits and
    so an e4m3 code of its own, which an error of some ulps does not change. What
    is left to differ are the sums of down and over the slots."""
    d, E, k0, width, shared = SHAPES[shape]
    k = k or k0
    g = gen(31 * T + seed)
    x = torch.zeros(T, d, device="cuda")
    x[torch.arange(T, device="cuda"), torch.randint(0, d, (T,), generator=g, device="cuda")] = 8.0
    w = {"W_gate": exact_bank(g, E, width, d, True), "W_up": exact_bank(g, E, width, d, False),
         "W_down": bank(g, E, d, width)}
    gate = None
    if shared:
        w |= {"Ws_gate": exact_bank(g, 1, shared, d, True),
              "Ws_up": exact_bank(g, 1, shared, d, False), "Ws_down": bank(g, 1, d, shared)}
        gate = torch.sigmoid(torch.randn(T, generator=g, device="cuda"))
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=-1).indices.to(torch.int32)
    alpha = torch.rand(T, k, generator=g, device="cuda") + 0.1
    return x.to(torch.bfloat16), ids, alpha, w, gate


def check_sums(out, x, ids, alpha, w, gate, r=None):
    """Elementwise: the additions of a block of 128 products, of the blocks and of
    the slots (a k split adds no more), each off by 2^-23 of the sum of magnitudes
    at most, and five roundings of a term (two scales, the weight, the split's and
    the residual's sum); a bf16 result is off by half a step, 2^-8, more."""
    ref = experts_ref(x, ids, alpha, w, gate, r)
    plain = {n: (c.float().abs().to(F8), s) for n, (c, s) in w.items()}
    mag = experts_ref(x, ids, alpha, plain, gate, None if r is None else r.abs())
    width = max(w["W_down"][0].shape[-1], w["Ws_down"][0].shape[-1] if "Ws_down" in w else 0)
    n = min(width, 128) + blocks(width) + ids.shape[1] + 1 + 5
    tol = n * 2.0 ** -23 * mag + 1e-30
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


PRECISE = [("tiny", 1), ("tiny", 16), ("tiny", 17), ("tiny", 200), ("ragged", 5), ("ragged", 40), ("wide", 3),
           ("wide", 64), ("wide", 300), ("apart", 10), ("apart", 33), ("apart", 260), ("e256", 1), ("e256", 8),
           ("e256", 17), ("e256", 64)]


@pytest.mark.parametrize("shape,T", PRECISE, ids=["%s-%d" % c for c in PRECISE])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_slot_rows_are_summed_in_fp32(shape, T, out_dtype):
    """Nothing between h's codes and the result is rounded to fewer than 32 bits."""
    x, ids, alpha, w, gate = make_exact(shape, T)
    r = torch.randn(x.shape, generator=gen(T), device="cuda") if out_dtype == torch.float32 else None
    layer = smr.Fp8Experts(config(shape, T), w)
    out = torch.full(x.shape, 9.0, dtype=out_dtype, device="cuda")
    layer.forward(x, ids, alpha, s_shared=gate, r_attn=r, out=out)
    check_sums(out, x, ids, alpha, w, gate, r)


@pytest.mark.parametrize("path", [smr.PATH_GEMV, smr.PATH_TC], ids=["few", "tc"])
@pytest.mark.parametrize("T", [3, 16])
def test_slot_rows_are_summed_in_fp32_on_either_path(path, T):
    x, ids, alpha, w, gate = make_exact("tiny", T)
    out = torch.empty(x.shape, device="cuda")
    smr.Fp8Experts(config("tiny", T, path), w).forward(x, ids, alpha, s_shared=gate, out=out)
    check_sums(out, x, ids, alpha, w, gate)


# ---------------------------------------------------------------------------
# many slots a token
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,k", [(16, 20), (16, 22), (16, 32), (15, 23), (11, 32), (10, 32), (1, 32), (17, 32)])
def test_experts_with_many_slots(T, k):
    """top_k up to 32 at every number of tokens."""
    x, ids, alpha, w, gate = make_exact("slots", T, k)
    out = torch.empty(x.shape, device="cuda")
    for path in (smr.PATH_AUTO,) + ((smr.PATH_GEMV,) if T <= 16 else ()):
        layer = smr.Fp8Experts(config("slots", T, path, top_k=k), w)
        out.fill_(9.0)
        layer.forward(x, ids, alpha, s_shared=gate, out=out)
        check_sums(out, x, ids, alpha, w, gate)
        assert layer.device_status()[0] == 0


# ---------------------------------------------------------------------------
# products: infinite scales
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 9, 16, 17, 40])
@pytest.mark.parametrize("K", [128, 100, 256, 640])
def test_matmul_infinite_scales_and_sums(M, K):
    """A row with an infinite scale (positive codes) gives infinity, and so does a
    product of scales above fp32's range, also where the number of blocks is odd."""
    g = gen(M + K)
    a = pitched((torch.rand(M, K, generator=g, device="cuda") * 100 + 1).to(F8))
    b = pitched((torch.rand(33, K, generator=g, device="cuda") * 100 + 1).to(F8))
    sa, sb = torch.ones(M, blocks(K), device="cuda"), torch.ones(1, blocks(K), device="cuda")
    out = torch.empty(M, 33, device="cuda")
    ws = smr.fp8_matmul_workspace(M, 33, K)
    sa[0] = math.inf
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    assert bool((out[0] == math.inf).all()) and bool(out[1:].isfinite().all())
    sa.fill_(2.0 ** 70)
    sb.fill_(2.0 ** 70)
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    assert bool((out == math.inf).all())


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
def test_results_are_allocated_on_the_calls_stream():
    """A result that the call allocates and the caller drops early is not handed
    out on the current stream while the call's stream may still write it."""
    T = 700
    x, ids, alpha, w, gate = make_exact("tiny", T)
    w["W_router"], w["w_shared"] = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in ((16, 256), 256))
    layer = smr.Fp8Experts(config("tiny", T), w)
    ids2, alpha2 = ids.clone(), alpha.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in (lambda: layer.forward(x, ids, alpha, s_shared=gate, stream=side),
                 lambda: layer.layer(x, ids2, alpha2, stream=side),
                 lambda: smr.fp8_matmul_workspace(64, 512, 8192, stream=side),
                 lambda: smr.fp8_alloc_workspace(config("tiny", T), stream=side),
                 lambda: smr.alloc_workspace(smr.MoEConfig(T=T, d_model=256, n_experts=16, top_k=4, d_ff=64),
                                             stream=side)):
        out = call()
        at, size, dtype = out.data_ptr(), out.shape, out.dtype
        del out
        assert torch.empty(size, dtype=dtype, device="cuda").data_ptr() != at
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# Fp8Linear
# ---------------------------------------------------------------------------
def test_linear_keeps_one_workspace_and_captures():
    """One workspace for every row count, made with the object: other row counts
    allocate nothing, not even inside a capture, and give the product's bits."""
    g = gen(6)
    N, K, rows = 512, 4096, 300
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16) * 0.02
    lin = smr.Fp8Linear(w, rows)
    x = torch.randn(rows, K, generator=g, device="cuda").to(torch.bfloat16)
    want = {}
    for M in (1, 16, 17, 128, 129, 300):
        xq, xs = smr.fp8_empty(M, K)
        smr.fp8_quantize(x[:M], xq, xs)
        want[M] = torch.empty(M, N, device="cuda")
        smr.fp8_matmul(xq, xs, lin.codes, lin.scales, want[M], smr.fp8_matmul_workspace(M, N, K))
    out = torch.empty(rows, N, device="cuda")
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()
    for M in want:
        lin(x[:M], out[:M])
        assert torch.equal(out[:M], want[M])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(x[:100], out[:100])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:100], want[128][:100])
    del graph
    assert torch.cuda.memory_allocated() == before
    with pytest.raises(ValueError):
        lin(torch.zeros(rows + 1, K, device="cuda"), torch.empty(rows + 1, N, device="cuda"))


def test_linear_reports_a_timeout():
    g = gen(7)
    lin = smr.Fp8Linear(torch.randn(300, 512, generator=g, device="cuda"), 200)
    x, out = torch.randn(200, 512, generator=g, device="cuda"), torch.empty(200, 300, device="cuda")
    want = lin(x, out).clone()
    assert lin.device_status()[0] == 0
    smr.inject_stall("f8_matmul", 2000)
    lin(x, out)
    assert lin.device_status()[0] == smr._STATUS.index("MOE_ERR_DEVICE_TIMEOUT")
    assert torch.equal(lin(x, out), want) and lin.device_status()[0] == 0


# ---------------------------------------------------------------------------
# one workspace, batches of several sizes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shape", ["tiny", "apart", "wide"])
def test_one_workspace_serves_every_number_of_tokens(shape):
    """Initialised once for the largest batch, then used for others in turn: bit
    for bit what a workspace of their own gives."""
    sizes = (64, 5, 200, 16, 1, 64, 9)
    ws = smr.fp8_alloc_workspace(config(shape, max(sizes)))
    for T in sizes:
        x, ids, alpha, w, gate = make_exact(shape, T)
        want = smr.Fp8Experts(config(shape, T), w).forward(x, ids, alpha, s_shared=gate)
        out = torch.empty_like(want)
        smr.fp8_experts_forward(config(shape, T), ws, x, ids, alpha, w["W_gate"], w["W_up"], w["W_down"], out,
                                s_shared=gate, Ws_gate=w.get("Ws_gate"), Ws_up=w.get("Ws_up"),
                                Ws_down=w.get("Ws_down"))
        assert torch.equal(out, want)
        assert smr.read_device_status(config(shape, T), ws)[0] == 0


# ---------------------------------------------------------------------------
# after a timeout
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shape,T", [("tiny", 5), ("apart", 16), ("tiny", 40)])
def test_reading_a_timeout_makes_the_workspace_usable(shape, T):
    """What a kernel that gave up leaves behind, made on the host: the status bit
    and counts of finished items (here ones that never come to an end)."""
    x, ids, alpha, w, gate = make_exact(shape, T)
    layer = smr.Fp8Experts(config(shape, T), w)
    want = layer.forward(x, ids, alpha, s_shared=gate).clone()
    layer.ws.fill_(0)
    layer.ws[256:].view(torch.int32).fill_(1000)
    layer.ws[:4].view(torch.int32).fill_(2)
    assert layer.device_status()[0] == smr._STATUS.index("MOE_ERR_DEVICE_TIMEOUT")
    assert torch.equal(layer.forward(x, ids, alpha, s_shared=gate), want)
    assert layer.device_status()[0] == 0


@pytest.mark.parametrize("kernel,shape,T", [("f8_tc_gateup", "tiny", 5), ("f8_tc_gateup", "e256", 8),
                                            ("f8_tc_down", "tiny", 5), ("f8_tc_down", "e256", 16)])
def test_few_token_waits_that_run_out_are_reported(kernel, shape, T):
    """The few-token kernels take the stall of the layer's gate/up and down."""
    x, ids, alpha, w, gate = make_exact(shape, T)
    layer = smr.Fp8Experts(config(shape, T), w)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    want = layer.forward(x, ids, alpha, s_shared=gate, out=out).clone()
    smr.inject_stall(kernel, 2000)
    layer.forward(x, ids, alpha, s_shared=gate, out=out)
    assert layer.device_status()[0] == smr._STATUS.index("MOE_ERR_DEVICE_TIMEOUT")
    layer.forward(x, ids, alpha, s_shared=gate, out=out)
    assert layer.device_status()[0] == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("M,N,K", [(1, 640, 256), (8, 4096, 2048), (16, 300, 1000)])
def test_few_row_product_wait_that_runs_out_is_reported(M, N, K):
    g = gen(M)
    (a, sa), (b, sb) = random_matrix(g, M, K, 1), random_matrix(g, N, K, 128)
    out, ws = torch.empty(M, N, device="cuda"), smr.fp8_matmul_workspace(M, N, K)
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    want = out.clone()
    cfg = smr.MoEConfig(T=1, d_model=128, n_experts=1, top_k=1, d_ff=128)
    smr.inject_stall("f8_matmul", 2000)
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    assert smr.read_device_status(cfg, ws)[0] == smr._STATUS.index("MOE_ERR_DEVICE_TIMEOUT")
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    assert smr.read_device_status(cfg, ws)[0] == 0
    assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# the object's own weights
# ---------------------------------------------------------------------------
def test_experts_hold_their_weights_themselves():
    """The banks stay alive and in use when the caller empties its dict."""
    x, ids, alpha, w, gate = make_exact("tiny", 5)
    layer = smr.Fp8Experts(config("tiny", 5), w)
    banks = dict(w)
    want = layer.forward(x, ids, alpha, s_shared=gate).clone()
    w.clear()
    assert all(layer.w[n][i] is banks[n][i] for n in banks for i in (0, 1))
    assert torch.equal(layer.forward(x, ids, alpha, s_shared=gate), want)


def test_experts_hold_their_configuration_themselves():
    """The sizes that a call checks are those that it was made for."""
    x, ids, alpha, w, gate = make_exact("tiny", 5)
    cfg = config("tiny", 5)
    layer = smr.Fp8Experts(cfg, w)
    want = layer.forward(x, ids, alpha, s_shared=gate).clone()
    for c in (cfg, layer.cfg):
        c.T = 3
        with pytest.raises(ValueError):
            layer.forward(x[:3], ids[:3], alpha[:3], s_shared=gate[:3])
        assert torch.equal(layer.forward(x, ids, alpha, s_shared=gate), want)


# ---------------------------------------------------------------------------
# sizes at which a block or a CTA takes more than one turn
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(4097, 1001), (4097, 1024), (2500, 1100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_quantize_many_blocks(rows, cols, dtype):
    x = torch.randn(rows, cols, generator=gen(rows + cols), device="cuda")
    x = (x * torch.exp(3 * torch.randn(rows, 1, generator=gen(7), device="cuda"))).to(dtype)
    codes, scales = smr.fp8_empty(rows, cols)
    smr.fp8_quantize(x, codes, scales)
    p = torch.nn.functional.pad(x.double(), (0, -cols % 128)).view(rows, -1, 128)
    m, e = torch.frexp(p.abs().amax(-1))
    s = torch.exp2(torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126).double())
    assert torch.equal(scales.double(), s)
    assert torch.equal(codes.double(), round_e4m3(p / s[..., None]).view(rows, -1)[:, :cols])
    assert torch.equal(values(codes, scales, 1), quantize64(x.double()))


@pytest.mark.parametrize("M,N,K", [(1700, 3000, 400), (1300, 300, 2048), (1025, 520, 1100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul_many_tiles(M, N, K, dtype):
    """More tiles than SMs (a CTA's second tile), and split k over more than one
    band of row blocks; bound of the sums as for the smaller products."""
    g = gen(M + N + K)
    (a, sa), (b, sb) = random_matrix(g, M, K, 1), random_matrix(g, N, K, 128)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    smr.fp8_matmul(a, sa, b, sb, out, smr.fp8_matmul_workspace(M, N, K))
    A, B = values(a, sa, 1), values(b, sb, 128)
    ref = A @ B.T
    tol = (128 + blocks(K) + 2) * 2.0 ** -23 * (A.abs() @ B.abs().T) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


# ---------------------------------------------------------------------------
# the sigmoid-group rule with 8-bit banks
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 16, 40])
def test_layer_with_the_sigmoid_group_rule(T):
    """ids and weights are bit for bit those of the routing call; the result is
    that of the experts for them."""
    d, E, k, width, shared = SHAPES["tiny"]
    x, _, _, w, _ = make_exact("tiny", T)
    g = gen(T)
    w["W_router"] = (torch.randn(E, d, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    w["w_shared"] = (torch.randn(d, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    w["expert_bias"] = torch.randn(E, generator=g, device="cuda") * 0.1
    rule = dict(router=smr.SIGMOID_GROUP_TOPK, n_group=4, topk_group=2, routed_scaling=2.5)
    layer = smr.Fp8Experts(config("tiny", T, **rule), w)
    ids, alpha = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out = layer.layer(x, ids, alpha, out=torch.empty(T, d, device="cuda"))
    base = smr.MoEConfig(T=T, d_model=d, n_experts=E, top_k=k, d_ff=width, d_ff_shared=shared,
                         path=smr.PATH_GEMV, **rule)  # the separate routing kernels
    ids16, alpha16 = torch.empty_like(ids), torch.empty_like(alpha)
    smr.route(base, smr.alloc_workspace(base), x, w["W_router"], ids16, alpha16, expert_bias=w["expert_bias"])
    assert torch.equal(ids, ids16) and torch.equal(alpha, alpha16)
    gate = torch.sigmoid(x.double() @ w["w_shared"].double())
    half = layer.forward(x, ids, alpha, s_shared=gate.float(), out=torch.empty(T, d, device="cuda"))
    banks = {n: b for n, b in w.items() if isinstance(b, tuple)}
    check_sums(half, x, ids, alpha, banks, gate.float())
    assert float((out - half).abs().max()) <= 1e-5 * float(half.abs().max())
