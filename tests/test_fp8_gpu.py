"""The 8-bit operators on the GPU against their plain 64-bit forms."""
import ctypes
import math

import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

import sparse_moe_routing_gb300 as smr  # noqa: E402
from fp8_util import (F8, bank, blocks, experts_ref, pitched, quantize64, quantize_ref,  # noqa: E402
                      random_matrix, values)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_routing_gb300 import build
    build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# quantise: codes and scales are exact
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (5, 64), (17, 2048), (130, 200),
                                       (129, 1001), (256, 384), (2, 4096), (300, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_matches_the_definition(rows, cols, dtype, block_rows):
    x = torch.randn(rows, cols, generator=gen(rows + cols), device="cuda")
    x = (x * torch.exp(3 * torch.randn(rows, 1, generator=gen(7), device="cuda"))).to(dtype)
    codes, scales = smr.fp8_empty(rows, cols, block_rows)
    smr.fp8_quantize(x, codes, scales, block_rows=block_rows)
    want, s = quantize_ref(x, block_rows)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.double().cpu(), want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_borders(block_rows):
    """Zeros, signed zero, values at 448 times a power of two and one step to
    either side, subnormal values, the largest ones, and exact ties."""
    x = torch.zeros(128 * 10, 128, device="cuda")
    rows = [0, 128, 256, 384, 512, 640, 768, 896, 1024, 1152]
    x[128, :4] = torch.tensor([448.0, -448.0, 1.0, -0.0])
    x[256, :2] = torch.tensor([math.nextafter(448.0, 449.0), 3.0], dtype=torch.float64).float()
    x[256, 0] = 448.00003
    x[384, :3] = torch.tensor([2.0 ** -149, 2.0 ** -140, -2.0 ** -126])
    x[512, :2] = torch.tensor([3.4028234e38, -1.7e38])
    x[640, :6] = torch.tensor([256.0, 17.0, 19.0, 21.0, 2.0 ** -10, 3 * 2.0 ** -10])   # ties
    x[768, :2] = torch.tensor([7.0 * 2.0 ** -120, 2.0 ** -126])
    x[896, :2] = torch.tensor([1.75, 1.7500001])
    x[1024, :2] = torch.tensor([-0.875, 0.01])
    x[1152, 5] = -1e-30
    assert len(rows) == 10
    codes, scales = smr.fp8_empty(*x.shape, block_rows)
    smr.fp8_quantize(x, codes, scales, block_rows=block_rows)
    want, s = quantize_ref(x, block_rows)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.double().cpu(), want)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_marks_only_blocks_that_are_not_finite(value, block_rows):
    x = torch.randn(256, 300, generator=gen(1), device="cuda")
    x[130, 129] = value
    codes, scales = smr.fp8_empty(256, 300, block_rows)
    smr.fp8_quantize(x, codes, scales, block_rows=block_rows)
    want, s = quantize_ref(x, block_rows)
    assert torch.equal(scales.isnan().cpu(), s.isnan()) and int(s.isnan().sum()) == 1
    assert torch.equal(codes.double().nan_to_num(777.0).cpu(), want.nan_to_num(777.0))


def test_quantize_strides_stacks_and_untouched_padding():
    """A column slice at an odd offset, a stack, and padding that stays as it was."""
    big = torch.randn(70, 500, generator=gen(2), device="cuda").to(torch.bfloat16)
    x = big[:, 3:300]
    room = torch.full((70, 400), 9, dtype=torch.uint8, device="cuda").view(F8)
    codes, (_, scales) = room[:, 5:302], smr.fp8_empty(70, 297)
    smr.fp8_quantize(x, codes, scales)
    want, s = quantize_ref(x, 1)
    assert torch.equal(codes.double().cpu(), want) and torch.equal(scales.cpu(), s)
    raw = room.view(torch.uint8)
    assert int((raw[:, :5] != 9).sum()) == 0 and int((raw[:, 302:] != 9).sum()) == 0
    st = torch.randn(3, 200, 144, generator=gen(3), device="cuda")
    for br in (1, 128):
        codes, scales = smr.fp8_empty(200, 144, br, count=3)
        smr.fp8_quantize(st, codes, scales, block_rows=br)
        for i in range(3):
            want, s = quantize_ref(st[i], br)
            assert torch.equal(codes[i].double().cpu(), want) and torch.equal(scales[i].cpu(), s)


def test_quantize_empty():
    codes, scales = smr.fp8_empty(0, 64)
    smr.fp8_quantize(torch.empty(0, 64, device="cuda"), codes, scales)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def check_matmul(a, sa, b, sb, out):
    """Elementwise: the products of a block of 128 and the blocks' sums are added
    in fp32, each addition off by at most 2^-23 of the running magnitude (a
    rounding or a truncation), the scaling by two roundings more; bf16 out is
    off by half a step, 2^-8, more."""
    A, B = values(a, sa, 1), values(b, sb, 128)
    ref = A @ B.T
    mag = A.abs() @ B.abs().T
    tol = (min(a.shape[1], 128) + blocks(a.shape[1]) + 2) * 2.0 ** -23 * mag + 1e-30
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def run_matmul(M, N, K, dtype, seed=0, **kw):
    g = gen(1000 * seed + M + N + K)
    a, sa = random_matrix(g, M, K, 1)
    b, sb = random_matrix(g, N, K, 128)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    ws = smr.fp8_matmul_workspace(M, N, K)
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    return a, sa, b, sb, out, ws


# few rows (1..16), one tile, several tiles, k split, ragged in each direction
MM = [(1, 1, 1), (1, 16, 128), (1, 64, 2048), (2, 17, 16), (3, 100, 333), (8, 256, 1408), (9, 130, 640),
      (16, 5632, 256), (16, 48, 130), (17, 1, 1), (17, 256, 128), (33, 257, 129), (64, 512, 4096),
      (127, 255, 1000), (128, 256, 512), (129, 1000, 2048), (300, 1408, 2048), (700, 640, 96)]


@pytest.mark.parametrize("M,N,K", MM, ids=["%dx%dx%d" % s for s in MM])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_matmul(M, N, K, dtype):
    a, sa, b, sb, out, _ = run_matmul(M, N, K, dtype)
    check_matmul(a, sa, b, sb, out)


@pytest.mark.parametrize("M", [5, 40])
def test_matmul_strided_output_and_operands(M):
    """out a slice of a wider matrix at an odd column; a and b slices of wider
    ones; what lies around out stays as it was."""
    g = gen(M)
    N, K = 333, 272
    a, sa = random_matrix(g, M, 512, 1)
    b, sb = random_matrix(g, N, 512, 128)
    a, b = a[:, 128:128 + K], b[:, 128:128 + K]
    sa, sb = sa[:, 1:1 + blocks(K)].contiguous(), sb[:, 1:1 + blocks(K)].contiguous()
    for dtype in (torch.float32, torch.bfloat16):
        room = torch.full((M, 400), 3.0, dtype=dtype, device="cuda")
        out = room[:, 7:7 + N]
        smr.fp8_matmul(a, sa, b, sb, out, smr.fp8_matmul_workspace(M, N, K))
        check_matmul(a, sa, b, sb, out)
        assert bool((room[:, :7] == 3).all()) and bool((room[:, 7 + N:] == 3).all())


@pytest.mark.parametrize("M", [4, 64, 200])
def test_matmul_keeps_nan_to_its_rows_and_columns(M):
    """A NaN code in one row of a, a NaN scale of another and a NaN code in one
    row of b leave every other element as it was."""
    N, K = 300, 512
    a, sa, b, sb, out, ws = run_matmul(M, N, K, torch.float32)
    want = out.clone()
    a, b, sa = a.clone(), b.clone(), sa.clone()
    a.view(torch.uint8)[1, 200] = 0x7F
    b.view(torch.uint8)[130, 3] = 0xFF
    sa[3, 0] = math.nan
    smr.fp8_matmul(a, sa, b, sb, out, ws)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1] = bad[3] = True
    bad[:, 130] = True
    assert torch.equal(out.isnan(), bad)
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("M,N,K", [(6, 512, 4096), (48, 512, 8192), (300, 512, 512)])
def test_matmul_is_deterministic_and_leaves_its_workspace_ready(M, N, K):
    a, sa, b, sb, out, ws = run_matmul(M, N, K, torch.float32)
    first = out.clone()
    for _ in range(5):
        out.fill_(0)
        smr.fp8_matmul(a, sa, b, sb, out, ws)
        assert torch.equal(out, first)


def test_matmul_captured_and_on_another_stream():
    a, sa, b, sb, out, ws = run_matmul(48, 512, 8192, torch.bfloat16)
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.fill_(0)
        smr.fp8_matmul(a, sa, b, sb, out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smr.fp8_matmul(a, sa, b, sb, out, ws)
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_matmul_of_nothing():
    for M, N in ((0, 64), (64, 0)):
        a, sa = random_matrix(gen(0), M, 128, 1)
        b, sb = random_matrix(gen(0), N, 128, 128)
        smr.fp8_matmul(a, sa, b, sb, torch.empty(M, N, device="cuda"), smr.fp8_matmul_workspace(M, N, 128))


def test_linear_quantises_and_multiplies():
    g = gen(5)
    w = torch.randn(640, 384, generator=g, device="cuda").to(torch.bfloat16) * 0.02
    lin = smr.Fp8Linear(w, 64)
    wv = values(*quantize_ref(w, 128), 128).cuda()
    for M in (1, 64):
        x = torch.randn(M, 384, generator=g, device="cuda").to(torch.bfloat16)
        out = lin(x, torch.empty(M, 640, device="cuda"))
        ref = quantize64(x.double()) @ wv.T
        mag = quantize64(x.double()).abs() @ wv.abs().T
        assert bool(((out.double() - ref).abs() <= 133 * 2.0 ** -23 * mag).all())


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------
# (d, E, k, width, shared width)
SHAPES = {
    "tiny": (256, 16, 4, 64, 64), "ragged": (272, 5, 2, 144, 80), "one": (128, 1, 1, 128, 0),
    "wide": (512, 8, 2, 896, 0), "apart": (384, 12, 4, 128, 512), "many": (256, 300, 8, 128, 128),
    "deep": (4096, 4, 2, 144, 400),
}


def make(shape, T, seed=0, ids=None, residual=False):
    d, E, k, width, shared = SHAPES[shape]
    g = gen(17 * T + seed)
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    # weights larger than a model's, so that h and y are of the order of one
    w = {"W_gate": bank(g, E, width, d), "W_up": bank(g, E, width, d), "W_down": bank(g, E, d, width)}
    gate = None
    if shared:
        w |= {"Ws_gate": bank(g, 1, shared, d), "Ws_up": bank(g, 1, shared, d), "Ws_down": bank(g, 1, d, shared)}
        gate = torch.sigmoid(torch.randn(T, generator=g, device="cuda"))
    if ids is None:
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=-1).indices.to(torch.int32)
    alpha = torch.rand(T, k, generator=g, device="cuda") + 0.1
    r = torch.randn(T, d, generator=g, device="cuda") if residual else None
    return x, ids, alpha, w, gate, r


def config(shape, T, path=smr.PATH_AUTO):
    d, E, k, width, shared = SHAPES[shape]
    return smr.MoEConfig(T=T, d_model=d, n_experts=E, top_k=k, d_ff=width, d_ff_shared=shared,
                         expert_dtype=smr.F8_E4M3_B128, path=path)


def check_experts(out, ref, shape, residual=None):
    """Row by row, in the 2-norm of what the experts add: half a step of bf16,
    2^-8, for the slots' rows and (bf16 out) for the result; and h, computed in
    fp32, may round to the neighbouring e4m3 code where it lies next to a tie:
    one code in a thousand, or one of a row's, off by a step of 2^-3."""
    width = SHAPES[shape][3]
    tol = 2 * 2.0 ** -8 + 2.0 ** -3 * math.sqrt(max(1e-3, 1.0 / width))
    y = ref if residual is None else ref - residual.double()
    err = (out.double() - ref).norm(dim=1)
    allow = tol * y.norm(dim=1) + (2.0 ** -8 * ref.norm(dim=1) if out.dtype == torch.bfloat16 else 0)
    assert bool((err <= allow).all()), float((err / allow).max())


CASES = [("tiny", 1), ("tiny", 2), ("tiny", 8), ("tiny", 9), ("tiny", 16), ("tiny", 17), ("tiny", 130),
         ("tiny", 700), ("ragged", 1), ("ragged", 5), ("ragged", 16), ("ragged", 40), ("ragged", 300),
         ("one", 1), ("one", 16), ("one", 129), ("wide", 1), ("wide", 3), ("wide", 64), ("wide", 257),
         ("apart", 1), ("apart", 10), ("apart", 33), ("apart", 260), ("many", 1), ("many", 16),
         ("many", 64), ("many", 600), ("deep", 1), ("deep", 8), ("deep", 16), ("deep", 20)]


@pytest.mark.parametrize("shape,T", CASES, ids=["%s-%d" % c for c in CASES])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_experts(shape, T, out_dtype):
    residual = out_dtype == torch.float32
    x, ids, alpha, w, gate, r = make(shape, T, residual=residual)
    layer = smr.Fp8Experts(config(shape, T), w)
    out = torch.full(x.shape, 9.0, dtype=out_dtype, device="cuda")
    layer.forward(x, ids, alpha, s_shared=gate, r_attn=r, out=out)
    check_experts(out, experts_ref(x, ids, alpha, w, gate, r), shape, r)
    assert layer.device_status()[0] == 0


@pytest.mark.parametrize("shape,T", [("tiny", 3), ("ragged", 16), ("apart", 7), ("wide", 12)])
def test_experts_tensor_core_path_for_few_tokens(shape, T):
    x, ids, alpha, w, gate, r = make(shape, T)
    out = smr.Fp8Experts(config(shape, T, smr.PATH_TC), w).forward(x, ids, alpha, s_shared=gate)
    check_experts(out, experts_ref(x, ids, alpha, w, gate), shape)


@pytest.mark.parametrize("T", [8, 16, 150])
def test_experts_uneven_and_repeated_ids(T):
    """Every token on one expert; the same expert in several slots of a token;
    all other experts idle."""
    d, E, k, _, _ = SHAPES["tiny"]
    for ids in (torch.full((T, k), 5, dtype=torch.int32, device="cuda"),
                torch.tensor([[3, 3, 15, 0]], dtype=torch.int32, device="cuda").repeat(T, 1),
                (torch.arange(T * k, dtype=torch.int32, device="cuda") % 2 * 15).view(T, k).contiguous()):
        x, _, alpha, w, gate, r = make("tiny", T)
        out = smr.Fp8Experts(config("tiny", T), w).forward(x, ids, alpha, s_shared=gate)
        check_experts(out, experts_ref(x, ids, alpha, w, gate), "tiny")


@pytest.mark.parametrize("T", [4, 150])
def test_experts_keep_a_bad_token_to_itself(T):
    """A token with an infinite value gives NaN; the others stay bit for bit."""
    x, ids, alpha, w, gate, _ = make("tiny", T)
    layer = smr.Fp8Experts(config("tiny", T), w)
    want = layer.forward(x, ids, alpha, s_shared=gate).clone()
    x = x.clone()
    x[2, 100] = math.inf
    out = layer.forward(x, ids, alpha, s_shared=gate)
    assert bool(out[2].isnan().all())
    keep = torch.arange(T, device="cuda") != 2
    assert torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("T", [1, 16, 130])
def test_experts_zero_tokens_and_zero_weights(T):
    """x = 0 gives y = 0 exactly, and so does alpha = 0 without the shared expert's gate."""
    x, ids, alpha, w, gate, r = make("tiny", T, residual=True)
    layer = smr.Fp8Experts(config("tiny", T), w)
    out = torch.empty_like(r)
    layer.forward(torch.zeros_like(x), ids, alpha, s_shared=gate, r_attn=r, out=out)
    assert torch.equal(out, r)
    layer.forward(x, ids, torch.zeros_like(alpha), s_shared=torch.zeros_like(gate), r_attn=r, out=out)
    assert torch.equal(out, r)


@pytest.mark.parametrize("T", [5, 16, 140])
def test_experts_repeat_in_place_stream_and_graph(T):
    """Bit for bit the same again, from a workspace full of NaN codes, in place
    on the residual, on another stream and from a captured graph."""
    x, ids, alpha, w, gate, r = make("apart", T, residual=True)
    layer = smr.Fp8Experts(config("apart", T), w)
    want = layer.forward(x, ids, alpha, s_shared=gate, r_attn=r, out=torch.empty_like(r)).clone()
    layer.ws.fill_(0xFF)
    st = smr.lib().moe_fp8_workspace_init(layer._cp, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    res = r.clone()
    layer.forward(x, ids, alpha, s_shared=gate, r_attn=res, out=res)
    assert torch.equal(res, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(r)
    with torch.cuda.stream(side):
        layer.forward(x, ids, alpha, s_shared=gate, r_attn=r, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, ids, alpha, s_shared=gate, r_attn=r, out=out)
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [6, 40])
def test_experts_report_an_id_out_of_range(T):
    x, ids, alpha, w, gate, _ = make("tiny", T)
    layer = smr.Fp8Experts(config("tiny", T), w)
    bad = ids.clone()
    bad[1, 2] = 16
    bad[3, 0] = -1
    out = layer.forward(x, bad, alpha, s_shared=gate).clone()
    st, word = layer.device_status()
    assert st == smr._STATUS.index("MOE_ERR_DEVICE_CHECK") and word & 1
    good = layer.forward(x, ids, alpha, s_shared=gate)
    assert layer.device_status()[0] == 0
    rows = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(out[rows], good[rows])


@pytest.mark.parametrize("T", [1, 7, 60, 200])
def test_layer_routes_then_runs_the_experts(T):
    """layer(): the routing of moe_route's separate kernels, the shared gate
    from w_shared, then the experts; against the expert half for its own ids."""
    d, E, k, width, shared = SHAPES["tiny"]
    x, _, _, w, _, r = make("tiny", T, residual=True)
    g = gen(T)
    w["W_router"] = (torch.randn(E, d, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    w["w_shared"] = (torch.randn(d, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    layer = smr.Fp8Experts(config("tiny", T), w)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    alpha = torch.empty(T, k, device="cuda")
    out = layer.layer(x, ids, alpha, r_attn=r, out=torch.empty_like(r)).clone()
    z = x.double() @ w["W_router"].double().T
    top, order = z.topk(k + 1, dim=-1)
    clear = (top[:, k - 1] - top[:, k]) > 1e-3
    assert torch.equal(ids[clear].sort(-1).values.long(), order[clear, :k].sort(-1).values)
    p = torch.softmax(z, -1).gather(1, ids.long())
    assert float((alpha.double() - p / p.sum(-1, keepdim=True)).abs().max()) < 1e-5
    gate = torch.sigmoid(x.double() @ w["w_shared"].double())
    check_experts(out, experts_ref(x, ids, alpha, w, gate, r), "tiny", r)
    # the expert half computes the gate itself when it is given w_shared only
    half = layer.forward(x, ids, alpha, r_attn=r, out=torch.empty_like(r))
    check_experts(half, experts_ref(x, ids, alpha, w, gate, r), "tiny", r)


def test_layer_from_bf16_weights():
    """Fp8Experts.from_bf16: the banks are the quantiser's of the bf16 weights,
    the ids are those of the bf16 layer's routing, and the layer computes with
    the banks' values."""
    d, E, k, width, shared = SHAPES["tiny"]
    g = gen(11)
    T = 33
    mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.03).to(torch.bfloat16)  # noqa: E731
    wb = {"W_router": mk(E, d), "W_gate": mk(E, width, d), "W_up": mk(E, width, d), "W_down": mk(E, d, width),
          "Ws_gate": mk(shared, d), "Ws_up": mk(shared, d), "Ws_down": mk(d, shared), "w_shared": mk(d)}
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    layer = smr.Fp8Experts.from_bf16(config("tiny", T), wb)
    for name in ("W_gate", "W_down"):
        codes, scales = layer.w[name]
        for e in (0, E - 1):
            want, s = quantize_ref(wb[name][e], 128)
            assert torch.equal(codes[e].double().cpu(), want) and torch.equal(scales[e].cpu(), s)
    ids, alpha = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out = layer.layer(x, ids, alpha)
    base = smr.MoEConfig(T=T, d_model=d, n_experts=E, top_k=k, d_ff=width, d_ff_shared=shared)
    ids16, alpha16 = torch.empty_like(ids), torch.empty_like(alpha)
    smr.route(base, smr.alloc_workspace(base), x, wb["W_router"], ids16, alpha16)
    assert torch.equal(ids, ids16) and torch.equal(alpha, alpha16)
    w = {n: layer.w[n] for n in ("W_gate", "W_up", "W_down")}
    w |= {n: (layer.w[n][0][None], layer.w[n][1][None]) for n in ("Ws_gate", "Ws_up", "Ws_down")}
    gate = torch.sigmoid(x.double() @ wb["w_shared"].double())
    check_experts(out, experts_ref(x, ids, alpha, w, gate), "tiny")


@pytest.mark.parametrize("kernel", ["f8_tc_gateup", "f8_tc_down", "f8_matmul"])
def test_a_wait_that_runs_out_is_reported(kernel):
    """The armed launch waits on a flag nothing sets, gives up, and the
    workspace is usable again."""
    if kernel == "f8_matmul":
        a, sa, b, sb, out, ws = run_matmul(200, 300, 512, torch.float32)
        want = out.clone()
        call = lambda: smr.fp8_matmul(a, sa, b, sb, out, ws)  # noqa: E731
        cfg = smr.MoEConfig(T=1, d_model=128, n_experts=1, top_k=1, d_ff=128)
        status = lambda: smr.read_device_status(cfg, ws)  # noqa: E731
    else:
        x, ids, alpha, w, gate, _ = make("tiny", 200)
        layer = smr.Fp8Experts(config("tiny", 200), w)
        out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        call = lambda: layer.forward(x, ids, alpha, s_shared=gate, out=out)  # noqa: E731
        call()
        want = out.clone()
        status = layer.device_status
    smr.inject_stall(kernel, 2000)
    call()
    assert status()[0] == smr._STATUS.index("MOE_ERR_DEVICE_TIMEOUT")
    call()
    assert status()[0] == 0
    assert torch.equal(out, want)


def test_example_runs_the_operators_together():
    """examples/fp8_layer.py on a small shape: quantised layer and projection.
    The projection's input and weights each round by at most 2^-4 of a value,
    2^-4 / sqrt(3) in the mean at worst, independently; bf16 out 2^-8 more."""
    import importlib.util
    import os

    import moe_inputs as mi
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("fp8_layer", os.path.join(root, "examples", "fp8_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    for tokens in (3, 40):
        off, off_y, us = ex.run(mi.DEEPSEEK_GROUP.with_(n_experts=16, d_model=1024), tokens, steps=2)
        # five roundings to e4m3 (x, gate and up as one, h, down, and the shared expert's in parallel)
        assert off < 3 * 2.0 ** -4 / math.sqrt(3)
        assert off_y < 2.0 ** -4 / math.sqrt(3) * math.sqrt(2) + 2.0 ** -8 and us > 0
