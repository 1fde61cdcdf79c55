"""The norm with the residual's addition and 8-bit output, on the GPU, against its definition in fp64."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr
from fp8_util import quantize_ref
from int8_util import STEP32, assert_near, codes32, half_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
# a value's room: s and t one rounding each, the factor f at most 24 (a sum of squares of at most 30 roundings in a
# chain, halved by the root; the mean, eps, the root and the quotient, half a step each), the last product one
ROOM = 28 * STEP32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, T, d, dtype, size=1.0):
    x = torch.randn(T, d, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    return (size * x).to(dtype)


def check(x, residual, gain, eps, out, sum_out, codes, scales):
    s32 = x.float() + residual.float() if residual is not None else x.float()  # one fp32 rounding
    t32 = s32 * gain.float() if gain is not None else s32                       # another
    s64 = x.double() + (residual.double() if residual is not None else 0)
    f = 1 / torch.sqrt(s64.square().mean(-1, keepdim=True) + eps)
    y = s64 * (gain.double() if gain is not None else 1) * f
    if sum_out is not None:
        assert torch.equal(sum_out, s32.to(sum_out.dtype))
    if out is not None:
        # what s lost by its rounding is relative to s
        assert_near(out, y, ROOM + half_step(out.dtype), what="out")
    if codes is not None and codes.dtype == torch.int8:
        want, s = codes32(t32.cpu())
        assert torch.equal(codes.cpu(), want)
        assert_near(scales.cpu(), s.double() * f[:, 0].cpu(), ROOM, what="scales")
    elif codes is not None:
        want, p = quantize_ref(t32, 1)
        assert torch.equal(codes.cpu().double(), want)
        assert_near(scales.cpu(), p.double() * f.cpu(), ROOM, what="scales")


CASES = [(1, 1), (1, 8), (3, 100), (9, 128), (5, 255), (17, 256), (8, 512), (2, 1000), (33, 1001), (4, 1024), (3, 1032),
         (1, 2048), (65, 2048), (333, 1001), (320, 2048), (2, 4096), (310, 4096), (310, 4100), (1, 8192), (305, 7000),
         (2, 16384), (305, 14336), (2, 16390), (3, 16392), (2, 32768)]


@pytest.mark.parametrize("kind", ["values", "int8", "e4m3", "all"])
@pytest.mark.parametrize("T,d", CASES)
def test_norm(T, d, kind):
    g = gen(T + d)
    i = (T + d + len(kind)) % 4
    xt, rt, gt = [(BF, F, BF), (F, BF, F), (BF, BF, F), (F, F, BF)][i]
    x, residual = rows(g, T, d, xt), rows(g, T, d, rt, 3.0)
    gain = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(gt)
    for r, gn in ((residual, gain), (None, gain), (residual, None), (None, None)):
        out = torch.empty(T, d, dtype=[BF, F][i % 2], device="cuda") if kind in ("values", "all") else None
        total = torch.empty(T, d, dtype=rt, device="cuda") if kind in ("values", "all") else None
        codes = scales = None
        if kind in ("int8", "all"):
            codes, scales = smr.int8_empty(T, d)
        elif kind == "e4m3":
            codes, scales = smr.fp8_empty(T, d)
        smr.add_rmsnorm(x, r, gn, 1e-5, out=out, sum_out=total, codes=codes, scales=scales)
        check(x, r, gn, 1e-5, out, total, codes, scales)


@pytest.mark.parametrize("d", [96, 1001, 2048])
def test_in_place(d):
    """The sum in the residual's or in x's place, the result in the other's."""
    g = gen(d)
    for T in (2, 400):
        x, r = rows(g, T, d, F), rows(g, T, d, F)
        gain = torch.rand(d, generator=g, device="cuda") + 0.5
        for sum_in_x in (False, True):
            a, b = x.clone(), r.clone()
            total, out = (a, b) if sum_in_x else (b, a)
            smr.add_rmsnorm(a, b, gain, out=out, sum_out=total)
            check(x, r, gain, 1e-6, out, total, None, None)


def test_views_and_neighbours():
    """Rows inside wider matrices at odd places; what lies around the outputs stays."""
    g = gen(2)
    T = 6
    for c0, d in ((0, 512), (8, 512), (4, 500), (1, 77), (3, 1100)):
        x, r = rows(g, T, 1200, BF)[:, c0:c0 + d], rows(g, T, 1200, F)[:, c0:c0 + d]
        room = torch.full((T + 2, 1300), 5.0, device="cuda")
        qroom = torch.full((T + 2, 1300), 55, dtype=torch.int8, device="cuda")
        out, codes = room[1:T + 1, c0:c0 + d], qroom[1:T + 1, c0:c0 + d]
        scales = torch.empty(T, device="cuda")
        smr.add_rmsnorm(x, r, out=out, codes=codes, scales=scales)
        check(x, r, None, 1e-6, out, None, codes, scales)
        out.fill_(5.0)
        codes.fill_(55)
        assert bool((room == 5.0).all()) and bool((qroom == 55).all())


@pytest.mark.parametrize("d", [64, 300, 3000, 4096])
def test_special_rows(d):
    """Zero rows, rows of the smallest numbers, an infinity or a NaN: each keeps to its own row."""
    T = 6
    x = torch.ones(T, d, device="cuda")
    x[1] = 0.0
    x[2] = 1e-42
    x[3, d // 2] = float("inf")
    x[4, d - 1] = float("nan")
    out = torch.empty(T, d, device="cuda")
    for make in (smr.int8_empty, smr.fp8_empty):
        codes, scales = make(T, d)
        smr.add_rmsnorm(x, eps=1e-6, out=out, codes=codes, scales=scales)
        good = [0, 1, 2, 5]
        check(x[good], None, None, 1e-6, out[good], None, codes[good], scales[good])
        v = codes.float()
        if make is smr.int8_empty:
            assert bool(scales[3:5].isnan().all()) and not bool(v[3:5].any())
        else:
            blk = (d // 2) // 128
            assert bool(scales[3, blk].isnan()) and bool(scales[4].isnan().all())
            assert bool((scales[3].nan_to_num(0.0) == 0).all())  # f is 0 beside an infinity
            assert bool(v[4, (d - 1) // 128 * 128:].isnan().all())
        assert bool(out[3, d // 2].isnan()) and bool(out[4].isnan().all())
        assert int(out[3].isnan().sum()) == 1 and bool((out[3].nan_to_num(0.0) == 0).all())


def test_eps_zero_and_large():
    x = torch.tensor([[3.0, -4.0]], device="cuda")
    out = torch.empty_like(x)
    smr.add_rmsnorm(x, eps=0.0, out=out)
    assert_near(out, x.double() / 12.5 ** 0.5, ROOM)
    smr.add_rmsnorm(x, eps=1e4, out=out)
    assert_near(out, x.double() / (12.5 + float(torch.tensor(1e4))) ** 0.5, ROOM)


def test_codes_feed_the_8_bit_float_product():
    """The e4m3 form is what fp8_matmul takes: its scales are fp32 of any value."""
    g = gen(12)
    T, d, N = 40, 384, 200
    x, r = rows(g, T, d, BF), rows(g, T, d, F)
    codes, scales = smr.fp8_empty(T, d)
    smr.add_rmsnorm(x, r, codes=codes, scales=scales)
    w = torch.randn(N, d, generator=g, device="cuda") * 0.05
    wq, ws = smr.fp8_empty(N, d, 128)
    smr.fp8_quantize(w, wq, ws, block_rows=128)
    out = torch.empty(T, N, device="cuda")
    smr.fp8_matmul(codes, scales, wq, ws, out, smr.fp8_matmul_workspace(T, N, d))
    a = codes.double() * scales.double().repeat_interleave(128, 1)[:, :d]
    b = wq.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :d]
    want = a @ b.T
    # three blocks of fp32 sums: 128 products, three scaled sums, with cancellation
    room = (140 * STEP32) * (a.abs() @ b.abs().T)
    assert bool(((out.double() - want).abs() <= room).all())


def test_graph_and_side_stream():
    g = gen(13)
    x, r = rows(g, 40, 2048, BF), rows(g, 40, 2048, F)
    codes, scales = smr.int8_empty(40, 2048)
    total, out = torch.empty_like(r), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    smr.add_rmsnorm(x, r, out=out, sum_out=total, codes=codes, scales=scales, stream=side)
    side.synchronize()
    check(x, r, None, 1e-6, out, total, codes, scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smr.add_rmsnorm(x, r, out=out, sum_out=total, codes=codes, scales=scales)
    for i in range(3):
        x.copy_(rows(g, 40, 2048, BF))
        graph.replay()
        check(x, r, None, 1e-6, out, total, codes, scales)


def test_large_and_small_numbers():
    """Rows of very large and very small values keep their scale; above 1e19 the sum of squares is infinite and f 0."""
    d = 520
    x = torch.randn(4, d, device="cuda")
    x[0] *= 1e15
    x[1] *= 1e-15
    x[2] *= 1e-30
    out = torch.empty_like(x)
    codes, scales = smr.int8_empty(4, d)
    smr.add_rmsnorm(x, eps=1e-6, out=out, codes=codes, scales=scales)
    check(x, None, None, 1e-6, out, None, codes, scales)
    x[3] = 1e20
    smr.add_rmsnorm(x, eps=1e-6, out=out, codes=codes, scales=scales)
    assert not bool(out[3].any()) and float(scales[3]) == 0.0 and bool((codes[3] == 127).all())


def test_many_rows():
    """More rows than the grid's other dimensions would hold, one warp each."""
    g = gen(16)
    x = rows(g, 300000, 24, BF)
    codes, scales = smr.int8_empty(300000, 24)
    out = torch.empty_like(x)
    smr.add_rmsnorm(x, out=out, codes=codes, scales=scales)
    check(x, None, None, 1e-6, out, None, codes, scales)
