"""8-bit integer products and quantiser on the GPU against exact integer sums in fp64."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_moe_routing_gb300 as smr
from int8_util import (STEP32, assert_near, codes32, gated_floor, gated_room, half_step, pitched, product_room,
                       random_codes, random_scales, scaled64, silu64, sums64)

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def product(a, sa, weights, dtype, ws=None, out=None, stream=None):
    M, K = a.shape
    N = weights[0][0].shape[0]
    gated = len(weights) == 2
    ws = smr.int8_matmul_workspace(M, N, K, gated=gated) if ws is None else ws
    out = torch.empty(M, N, dtype=dtype, device="cuda") if out is None else out
    call = smr.int8_gated_matmul if gated else smr.int8_matmul
    call(a, sa, *(t for w in weights for t in w), out, ws, stream=stream)
    return out


def status(ws):
    return smr.read_device_status(smr.MoEConfig(T=1, d_model=128, n_experts=1, top_k=1, d_ff=128), ws)


def check_product(M, N, K, gated, dtype, seed=0, lo=-127, hi=127):
    g = gen(1000 * seed + M + 7 * N + 13 * K)
    a, sa = random_codes(g, M, K, lo, hi), random_scales(g, M, 0.02)
    # the gate's products of the size of a few units, where SiLU bends
    w = [(random_codes(g, N, K, lo, hi), random_scales(g, N, 0.01 / max(K, 1) ** 0.5)) for _ in range(1 + gated)]
    got = product(a, sa, w, dtype)
    first = scaled64(a, sa, *w[0])
    if not gated:
        assert_near(got, first, product_room(dtype), what="product %s" % ((M, N, K),))
    else:
        second = scaled64(a, sa, *w[1])
        assert_near(got, silu64(first) * second, gated_room(first, dtype), gated_floor(first, second),
                    "gated %s" % ((M, N, K),))


# one to eight rows stream, more run on the tensor cores: 16, 32, 64 and 128 rows a block, two blocks a tile
# where there are tiles enough (257 x 19400); few tiles are cut along k over clusters, several waves of tiles with
# steps odd in number share the rings (100 x 30000 x 333), and a last wave may be cut behind whole ones
SHAPES = [(1, 1, 1), (1, 16, 16), (3, 17, 63), (8, 128, 64), (8, 130, 1000), (7, 4096, 4097), (2, 33, 14336),
          (9, 1, 1), (9, 128, 128), (16, 129, 127), (17, 1000, 1024), (33, 255, 1025), (64, 4096, 2048),
          (65, 300, 300), (128, 128, 4096), (129, 640, 129), (333, 1001, 1400), (257, 19400, 513),
          (1024, 2561, 1111), (700, 9800, 1100), (100, 30000, 333), (16, 41000, 600), (50, 25000, 4096),
          (20, 12300, 4200), (200, 2000, 10000), (128, 5632, 2048), (600, 9740, 1300), (600, 5000, 700)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, gated, dtype):
    check_product(M, N, K, gated, dtype)


@pytest.mark.parametrize("M", [3, 12, 130, 300])
@pytest.mark.parametrize("K", [1023, 1024, 1040, 3000, 131071])
def test_sums_are_exact_at_the_largest_codes(M, K):
    """Codes of one sign and nearly all at their ends: sums up to 2^31 - 2^14, odd and even, in which a single lost unit
    of any 1024 products would show. Scales of one: the result is the sum rounded to fp32."""
    g = gen(K + M)
    N = 200
    a = pitched(torch.full((M, K), -128, dtype=torch.int8, device="cuda"))
    b = pitched(torch.full((N, K), -128, dtype=torch.int8, device="cuda"))
    a += (torch.rand(M, K, generator=g, device="cuda") < 0.01).to(torch.int8)
    b += (torch.rand(N, K, generator=g, device="cuda") < 0.003).to(torch.int8)
    b[N // 2:] = torch.where(b[N // 2:] == -128, 127, -127).to(torch.int8)  # and sums of the other sign
    one = torch.ones(max(M, N), device="cuda")
    got = product(a, one[:M], [(b, one[:N])], torch.float32)
    assert torch.equal(got, sums64(a, b).to(torch.float32))


def test_sums_are_exact_where_they_cancel():
    """Chunks of 1024 products near +2^24 and -2^24 in turn that leave a few units."""
    g = gen(5)
    M, N, K = 40, 150, 4096
    sign = torch.tensor([1, -1, 1, -1], device="cuda", dtype=torch.int8).repeat_interleave(1024)
    a = (127 * sign).repeat(M, 1).contiguous()
    b = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    b -= (torch.rand(N, K, generator=g, device="cuda") < 0.002).to(torch.int8)
    one = torch.ones(N, device="cuda")
    got = product(a, one[:M], [(b, one)], torch.float32)
    want = sums64(a, b)
    assert want.abs().max() < 10000 and torch.equal(got, want.to(torch.float32))


def test_rows_are_the_same_whatever_their_number():
    """A row's result does not depend on the other rows nor on the kernel that runs."""
    g = gen(3)
    N, K = 700, 1500
    a, sa = random_codes(g, 400, K), random_scales(g, 400, 0.02)
    w = [(random_codes(g, N, K), random_scales(g, N, 0.001)) for _ in range(2)]
    for use in (w[:1], w):
        whole = product(a, sa, use, torch.float32)
        for M in (1, 8, 9, 17, 64, 128, 257):
            assert torch.equal(product(a[:M], sa[:M], use, torch.float32), whole[:M]), M


@pytest.mark.parametrize("M", [5, 20, 200])
def test_pitches_and_what_lies_around(M):
    """Rows inside wider matrices: bytes between a row's codes change nothing, values around the result stay."""
    g = gen(4)
    N, K = 333, 200
    a, b = random_codes(g, M, 2 * K, -128), random_codes(g, N, 3 * K + 8, -128)
    sa, sb = random_scales(g, M, 0.02), random_scales(g, N, 0.001)
    room = torch.full((M + 2, N + 11), 7.0, device="cuda")
    out = room[1:M + 1, 3:N + 3]
    product(a[:, :K], sa, [(b[:, 16:16 + K], sb)], torch.float32, out=out)
    assert_near(out, scaled64(a[:, :K], sa, b[:, 16:16 + K], sb), product_room(torch.float32))
    room[1:M + 1, 3:N + 3] = 7.0
    assert bool((room == 7.0).all())


def test_scales_of_zero_nan_and_infinity_stay_in_their_rows_and_columns():
    g = gen(6)
    for M in (4, 40):
        a, sa = random_codes(g, M, 300), random_scales(g, M, 0.02)
        b, sb = random_codes(g, 200, 300), random_scales(g, 200, 0.001)
        sa[1], sa[2], sb[7] = float("nan"), 0.0, float("inf")
        got = product(a, sa, [(b, sb)], torch.float32)
        assert bool(got[1].isnan().all()) and bool((got[2, :7] == 0).all()) and bool(got[2, 7].isnan())
        keep = [i for i in range(M) if i not in (1, 2)]
        cols = [j for j in range(200) if j != 7]
        assert bool(got[keep][:, cols].isfinite().all()) and bool((~got[keep][:, 7].isfinite()).all())


def test_one_row_needs_no_pitch():
    """A single row of any length, whatever its tensor's strides say."""
    g = gen(14)
    K = 1001
    a, w = (random_codes(g, 1, K)[0].clone().view(1, K) for _ in range(2))
    assert a.stride(0) == K
    one = torch.ones(1, device="cuda")
    got = product(a, one, [(w, one)], torch.float32)
    assert torch.equal(got, sums64(a, w).to(torch.float32))
    b = random_codes(g, 40, K)
    got = product(a, one, [(b, torch.ones(40, device="cuda"))], torch.float32)
    assert torch.equal(got, sums64(a, b).to(torch.float32))


def test_nothing_to_do():
    one = torch.ones(4, device="cuda")
    ws = smr.int8_matmul_workspace(64, 64, 64)
    codes = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    n = smr.launch_count()
    smr.int8_matmul(codes[:0], one[:0], codes, one, torch.empty(0, 4, device="cuda"), ws)
    smr.int8_matmul(codes, one, codes[:0], one[:0], torch.empty(4, 0, device="cuda"), ws)
    smr.int8_quantize(torch.zeros(0, 64, device="cuda"), codes[:0], one[:0])
    smr.add_rmsnorm(torch.zeros(0, 64, device="cuda"), out=torch.empty(0, 64, device="cuda"))
    assert smr.launch_count() == n


def test_one_workspace_for_many_products():
    """The largest of several products' workspaces serves them all, one after the other, with nothing left behind."""
    g = gen(8)
    shapes = [(200, 300, 4000, False), (17, 129, 9000, True), (64, 4096, 700, False), (9, 64, 64, True)]
    ws = max((smr.int8_matmul_workspace(M, N, K, gated=two) for M, N, K, two in shapes), key=lambda t: t.numel())
    for M, N, K, two in shapes * 2:
        a, sa = random_codes(g, M, K), random_scales(g, M, 0.02)
        w = [(random_codes(g, N, K), random_scales(g, N, 0.001)) for _ in range(1 + two)]
        out = product(a, sa, w, torch.float32, ws)
        first = scaled64(a, sa, *w[0])
        if two:
            second = scaled64(a, sa, *w[1])
            assert_near(out, silu64(first) * second, gated_room(first, torch.float32), gated_floor(first, second))
        else:
            assert_near(out, first, product_room(torch.float32))
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("M,N,K", [(4, 500, 700), (40, 500, 4096), (300, 5000, 700)])
def test_graph_and_side_stream(M, N, K):
    """Captured once and replayed on new codes, on a stream of its own; and called with stream=."""
    g = gen(9)
    a, sa = random_codes(g, M, K), random_scales(g, M, 0.02)
    w = [(random_codes(g, N, K), random_scales(g, N, 0.001)) for _ in range(2)]
    ws = smr.int8_matmul_workspace(M, N, K, gated=True)
    out = torch.empty(M, N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    product(a, sa, w, torch.float32, ws, out, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        product(a, sa, w, torch.float32, ws, out)
    for i in range(3):
        a.copy_(random_codes(g, M, K))
        out.zero_()
        graph.replay()
        first, second = scaled64(a, sa, *w[0]), scaled64(a, sa, *w[1])
        assert_near(out, silu64(first) * second, gated_room(first, torch.float32), gated_floor(first, second))
        again = out.clone()
        graph.replay()
        assert torch.equal(out, again)


def test_two_streams_with_a_workspace_each():
    """Products that overlap on the GPU, each with a workspace of its own."""
    g = gen(15)
    cases = []
    for M, N, K in ((40, 3000, 4096), (300, 5000, 900), (5, 4000, 4096), (130, 700, 6000)):
        a, sa = random_codes(g, M, K), random_scales(g, M, 0.02)
        w = [(random_codes(g, N, K), random_scales(g, N, 0.001))]
        cases.append((a, sa, w, smr.int8_matmul_workspace(M, N, K), torch.empty(M, N, device="cuda")))
    want = [product(a, sa, w, torch.float32, ws) for a, sa, w, ws, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (a, sa, w, ws, out) in zip(streams, cases):
            product(a, sa, w, torch.float32, ws, out, stream=st)
    torch.cuda.synchronize()
    for y, (*_, ws, out) in zip(want, cases):
        assert torch.equal(out, y) and status(ws) == (0, 0)


def test_captured_first():
    """A graph whose capture is the first call of its kernels in the process (a child)."""
    code = """
import torch, sparse_moe_routing_gb300 as smr
torch.manual_seed(1)
graphs = []
for M, N, K, gated in ((4, 64, 512, False), (12, 300, 4096, True), (200, 900, 4096, False), (300, 20000, 256, True)):
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    w = [torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda") for _ in range(1 + gated)]
    sa, sb = torch.full((M,), 1e-3, device="cuda"), torch.full((N,), 1e-3, device="cuda")
    out = torch.zeros(M, N, device="cuda")
    x = torch.randn(M, K, device="cuda")
    q, qs = smr.int8_empty(M, K)
    ws = smr.int8_matmul_workspace(M, N, K, gated=gated)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    def calls():
        smr.add_rmsnorm(x, codes=q, scales=qs)
        if gated:
            smr.int8_gated_matmul(a, sa, w[0], sb, w[1], sb, out, ws)
        else:
            smr.int8_matmul(a, sa, w[0], sb, out, ws)
    with torch.cuda.graph(graph):
        calls()
    graph.replay()
    torch.cuda.synchronize()
    first, fq = out.clone(), q.clone()
    out.zero_(); q.zero_()
    calls()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(q, fq) and bool(first.any()) and bool(fq.any())
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240, cwd=root)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_tensors_elsewhere_are_refused():
    one = torch.ones(4, device="cuda")
    codes = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    ws = smr.int8_matmul_workspace(4, 4, 64)
    out = torch.empty(4, 4, device="cuda")
    for bad in (dict(a=codes.cpu()), dict(a_scale=one.cpu()), dict(b=codes.cpu()), dict(b_scale=one.cpu()),
                dict(out=out.cpu()), dict(workspace=ws.cpu())):
        args = dict(a=codes, a_scale=one, b=codes, b_scale=one, out=out, workspace=ws)
        args.update(bad)
        with pytest.raises(ValueError, match="current CUDA device"):
            smr.int8_matmul(**args)
    with pytest.raises(ValueError, match="gain must be on"):
        smr.add_rmsnorm(torch.zeros(4, 64, device="cuda"), gain=torch.ones(64), out=torch.zeros(4, 64, device="cuda"))
    with pytest.raises(smr.MoEError):  # codes off 16 bytes
        smr.int8_matmul(torch.zeros(4, 72, dtype=torch.int8, device="cuda")[:, 8:], one, codes, one, out, ws)


def test_small_workspaces_are_refused():
    a = torch.zeros(100, 256, dtype=torch.int8, device="cuda")
    one, out = torch.ones(100, device="cuda"), torch.empty(100, 100, device="cuda")
    ws = smr.int8_matmul_workspace(16, 100, 256)
    with pytest.raises(smr.MoEError, match="WORKSPACE"):
        smr.int8_matmul(a, one, a, one, out, ws)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(40, 500, 4096), (300, 20000, 300), (12, 700, 4096)])
def test_a_wait_that_runs_out(M, N, K, gated):
    """A stalled launch reports a timeout and returns; the next call on the same workspace is right."""
    g = gen(10)
    a, sa = random_codes(g, M, K), random_scales(g, M, 0.02)
    w = [(random_codes(g, N, K), random_scales(g, N, 0.001)) for _ in range(1 + gated)]
    ws = smr.int8_matmul_workspace(M, N, K, gated=gated)
    want = product(a, sa, w, torch.float32, ws)
    smr.inject_stall("i8_matmul", 2000)
    product(a, sa, w, torch.float32, ws)
    st, word = status(ws)
    assert smr.status_string(st).startswith("MOE_ERR_DEVICE_TIMEOUT") and word >> 16 == 12, (st, hex(word))
    assert torch.equal(product(a, sa, w, torch.float32, ws), want)
    assert status(ws) == (0, 0)


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------
def rows_of_all_sizes(g, rows, cols, dtype):
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (x * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (5, 8), (9, 255), (3, 256), (17, 513), (8, 1024), (3, 1025),
                                       (2, 2048), (401, 2056), (5, 4096), (400, 5001), (2, 8192), (310, 8192),
                                       (3, 14336), (400, 16384), (2, 16385), (2, 16392), (3, 32768)])
def test_quantize(rows, cols, dtype):
    """Codes and scales are those of the definition, bit for bit, and stand for values half a step off at most."""
    g = gen(rows + cols)
    x = rows_of_all_sizes(g, rows, cols, dtype)
    codes, scales = smr.int8_empty(rows, cols)
    smr.int8_quantize(x, codes, scales)
    want, s = codes32(x.float().cpu())
    assert torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), s)
    back = codes.double() * scales.double()[:, None]
    # the factor 127 / m, its product with the value and m / 127 are rounded once each, at most 127.5 steps
    # of 2^-24 each from the exact quotient
    assert_near(back, x.double(), 0.0, (0.5 + 3 * 127.5 * STEP32) * scales.double()[:, None])


def test_quantize_views_and_neighbours():
    """Rows inside wider matrices at odd places: what lies around the codes stays."""
    g = gen(11)
    x = rows_of_all_sizes(g, 20, 700, torch.bfloat16)
    for c0, cols in ((0, 512), (8, 512), (1, 512), (3, 301)):
        room = torch.full((22, 640), 99, dtype=torch.int8, device="cuda")
        part, codes = x[:, c0:c0 + cols], room[1:21, 5:5 + cols]
        scales = torch.empty(20, device="cuda")
        smr.int8_quantize(part, codes, scales)
        want, s = codes32(part.float().cpu())
        assert torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), s)
        room[1:21, 5:5 + cols] = 99
        assert bool((room == 99).all())


@pytest.mark.parametrize("cols", [64, 100, 3000, 20000])
def test_quantize_special_rows(cols):
    """Zeros, the smallest and the largest numbers, ties; an infinity or a NaN spoils its own row alone."""
    big = torch.finfo(torch.float32).max
    x = torch.zeros(9, cols)
    x[1, 3] = 2.0 ** -149
    x[2, :] = 1e-41
    x[3, 0], x[3, 1] = big, -big
    x[4, 0], x[4, 1:50] = 127.0, torch.arange(49) - 24.5  # ties, to even
    x[5, 5] = float("inf")
    x[6, cols - 1] = float("nan")
    x[7, :] = -1.0
    x[8, 0] = 127.0 * 2.0 ** -126
    codes, scales = smr.int8_empty(9, cols)
    smr.int8_quantize(x.cuda(), codes, scales)
    want, s = codes32(x)
    assert torch.equal(codes.cpu(), want)
    assert torch.equal(scales.cpu()[[0, 1, 2, 3, 4, 7, 8]], s[[0, 1, 2, 3, 4, 7, 8]])
    assert bool(scales[5:7].isnan().all()) and not bool(codes[0].any()) and not bool(codes[5:7].any())


# ---------------------------------------------------------------------------
# projections and the feed-forward block
# ---------------------------------------------------------------------------
def linear64(x, w):
    """The value of x through a weight in 8 bits, both quantised by the definition, in fp64; its codes and scales."""
    xq, xs = codes32(x.float().cpu())
    wq, ws = codes32(w.float().cpu())
    return scaled64(xq, xs, wq, ws)


@pytest.mark.parametrize("rows", [1, 8, 100])
def test_linear(rows):
    g = gen(rows)
    w = (torch.randn(301, 500, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    x = torch.randn(rows, 500, generator=g, device="cuda")
    lin = smr.Int8Linear(w, 100)
    y = lin(x, torch.empty(rows, 301, device="cuda"))
    assert_near(y.cpu(), linear64(x, w), product_room(torch.float32))
    q = smr.int8_empty(rows, 500)
    smr.int8_quantize(x, *q)
    assert torch.equal(lin(q, torch.empty(rows, 301, device="cuda")), y)
    assert lin.device_status() == (0, 0)
    small = smr.Int8Linear(w, 4)  # (whose workspace holds the control block alone)
    if rows <= 4:
        assert torch.equal(small(x, torch.empty(rows, 301, device="cuda")), y)
    assert small.device_status() == (0, 0)
    with pytest.raises(ValueError, match="made for"):
        lin(torch.zeros(101, 500, device="cuda"), torch.empty(101, 301, device="cuda"))


@pytest.mark.parametrize("rows", [1, 6, 64, 200])
def test_norm_feed_forward_norm_experts(rows):
    """A dense layer's second half and the norm in front of an expert layer: norm to int8, the feed-forward block on
    the codes, the residual's addition with the next norm, and the layer on its result. Each step is checked against
    its definition on the inputs that the step got."""
    g = gen(20 + rows)
    d, I, E, k, width = 256, 640, 16, 4, 64
    mat = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.05).to(torch.bfloat16)  # noqa: E731
    Wg, Wu, Wd = mat(I, d), mat(I, d), mat(d, I)
    gain = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    attn, residual = mat(rows, d) * 10, 3 * torch.randn(rows, d, generator=g, device="cuda")
    ffn = smr.Int8FeedForward(Wg, Wu, Wd, 200)
    codes, scales = smr.int8_empty(rows, d)
    before = residual.clone()
    smr.add_rmsnorm(attn, residual, gain, codes=codes, scales=scales, sum_out=residual)
    assert torch.equal(residual, before + attn.float())
    t = (residual.cpu() * gain.float().cpu())
    want, s = codes32(t)
    f = 1 / torch.sqrt(residual.double().cpu().square().mean(-1) + 1e-6)
    assert torch.equal(codes.cpu(), want)
    assert_near(scales.cpu(), s.double() * f, 32 * STEP32)

    y = ffn((codes, scales), torch.empty(rows, d, device="cuda"))
    q = lambda w: codes32(w.float().cpu())  # noqa: E731
    xq, xs = codes.cpu(), scales.cpu()
    g64, u64 = scaled64(xq, xs, *q(Wg)), scaled64(xq, xs, *q(Wu))
    assert_near(ffn.h[:rows].cpu(), silu64(g64) * u64, gated_room(g64, torch.bfloat16), gated_floor(g64, u64))
    hq, hs = codes32(ffn.h[:rows].float().cpu())
    assert torch.equal(ffn.hq[:rows].cpu(), hq)
    assert_near(y.cpu(), scaled64(hq, hs, *q(Wd)), product_room(torch.float32))
    assert torch.equal(ffn((codes, scales), torch.empty(rows, d, device="cuda")), y)

    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    kept = residual.clone()
    smr.add_rmsnorm(y, residual, gain, out=x, sum_out=residual)
    assert torch.equal(residual, kept + y)
    s64 = residual.double()
    want = s64 * gain.double() / torch.sqrt(s64.square().mean(-1, keepdim=True) + 1e-6)
    assert_near(x, want, 32 * STEP32 + half_step(torch.bfloat16))
    layer = smr.MoELayer(smr.MoEConfig(T=rows, d_model=d, n_experts=E, top_k=k, d_ff=width), {
        "W_router": mat(E, d), "W_gate": mat(E, width, d), "W_up": mat(E, width, d), "W_down": mat(E, d, width)})
    out, ids, alpha = layer.forward(x, residual)
    w = layer.w
    ref = residual.double()
    for slot in range(k):
        e = ids[:, slot].long()
        gt = torch.einsum("td,tid->ti", x.double(), w["W_gate"][e].double())
        up = torch.einsum("td,tid->ti", x.double(), w["W_up"][e].double())
        ref = ref + alpha[:, slot:slot + 1].double() * torch.einsum("ti,tdi->td", silu64(gt) * up, w["W_down"][e].double())
    # the layer rounds h and its pairs' rows to bf16: as its own parity tests
    assert float((out.double() - ref).abs().max()) <= 2e-2 * float(ref.square().mean().sqrt())
    assert layer.device_status() == (0, 0) and ffn.device_status() == (0, 0)
