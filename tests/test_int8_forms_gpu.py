"""The 8-bit integer products on the GPU where their form matters: sums at the ends of what it holds and rows' equality
on every kernel, gates far from zero, very large results, values next to the quantiser's borders."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr
from int8_util import (CUT_FORMS, FORM_KS, FORMS, assert_near, gated_floor, gated_room, pitched, random_codes,
                       random_scales, scaled64, silu64, sums64)
from test_int8_gpu import gen, product, status

pytestmark = pytest.mark.gpu


SHAPES = [(M, N, K) for M, N, _ in FORMS for K in FORM_KS]
CUT = [c[:4] for c in CUT_FORMS]


def codes_at_the_ends(g, M, N, K):
    """Codes of one sign and nearly all at their ends: sums of up to 2^14 K, odd and even, of either sign."""
    a = pitched(torch.full((M, K), -128, dtype=torch.int8, device="cuda"))
    b = pitched(torch.full((N, K), -128, dtype=torch.int8, device="cuda"))
    a += (torch.rand(M, K, generator=g, device="cuda") < 0.01).to(torch.int8)
    b += (torch.rand(N, K, generator=g, device="cuda") < 0.003).to(torch.int8)
    a[0] = b[0] = -128  # and the largest sum itself
    b[N // 2:] = torch.where(b[N // 2:] == -128, 127, -127).to(torch.int8)
    return a, b


@pytest.mark.parametrize("M,N,K", SHAPES + [c[:3] for c in CUT if not c[3]])
def test_sums_at_the_ends(M, N, K):
    """Scales of one: the result is the sum rounded to fp32, and any lost unit of it shows."""
    g = gen(K + M)
    a, b = codes_at_the_ends(g, M, N, K)
    one = torch.ones(max(M, N), device="cuda")
    got = product(a, one[:M], [(b, one[:N])], torch.float32)
    want = sums64(a, b)
    assert float(want[0, 0]) == K * 2.0 ** 14
    assert torch.equal(got, want.to(torch.float32))


@pytest.mark.parametrize("block", [64, 128, 256, 512, 1024])
@pytest.mark.parametrize("M,N", [(M, N) for M, N, _ in FORMS if N < 10000 or M == 100])
def test_sums_that_cancel(M, N, block):
    """Stretches of one sign and of the other in turn, which leave a few units: within a step of 128, between the steps of
    two issuers, within one accumulator and between its reads."""
    g = gen(block + M)
    for K in (1024, 4096):
        sign = 1 - 2 * ((torch.arange(K, device="cuda") // block) % 2)
        a = (127 * sign).to(torch.int8).repeat(M, 1).contiguous()
        b = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
        b -= (torch.rand(N, K, generator=g, device="cuda") < 0.002).to(torch.int8)
        one = torch.ones(max(M, N), device="cuda")
        got = product(a, one[:M], [(b, one[:N])], torch.float32)
        want = sums64(a, b)
        if block < K:
            assert want.abs().max() < 10000
        assert torch.equal(got, want.to(torch.float32)), K


@pytest.mark.parametrize("M,N,K,gated", [(M, N, K, gated) for M, N, K in SHAPES if M > 16 and K != 1023
                                         for gated in (False, True)] + CUT)
def test_a_row_is_the_same_on_every_kernel(M, N, K, gated):
    """Rows of a product against the same rows by themselves, on the kernels for up to 8 and up to 16 rows, bit for bit; a
    gated result also against its definition."""
    g = gen(M + N + K)
    a, sa = random_codes(g, M, K, -128), random_scales(g, M, 0.02)
    w = [(random_codes(g, N, K, -128), random_scales(g, N, 0.01 / K ** 0.5)) for _ in range(1 + gated)]
    ws = smr.int8_matmul_workspace(M, N, K, gated=gated)
    whole = product(a, sa, w, torch.float32, ws)
    for r0, r1 in ((0, 1), (M // 2, M // 2 + 8), (M - 13, M), (128 % M, min(128 % M + 16, M))):
        assert torch.equal(product(a[r0:r1], sa[r0:r1], w, torch.float32, ws), whole[r0:r1]), (r0, r1)
    assert torch.equal(product(a, sa, w, torch.bfloat16, ws), whole.to(torch.bfloat16))
    if gated:
        first, second = scaled64(a, sa, *w[0]), scaled64(a, sa, *w[1])
        assert_near(whole, silu64(first) * second, gated_room(first, torch.float32), gated_floor(first, second))
    assert status(ws) == (0, 0)


@pytest.mark.parametrize("M", [1, 5, 12, 40, 300])
def test_gates_of_every_size(M):
    """Gates from -130 to 130 in the documented distance, fp32 results: the fast exponential's error grows with the gate,
    and below -87 its quotient may be 0."""
    N, K = 1000, 1
    steps = torch.arange(N, device="cuda")
    a = pitched(torch.full((M, K), 127, dtype=torch.int8, device="cuda"))
    gate = pitched((steps % 255 - 127).to(torch.int8)[:, None])
    up = pitched(torch.full((N, K), 101, dtype=torch.int8, device="cuda"))
    sa = torch.linspace(1e-3, 130 / 127, M, device="cuda") if M > 1 else torch.ones(1, device="cuda")
    sg, su = 1 / 127 * (0.9 + 0.1 * torch.rand(N, generator=gen(M), device="cuda")), torch.ones(N, device="cuda") / 101
    got = product(a, sa, [(gate, sg), (up, su)], torch.float32)
    first, second = scaled64(a, sa, gate, sg), scaled64(a, sa, up, su)
    assert_near(got, silu64(first) * second, (8 + 2.7 * first.abs()) * 2.0 ** -23, gated_floor(first, second))
    assert float(first.min()) < -100


@pytest.mark.parametrize("M,N", [(131077, 131073), (16, 2 ** 29 + 77), (2 ** 30 - 1, 3)])
def test_the_largest_results(M, N):
    """More than 2^34 values, and as many rows as there may be: tiles and places past what 32 bits of values or bytes
    hold. Every value is the sum, which fp32 holds, times two powers of two."""
    K = 16
    need = M * N * 2 + (M + N) * (K + 8) + M * K * 2
    if torch.cuda.mem_get_info()[0] < need + (30 << 30):
        pytest.skip("needs %d GB" % ((need >> 30) + 30))
    g = gen(M)
    a, b = random_codes(g, M, K), random_codes(g, N, K)
    sa = torch.exp2(torch.randint(-3, 4, (M,), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-3, 4, (N,), generator=g, device="cuda").float())
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    smr.int8_matmul(a, sa, b, sb, out, smr.int8_matmul_workspace(M, N, K))
    rows, cols = (max(16, (1 << 28) // N), min(N, 1 << 24))
    for i in range(0, M, rows):
        for j in range(0, N, cols):
            want = (a[i:i + rows].float() * sa[i:i + rows, None]) @ (b[j:j + cols].float() * sb[j:j + cols, None]).T
            assert torch.equal(out[i:i + rows, j:j + cols], want.to(torch.bfloat16)), (i, j)


def test_codes_are_within_the_documented_distance():
    """Values next to the borders between two codes, where the distance is largest: half a step of the scale and three
    roundings (127 / m, its product with the value, m / 127) of 2^-24, relative, of up to 127 steps: 0.5 + 2.3e-5."""
    g = gen(21)
    m = torch.exp(20 * (torch.rand(400, 1, generator=g, device="cuda") - 0.5))
    k = torch.randint(100, 127, (400, 2000), generator=g, device="cuda")
    x = (m.double() * (k + 0.5) / 127).float()
    x = torch.cat([m, x, torch.nextafter(x, 0 * x), torch.nextafter(x, 2 * m.expand_as(x))], 1)
    codes, scales = smr.int8_empty(*x.shape)
    smr.int8_quantize(x, codes, scales)
    off = ((codes.double() * scales.double()[:, None] - x.double()).abs() / scales.double()[:, None]).max()
    assert 0.5000001 < float(off) <= 0.50003, float(off)
