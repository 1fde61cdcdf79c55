"""The 8-bit integer products on the GPU where their form matters: very large results,
values next to the quantiser's borders."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr
from test_int8_gpu import gen, random_codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(131077, 131073), (16, 2 ** 29 + 77)])
def test_results_of_more_than_2_to_the_34_values(M, N):
    """Tiles and places past what 32 bits of values or bytes hold: every value is the sum, which fp32 holds, times two
    powers of two."""
    K = 16
    need = M * N * 2 + (M + N) * (K + 8)
    if torch.cuda.mem_get_info()[0] < need + (30 << 30):
        pytest.skip("needs %d GB" % ((need >> 30) + 30))
    g = gen(M)
    a, b = random_codes(g, M, K), random_codes(g, N, K)
    sa = torch.exp2(torch.randint(-3, 4, (M,), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-3, 4, (N,), generator=g, device="cuda").float())
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    smr.int8_matmul(a, sa, b, sb, out, smr.int8_matmul_workspace(M, N, K))
    rows, cols = (2048, N) if M > 16 else (M, 1 << 24)
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
