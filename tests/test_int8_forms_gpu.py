"""The 8-bit integer products on the GPU where their form matters: very large results."""
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
