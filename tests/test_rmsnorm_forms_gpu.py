"""The norm and the row quantiser on the GPU where their kernels take another form: very large values, many rows."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr
from test_rmsnorm_gpu import BF, F, check, gen, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(1, 8), (5, 520), (3, 4096), (2, 1001), (2, 12000), (3, 32768), (1300, 512),
                                 (1301, 100)])
@pytest.mark.parametrize("size", [1e16, 2e17, 6e18 / 4.5])
def test_squares_past_the_largest_number(T, d, size):
    """Rows whose squares sum past fp32's largest number are normed all the same, next to ordinary rows. (Values of up
    to 4.5 size, cut there: 6e18 is the bound that the documentation gives.)"""
    g = gen(d + T)
    x = torch.randn(T, d, generator=g, device="cuda").clamp(-4.5, 4.5)
    x[::2] *= size
    residual = torch.randn(T, d, generator=g, device="cuda").clamp(-4.5, 4.5)
    gain = 1 + 0.2 * torch.rand(d, generator=g, device="cuda")
    out, total = torch.empty_like(x), torch.empty_like(x)
    for make in (smr.int8_empty, smr.fp8_empty):
        for r, gn in ((None, None), (residual, gain)):
            codes, scales = make(T, d)
            smr.add_rmsnorm(x, r, gn, 1e-5, out=out, sum_out=total, codes=codes, scales=scales)
            check(x, r, gn, 1e-5, out, total, codes, scales)
            assert bool((scales > 0).all()) and bool(out.any(-1).all())


def test_every_value_at_the_bound():
    """Rows of one value: the documented bound itself, and numbers above it, whose squares overflow one by one."""
    for d in (1, 7, 256, 4100, 32768):
        x = torch.full((2, d), 6e18, device="cuda")
        x[1] = -3e19
        out = torch.empty_like(x)
        codes, scales = smr.int8_empty(2, d)
        smr.add_rmsnorm(x, out=out, codes=codes, scales=scales)
        check(x[:1], None, None, 1e-6, out[:1], None, codes[:1], scales[:1])
        assert not bool(out[1].any()) and float(scales[1]) == 0.0


@pytest.mark.parametrize("T,d", [(4, 96), (3, 4100), (2000, 200)])
def test_eps_zero_where_nothing_is_left_of_the_squares(T, d):
    """0 / 0 is NaN: a row of zeros, and one whose squares are below every fp32 number; their neighbours are as ever."""
    x = torch.randn(T, d, generator=gen(T), device="cuda")
    x[0] = 0.0
    x[1] = 2e-23
    x[1, 3] = 0.0
    out = torch.empty_like(x)
    for make in (smr.int8_empty, smr.fp8_empty):
        codes, scales = make(T, d)
        smr.add_rmsnorm(x, eps=0.0, out=out, codes=codes, scales=scales)
        check(x[2:], None, None, 0.0, out[2:], None, codes[2:], scales[2:])
        assert bool(out[0].isnan().all()) and bool(out[1, 3].isnan()) and int(out[1].isinf().sum()) == d - 1
        assert bool(scales[:2].isinf().all()) and not bool(codes[0].float().any())
        assert bool((codes[1].float() > 0).sum() == d - 1)
