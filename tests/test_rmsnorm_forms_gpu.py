"""The norm and the row quantiser on the GPU where their kernels take another form: very large values, many rows."""
import pytest
import torch

import sparse_moe_routing_gb300 as smr
from int8_util import assert_near, codes32
from test_rmsnorm_gpu import BF, F, ROOM, check, gen, rows

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


# ---------------------------------------------------------------------------
# many rows: more than eight an SM, where a row has a warp, or a CTA more pieces a thread
# ---------------------------------------------------------------------------
def many(extra=5):
    return 8 * torch.cuda.get_device_properties(0).multi_processor_count + extra


@pytest.mark.parametrize("kind", ["values", "int8", "e4m3", "all"])
@pytest.mark.parametrize("d", [1, 8, 100, 128, 255, 256, 264, 500, 512, 513, 1024, 2048, 4100, 9000, 16384, 16392])
def test_norm_of_many_rows(d, kind):
    """With and without the residual and the gain; the sum in the residual's type and in the other one."""
    T = many(d % 8)
    look = list(range(T)) if d <= 1024 else [*range(0, T - 9, 17), *range(T - 9, T)]  # (the reference takes its time)
    g = gen(d + len(kind))
    i = (d + len(kind)) % 4
    xt, rt, gt = [(BF, F, BF), (F, BF, F), (BF, BF, F), (F, F, BF)][i]
    x, residual = rows(g, T, d, xt), rows(g, T, d, rt, 3.0)
    gain = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(gt)
    for k, (r, gn) in enumerate(((residual, gain), (None, gain), (residual, None), (None, None))):
        out = torch.empty(T, d, dtype=[BF, F][(i + k) % 2], device="cuda") if kind in ("values", "all") else None
        total = torch.empty(T, d, dtype=[BF, F][k // 2], device="cuda") if kind in ("values", "all") else None
        codes = scales = None
        if kind == "int8" or kind == "all" and k % 2:
            codes, scales = smr.int8_empty(T, d)
        elif kind != "values":
            codes, scales = smr.fp8_empty(T, d)
        smr.add_rmsnorm(x, r, gn, 1e-5, out=out, sum_out=total, codes=codes, scales=scales)
        at = lambda t: t[look] if t is not None else None  # noqa: E731
        check(x[look], at(r), gn, 1e-5, at(out), at(total), at(codes), at(scales))


@pytest.mark.parametrize("d", [96, 511, 512, 2048])
def test_many_rows_in_place_and_their_neighbours(d):
    """The sum in the residual's place and the result in x's, rows inside wider matrices whose rest stays; a row with a
    NaN keeps to itself."""
    g, T = gen(d), many(3)
    xroom, rroom = torch.full((T + 2, d + 24), 5.0, device="cuda"), torch.full((T + 2, d + 24), 6.0, device="cuda")
    for c0 in (8, 3):
        x, r = rows(g, T, d, F), rows(g, T, d, F)
        x[7, d // 2] = float("nan")
        a, b = xroom[1:T + 1, c0:c0 + d], rroom[1:T + 1, c0:c0 + d]
        a.copy_(x)
        b.copy_(r)
        codes, scales = smr.int8_empty(T, d)
        smr.add_rmsnorm(a, b, out=a, sum_out=b, codes=codes, scales=scales)
        keep = [i for i in range(T) if i != 7]
        check(x[keep], r[keep], None, 1e-6, a[keep], b[keep], codes[keep], scales[keep])
        assert bool(a[7].isnan().all()) and bool(scales[7].isnan()) and not bool(codes[7].any())
        a.fill_(5.0)
        b.fill_(6.0)
        assert bool((xroom == 5.0).all()) and bool((rroom == 6.0).all())


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("cols", [1, 8, 100, 255, 256, 300, 512, 513, 768, 1000, 1024, 1025, 1032, 2048, 2049, 4096, 4104,
                                  16384, 16392])
def test_quantize_many_rows(cols, dtype):
    """Bit for bit those of the definition, in aligned rows and in rows one value on, with special rows among them."""
    g, T = gen(cols), many(cols % 8)
    room = rows(g, T, cols + 1, dtype)
    for x in (room[:, :cols].contiguous(), room[:, 1:]):
        x[3] = 0.0
        x[T - 2, cols - 1] = float("nan")
        x[T - 3, cols // 2] = float("-inf")
        codes, scales = smr.int8_empty(T, cols)
        smr.int8_quantize(x, codes, scales)
        want, s = codes32(x.float().cpu())
        assert torch.equal(codes.cpu(), want)
        good, got = ~s.isnan(), scales.cpu()
        assert int(good.sum()) == T - 2 and torch.equal(got[good], s[good]) and bool(got[~good].isnan().all())


@pytest.mark.parametrize("d", [300, 512, 4096, 9000])
def test_a_rows_codes_and_sum_do_not_depend_on_the_others(d):
    """Alone or among many, a row's codes and sum are the same bits; its values and scales are near."""
    T = many()
    g = gen(d)
    x, r = rows(g, T, d, BF), rows(g, T, d, F)
    for make in (smr.int8_empty, smr.fp8_empty):
        whole, wscales = make(T, d)
        wsum = torch.empty_like(r)
        smr.add_rmsnorm(x, r, sum_out=wsum, codes=whole, scales=wscales)
        for r0, r1 in ((0, 1), (T - 7, T)):
            codes, scales = make(r1 - r0, d)
            total = torch.empty_like(r[r0:r1])
            smr.add_rmsnorm(x[r0:r1], r[r0:r1], sum_out=total, codes=codes, scales=scales)
            assert torch.equal(codes.float(), whole[r0:r1].float()) and torch.equal(total, wsum[r0:r1])
            assert_near(scales, wscales[r0:r1].double(), 2 * ROOM)
