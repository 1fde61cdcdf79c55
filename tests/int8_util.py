"""Plain forms of the norm and of the 8-bit integer operators, for the tests."""
import torch

STEP32, STEP_BF16 = 2.0 ** -24, 2.0 ** -8  # half a step, relative


def half_step(dtype):
    return {torch.float32: 0.0, torch.bfloat16: STEP_BF16}[dtype]


def pitched(codes, fill=77):
    """The same codes with rows a multiple of 16 bytes apart; the bytes between hold `fill`."""
    R, C = codes.shape
    room = torch.full((R, -(-C // 16) * 16), fill, dtype=torch.int8, device=codes.device)
    room[:, :C] = codes
    return room[:, :C]


def codes32(t):
    """(codes, scales) of rows t (fp32, CPU) by the definition, each step in fp32."""
    assert t.dtype == torch.float32 and not t.is_cuda
    m = t.abs().amax(-1).clamp(min=127.0 * 2.0 ** -126)
    c = torch.full_like(m, 127.0)
    good = torch.isfinite(t).all(-1)
    inv, scale = c / m, m / c
    codes = torch.where(good[:, None], torch.round(t * inv[:, None]), torch.zeros_like(t))
    return codes.to(torch.int8), torch.where(good, scale, torch.full_like(scale, float("nan")))


def random_codes(g, R, C, lo=-127, hi=127):
    return pitched(torch.randint(lo, hi + 1, (R, C), generator=g, device="cuda", dtype=torch.int8))


def random_scales(g, n, base):
    return base * torch.exp(torch.randn(n, generator=g, device="cuda"))


def sums64(a, b):
    """Exact integer sums a b^T as fp64 (below 2^53)."""
    return a.double() @ b.double().T


def scaled64(a, sa, b, sb):
    return sums64(a, b) * sa.double()[:, None] * sb.double()[None, :]


def silu64(v):
    return v * torch.sigmoid(v)


def assert_near(got, want, rel, absolute=0.0, what=""):
    """|got - want| <= rel |want| + absolute for every value; rel a number or a tensor."""
    off = (got.double() - want).abs()
    room = rel * want.abs() + absolute
    bad = ~(off <= room)
    assert not bool(bad.any()), "%s: %d of %d off; first at %s: %r for %r (room %r)" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]),
        float((room + 0 * want)[bad][0]))


def product_room(dtype):
    """The sum rounded to fp32, two products, one rounding to the result's type."""
    return (3 * STEP32 + half_step(dtype)) * 1.001


def gated_room(g64, dtype):
    """|result| times this: g and u as by product_room in fp32; SiLU's condition is at most 1 + |g| (3 roundings of g);
    __expf is off by 2 + 1.173 |g| units in the last place (2^-23), __fdividef by 2, the sum below it and the last
    product by half a unit each, u by three halves."""
    v = g64.abs()
    halves = 3 * (1 + v) + 2 * (2 + 1.173 * v) + 4 + 1 + 1 + 3
    return (halves * STEP32 + half_step(dtype)) * 1.001


def gated_floor(g64, u64):
    """What a gated result may be off whatever its size: __fdividef(g, y) is 0 for a y = 1 + exp(-g) above 2^126, where the
    quotient is below |g| 2^-126; u multiplies that."""
    return g64.abs() * u64.abs() * 2.0 ** -126


# Rows and columns of products, plain and gated, by the rows of a tile that they take for every K of FORM_KS: each kernel
# that a product can run on, with a few tiles and with several waves of them. K on both sides of 1024, up to which blocks
# of 128 keep their sums in fp32.
FORM_KS = [1023, 1024, 1040, 3000]
FORMS = [(3, 200, 0), (12, 200, 16), (16, 41000, 16), (40, 300, 32), (50, 25000, 64), (100, 30000, 128), (70, 20000, 128),
         (300, 5120, 256), (300, 20000, 256)]
# the same where the few tiles are cut along k over clusters: (M, N, K, gated, rows of a tile)
CUT_FORMS = [(200, 2000, 1024, False, 128), (200, 2000, 10000, True, 128), (200, 2000, 10000, False, 128),
             (257, 2432, 3000, True, 256), (257, 2432, 4096, True, 256), (300, 5120, 1024, True, 256),
             (300, 5120, 4096, True, 256), (600, 9740, 1300, False, 256)]
