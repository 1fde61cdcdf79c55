"""Refusals of the norm's and of the 8-bit integer calls, on the host, in the C ABI and in the binding: every bad
argument is answered before anything touches a device. Nothing here launches a kernel."""
import ctypes
import os
import random
import subprocess
import sys

import pytest
import torch

import sparse_moe_routing_gb300 as smr
from sparse_moe_routing_gb300 import build as smr_build
from int8_util import CUT_FORMS, FORM_KS, FORMS

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    smr_build.build()
    return smr.lib()


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
X, RES, GAIN, SUM, OUT, CODES, SCALES = 0x1000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000


def norm(L, x=X, residual=RES, gain=GAIN, sum_out=SUM, out=OUT, codes=CODES, scales=SCALES, **kw):
    a = dict(T=4, d=256, x_dtype=smr.BF16, residual_dtype=smr.F32, gain_dtype=smr.BF16, sum_dtype=smr.F32,
             out_dtype=smr.BF16, codes_dtype=smr.I8_ROW, ldx=256, ldr=256, lds=256, ldo=256, ldq=256, eps=1e-6)
    a.update(kw)
    n = smr._RmsNorm(*[a[f] for f, _ in smr._RmsNorm._fields_])
    return L.moe_add_rmsnorm(ctypes.byref(n), x, residual, gain, sum_out, out, codes, scales, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=-3), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x_dtype=2), INVALID), (dict(x_dtype=smr.I8_ROW), INVALID),
    (dict(residual_dtype=3), INVALID), (dict(gain_dtype=9), INVALID), (dict(sum_dtype=-1), INVALID),
    (dict(out_dtype=smr.F8_E4M3_B128), INVALID), (dict(codes_dtype=smr.BF16), INVALID), (dict(codes_dtype=0), INVALID),
    (dict(ldx=255), INVALID), (dict(ldr=255), INVALID), (dict(lds=255), INVALID), (dict(ldo=255), INVALID),
    (dict(ldq=255), INVALID), (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(sum_out=None, out=None, codes=None, scales=None), INVALID),
    (dict(x=X + 1), INVALID), (dict(residual=RES + 2), INVALID), (dict(gain=GAIN + 1), INVALID),
    (dict(sum_out=SUM + 2), INVALID), (dict(out=OUT + 1), INVALID), (dict(scales=SCALES + 2), INVALID),
    # places that may not meet: another type or pitch, both outputs in one, codes in anything
    (dict(sum_out=X), INVALID), (dict(out=RES), INVALID), (dict(out=X, ldo=512), INVALID),
    (dict(sum_out=RES, lds=300), INVALID), (dict(out=SUM, out_dtype=smr.F32), INVALID), (dict(out=GAIN), INVALID),
    (dict(sum_out=GAIN), INVALID), (dict(codes=X), INVALID), (dict(codes=OUT), INVALID), (dict(codes=SCALES), INVALID),
    (dict(scales=RES), INVALID), (dict(scales=SUM), INVALID), (dict(codes=GAIN), INVALID),
    (dict(d=32769, ldx=40000, ldr=40000, lds=40000, ldo=40000, ldq=40000), UNSUPPORTED),
    (dict(T=0), 0), (dict(T=0, x=None, residual=None, gain=None, sum_out=None, out=None, codes=None, scales=None), 0)])
def test_norm_refusals(L, bad, want):
    assert norm(L, **bad) == want


def test_norm_without_a_structure(L):
    assert L.moe_add_rmsnorm(None, X, None, None, None, OUT, None, None, None) == INVALID


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(s=None), INVALID), (dict(x=0x1001), INVALID),
    (dict(dt=smr.F32, x=0x1002), INVALID), (dict(s=0x3002), INVALID), (dict(dt=2), INVALID), (dict(dt=4), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ldx=255), INVALID), (dict(ldq=255), INVALID),
    (dict(codes=0x1000), INVALID), (dict(s=0x1000), INVALID), (dict(s=0x2000), INVALID),
    (dict(cols=32769, ldx=40000, ldq=40000), UNSUPPORTED), (dict(rows=0, x=None, codes=None, s=None), 0)])
def test_quantize_refusals(L, bad, want):
    a = dict(x=0x1000, dt=smr.BF16, ldx=256, rows=4, cols=256, codes=0x2000, ldq=256, s=0x3000)
    a.update(bad)
    assert L.moe_i8_quantize(a["x"], a["dt"], a["ldx"], a["rows"], a["cols"], a["codes"], a["ldq"], a["s"],
                             None) == want


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def mm(**kw):
    a = dict(M=32, N=512, K=256, out_dtype=smr.BF16, gated=0, lda=256, ldb=256, ldo=512, workspace=0x100000,
             workspace_bytes=1 << 40)
    a.update(kw)
    return smr._I8Matmul(*[a[f] for f, _ in smr._I8Matmul._fields_])


def call(L, m, p=(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000)):
    """With a structure of either form: (a, a_scale, b | gate, scale, up, scale, out)."""
    if m.gated:
        return L.moe_i8_gated_matmul(*p[:6], ctypes.byref(m), p[6], None)
    return L.moe_i8_matmul(*p[:4], ctypes.byref(m), p[6], None)


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(out_dtype=3), INVALID),
    (dict(lda=240), INVALID), (dict(lda=264), INVALID), (dict(ldb=248), INVALID), (dict(ldo=511), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=0x100010), WORKSPACE), (dict(workspace_bytes=255), WORKSPACE),
    (dict(lda=1 << 41), UNSUPPORTED), (dict(K=131072, lda=131072, ldb=131072), UNSUPPORTED),
    (dict(N=(1 << 30) + 1, ldo=1 << 31), UNSUPPORTED), (dict(M=1 << 30), UNSUPPORTED), (dict(M=0), 0), (dict(N=0), 0)])
def test_product_refusals(L, gated, bad, want):
    m = mm(gated=gated, **bad)
    assert call(L, m) == want
    if want in (INVALID, UNSUPPORTED):
        assert L.moe_i8_matmul_workspace_bytes(ctypes.byref(m)) == 0
        assert L.moe_i8_matmul_init(ctypes.byref(m), None) == want


@pytest.mark.parametrize("gated", [0, 1])
def test_product_tensors(L, gated):
    good = (0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000)
    m = mm(gated=gated)
    for i in (0, 1, 2, 3, 6) if not gated else range(7):
        for bad in (None, good[i] + 1):
            assert call(L, m, good[:i] + (bad,) + good[i + 1:]) == INVALID, i
    for i in (0, 2) if not gated else (0, 2, 4):
        assert call(L, m, good[:i] + (good[i] + 8,) + good[i + 1:]) == INVALID  # codes lie on 16 bytes
        assert call(L, m, good[:6] + (good[i],)) == INVALID                     # and the result in none of them
        assert call(L, m, good[:6] + (good[i + 1],)) == INVALID
    assert L.moe_i8_matmul(*good[:4], None, good[6], None) == INVALID


def test_the_structure_names_its_call(L):
    p = (0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000)
    assert L.moe_i8_matmul(*p[:4], ctypes.byref(mm(gated=1)), 0x7000, None) == INVALID
    assert L.moe_i8_gated_matmul(*p, ctypes.byref(mm(gated=0)), 0x7000, None) == INVALID
    assert L.moe_i8_matmul(*p[:4], ctypes.byref(mm(gated=2)), 0x7000, None) == INVALID


@pytest.mark.parametrize("gated", [0, 1])
def test_sizes_on_each_side_of_the_limits(L, gated):
    """As the header has them: 2^30 rows or columns, 2^44 values (gated 2^43), 2^40 codes of a."""
    side = 1 << 22 if not gated else 1 << 21
    for M, N, K, good in [
            (131072, 131072, 4096, True), (1048576, 16384, 128, True), (16, (1 << 30) - 1, 64, True),
            ((1 << 30) - 1, 64, 16, True), ((1 << 30) - 1, 64, 1024, True), ((1 << 30) - 1, 64, 1040, False),
            (1 << 30, 1, 1, False), (1, 1 << 30, 1, False), (side, 1 << 22, 128, True), (side + 1, 1 << 22, 128, False),
            (1 << 23, 1, 131071, True), ((1 << 23) + 256, 1, 131071, False)]:
        p = -(-K // 16) * 16
        m = mm(M=M, N=N, K=K, gated=gated, lda=p, ldb=p, ldo=N, workspace_bytes=1 << 50)
        assert (L.moe_i8_matmul_workspace_bytes(ctypes.byref(m)) > 0) == good, (M, N, K)
        assert call(L, m, (None,) * 7) == (INVALID if good else UNSUPPORTED), (M, N, K)  # (tensors are looked at last)


def test_workspace_that_serves_every_number_of_rows(L):
    """What Int8Linear and Int8FeedForward allocate is enough for each product that they run: it grows with the rows
    and with the sums' length and asks for nothing else."""
    rng = random.Random(1)
    for _ in range(60):
        N, K, most = rng.randint(1, 3000), rng.randint(1, 9000), rng.randint(1, 700)
        for gated in (False, True):
            need = max(smr._i8_workspace_bytes(M, N, K, gated) for M in range(1, most + 1))
            assert smr._i8_workspace_bytes(most, N, K, gated) == need, (N, K, most, gated)
            assert need <= smr._i8_workspace_bytes(most, rng.randint(1, 3000), K + rng.randint(0, 500), not gated)


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------
def i8(*s):
    return torch.zeros(s, dtype=torch.int8)


def test_norm_binding_refusals():
    x, ok = torch.zeros(4, 64), torch.zeros(4, 64)
    bf, one = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    for kw, match in [
            (dict(x=torch.zeros(64), out=ok), "two dim"), (dict(x=x.half(), out=ok), "float32 or bfloat16"),
            (dict(x=torch.zeros(64, 4).T, out=ok), "x must have contiguous rows"),
            (dict(x=x, residual=torch.zeros(4, 63), out=ok), "residual has shape"),
            (dict(x=x, residual=ok.double(), out=ok), "float32 or bfloat16"),
            (dict(x=x, gain=torch.ones(63), out=ok), "gain must be"),
            (dict(x=x, gain=torch.ones(1, 64), out=ok), "gain must be"),
            (dict(x=x, gain=torch.ones(128)[::2], out=ok), "gain must be"),
            (dict(x=x, gain=one.half(), out=ok), "float32 or bfloat16"),
            (dict(x=x, out=torch.zeros(3, 64)), "out has shape"), (dict(x=x, sum_out=torch.zeros(4, 65)), "sum_out has shape"),
            (dict(x=x, codes=i8(4, 64)), "belong together"), (dict(x=x, scales=torch.ones(4)), "belong together"),
            (dict(x=x, codes=i8(4, 63), scales=torch.ones(4)), "codes has shape"),
            (dict(x=x, codes=i8(4, 64), scales=torch.ones(4, 1)), "scales has shape"),
            (dict(x=x, codes=i8(4, 64), scales=torch.ones(4).double()), "float32"),
            (dict(x=x, codes=bf, scales=torch.ones(4, 1)), "float8_e4m3fn"),
            (dict(x=x, codes=bf.to(torch.float8_e4m3fn), scales=torch.ones(4)), "scales has shape"),
            (dict(x=x, codes=bf.to(torch.float8_e4m3fn), scales=torch.ones(8, 1)[::2]), "scales must be contiguous")]:
        with pytest.raises(ValueError, match=match):
            smr.add_rmsnorm(**kw)


def test_quantize_binding_refusals():
    x, s = torch.zeros(4, 64), torch.ones(4)
    for args, match in [((torch.zeros(4, 4, 4), i8(4, 64), s), "two dim"), ((x, i8(4, 63), s), "codes has shape"),
                        ((x, x, s), "int8 matrix"), ((x, i8(4, 64), torch.ones(3)), "scales has shape"),
                        ((x, i8(4, 64), s.bfloat16()), "float32"), ((x.half(), i8(4, 64), s), "float32 or bfloat16"),
                        ((x, i8(4, 64), torch.ones(8)[::2]), "scales must be"), ((x, i8(64, 4).T, s), "contiguous rows")]:
        with pytest.raises(ValueError, match=match):
            smr.int8_quantize(*args)


def test_product_binding_refusals():
    a, b, sa, sb, out, ws = i8(4, 64), i8(8, 64), torch.ones(4), torch.ones(8), torch.zeros(4, 8), i8(512)
    for kw, match in [
            (dict(a=a.float()), "a must be an int8"), (dict(b=b.to(torch.uint8)), "b must be an int8"),
            (dict(b=i8(8, 80)[:, :63]), "b has shape"), (dict(b_scale=torch.ones(7)), "b_scale has shape"),
            (dict(a_scale=torch.ones(4, 1)), "a_scale has shape"), (dict(a_scale=torch.ones(4).double()), "float32"),
            (dict(b_scale=torch.ones(16)[::2]), "b_scale must be"), (dict(out=torch.zeros(4, 9)), "out has shape"),
            (dict(out=out.half()), "float32 or bfloat16"), (dict(out=torch.zeros(8, 4).T), "out must have contiguous"),
            (dict(workspace=i8(1024)[::2]), "workspace must be contiguous"),
            (dict(a=i8(64, 4).T), "a must have contiguous")]:
        args = dict(a=a, a_scale=sa, b=b, b_scale=sb, out=out, workspace=ws)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            smr.int8_matmul(**args)
    with pytest.raises(ValueError, match="same row pitch"):
        smr.int8_gated_matmul(a, sa, b, sb, i8(8, 80)[:, :64], sb, out, ws)
    with pytest.raises(ValueError, match="up has shape"):
        smr.int8_gated_matmul(a, sa, b, sb, i8(9, 64), torch.ones(9), out, ws)


@pytest.mark.skipif(torch.cuda.is_available(), reason="what a machine without a GPU answers")
def test_tensors_on_the_host():
    """Good arguments but for their place: the last check refuses them."""
    a, s, out, ws = i8(4, 64), torch.ones(4), torch.zeros(4, 4), i8(512)
    with pytest.raises(RuntimeError, match="CUDA device"):
        smr.int8_matmul(a, s, a, s, out, ws)
    with pytest.raises(RuntimeError, match="CUDA device"):
        smr.add_rmsnorm(torch.zeros(4, 64), out=torch.zeros(4, 64))


def test_feed_forward_shapes():
    w = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="W_up has shape"):
        smr.Int8FeedForward(w(64, 32), w(63, 32), w(32, 64), 4)
    with pytest.raises(ValueError, match="W_down has shape"):
        smr.Int8FeedForward(w(64, 32), w(64, 32), w(64, 32), 4)


def test_every_kernel_is_among_the_tested_shapes(L):
    """The shapes that stand for a kernel in the GPU tests run on it: a change of the choice has to bring others."""
    for M, N, form in FORMS:
        for K in FORM_KS:
            for gated in (False, True):
                assert smr.int8_matmul_form(M, N, K, gated) == form, (M, N, K, gated)
    for M, N, K, gated, form in CUT_FORMS:
        assert smr.int8_matmul_form(M, N, K, gated) == form, (M, N, K, gated)
    assert {f for _, _, f in FORMS} == {0, 16, 32, 64, 128, 256}


def test_form_of_nothing(L):
    assert L.moe_i8_matmul_form(None) == -1 and L.moe_i8_matmul_form(ctypes.byref(mm(K=0))) == -1
    assert smr.int8_matmul_form(0, 5, 5) == smr.int8_matmul_form(8, 5, 5) == smr.int8_matmul_form(9, 0, 5) == 0
    with pytest.raises(smr.MoEError):
        smr.int8_matmul_form(9, 9, 131072)


@pytest.mark.skipif(torch.cuda.is_available(), reason="what a machine without a GPU answers")
@pytest.mark.parametrize("M", [4, 12, 40])
def test_a_failure_of_cuda_has_a_text(M):
    """Every kernel's way to MOE_ERR_CUDA leaves the reason behind. (No call before leaves one: this is a child.)"""
    code = """
import ctypes, sys
sys.path[:0] = ["tests"]
import sparse_moe_routing_gb300 as smr
from test_int8_abi_cpu import call, mm
L = smr.lib()
assert L.moe_last_cuda_error() == b"no error"
assert call(L, mm(M=%d)) == 4 and L.moe_last_cuda_error() != b"no error", L.moe_last_cuda_error()
""" % M
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
