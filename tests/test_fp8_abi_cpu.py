"""Refusals of the 8-bit entry points, on the host: every bad argument is
answered before anything touches a device. Nothing here launches a kernel."""
import ctypes

import pytest
import torch

import sparse_moe_routing_gb300 as smr
from sparse_moe_routing_gb300 import build as smr_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    smr_build.build()
    return smr.lib()


def quantize(L, **kw):
    a = dict(x=0x1000, dt=smr.BF16, ldx=256, count=1, rows=4, cols=256, br=1, codes=0x2000, ldq=256, s=0x3000)
    a.update(kw)
    return L.moe_fp8_quantize(a["x"], a["dt"], a["ldx"], a["count"], a["rows"], a["cols"], a["br"],
                              a["codes"], a["ldq"], a["s"], None)


@pytest.mark.parametrize("bad,want", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(s=None), INVALID),
    (dict(x=0x1001), INVALID), (dict(dt=smr.F32, x=0x1002), INVALID), (dict(s=0x3002), INVALID),
    (dict(dt=2), INVALID), (dict(dt=9), INVALID), (dict(br=0), INVALID), (dict(br=64), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(count=-1), INVALID),
    (dict(ldx=255), INVALID), (dict(ldq=255), INVALID),
    (dict(count=70000, rows=70000), UNSUPPORTED), (dict(rows=0), 0), (dict(cols=0, x=None), 0),
    (dict(count=0, codes=None), 0)])
def test_quantize_refusals(L, bad, want):
    assert quantize(L, **bad) == want


def mm(**kw):
    a = dict(M=32, N=512, K=256, out_dtype=smr.BF16, lda=256, ldb=256, ldo=512, workspace=0x100000,
             workspace_bytes=1 << 40)
    a.update(kw)
    return smr._Fp8Matmul(*[a[f] for f, _ in smr._Fp8Matmul._fields_])


@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(out_dtype=3), INVALID),
    (dict(lda=240), INVALID), (dict(lda=264), INVALID), (dict(ldb=248), INVALID), (dict(ldo=511), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=0x100010), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE), (dict(lda=1 << 41), UNSUPPORTED),
    (dict(N=(1 << 30) + 1, ldo=1 << 31), UNSUPPORTED), (dict(M=0), 0), (dict(N=0), 0)])
def test_matmul_refusals(L, bad, want):
    m = mm(**bad)
    assert L.moe_fp8_matmul(0x1000, 0x2000, 0x3000, 0x4000, ctypes.byref(m), 0x5000, None) == want
    if want in (INVALID, UNSUPPORTED):
        assert L.moe_fp8_matmul_workspace_bytes(ctypes.byref(m)) == 0
        assert L.moe_fp8_matmul_init(ctypes.byref(m), None) == want


def test_matmul_null_and_misaligned_tensors(L):
    good = [0x1000, 0x2000, 0x3000, 0x4000, 0x5000]
    m = mm()
    for i in range(5):
        for bad in (None, good[i] + 1):
            p = list(good)
            p[i] = bad
            assert L.moe_fp8_matmul(*p[:4], ctypes.byref(m), p[4], None) == INVALID
    assert L.moe_fp8_matmul(0x1008, 0x2000, 0x3000, 0x4000, ctypes.byref(m), 0x5000, None) == INVALID
    assert L.moe_fp8_matmul(0x1000, 0x2000, 0x3000, 0x4000, ctypes.byref(m), 0x3000, None) == INVALID
    assert L.moe_fp8_matmul(*good[:4], None, 0x5000, None) == INVALID


def test_matmul_workspace_covers_the_split(L):
    """Few tiles and a long k need room for partial sums; others the control block only."""
    small = L.moe_fp8_matmul_workspace_bytes(ctypes.byref(mm(M=8, K=14336, lda=14336, ldb=14336)))
    split = L.moe_fp8_matmul_workspace_bytes(ctypes.byref(mm(M=64, K=14336, lda=14336, ldb=14336)))
    large = L.moe_fp8_matmul_workspace_bytes(ctypes.byref(mm(M=8192, N=14336, ldo=14336)))
    assert small == large == 256 and split > 2 * 128 * 256 * 4


def cfg(**kw):
    a = dict(T=32, d_model=256, n_experts=16, top_k=4, d_ff=64, d_ff_shared=64,
             expert_dtype=smr.F8_E4M3_B128)
    a.update(kw)
    return smr.MoEConfig(**a)


def bank(w=0x10000, s=0x20000):
    return smr._Bank(w, s, None)


def experts(L, c, x=0x1000, r=None, ids=0x2000, alpha=0x3000, s_shared=0x4000, banks=None, w_shared=None,
            out=0x5000, dt=smr.BF16):
    banks = banks or [bank()] * 6
    return L.moe_fp8_experts_forward(x, r, ids, alpha, s_shared, *banks, w_shared, ctypes.byref(c), out, dt, None)


def with_workspace(c, n=1 << 40, at=0x100000):
    s = c._c()
    s.workspace, s.workspace_bytes = at, n
    return s


@pytest.mark.parametrize("bad,want", [
    (dict(expert_dtype=smr.BF16), INVALID), (dict(expert_dtype=smr.Q4_AFFINE_G64), INVALID),
    (dict(act_dtype=smr.F32), UNSUPPORTED), (dict(path=smr.PATH_FUSED), UNSUPPORTED), (dict(path=9), INVALID),
    (dict(path=smr.PATH_GEMV), UNSUPPORTED), (dict(path=smr.PATH_GEMV, T=17), UNSUPPORTED),
    (dict(d_model=264), UNSUPPORTED), (dict(d_ff=72), UNSUPPORTED), (dict(d_ff_shared=8), UNSUPPORTED),
    (dict(d_model=100), INVALID), (dict(d_ff=0), INVALID), (dict(d_ff_shared=-16), INVALID),
    (dict(T=-1), INVALID), (dict(top_k=17), INVALID), (dict(n_experts=0), INVALID),
    (dict(n_experts=1024), UNSUPPORTED), (dict(T=1 << 27), UNSUPPORTED)])
def test_layer_configurations_refused(L, bad, want):
    c = cfg(**bad)
    assert L.moe_fp8_workspace_bytes(ctypes.byref(c._c())) == 0
    assert experts(L, with_workspace(c)) == want
    assert L.moe_fp8_workspace_init(ctypes.byref(with_workspace(c)), None) == want
    assert L.moe_fp8_layer_forward(0x1000, None, 0x2000, None, *[bank()] * 6, 0x4000,
                                   ctypes.byref(with_workspace(c)), 0x5000, 0, 0x6000, 0x7000, None) == want


def test_layer_workspace_and_tensors_refused(L):
    c = with_workspace(cfg())
    need = smr.fp8_workspace_bytes(cfg())
    assert experts(L, with_workspace(cfg(), need - 1)) == WORKSPACE
    assert experts(L, with_workspace(cfg(), at=0x100010)) == WORKSPACE
    assert experts(L, cfg()._c()) == WORKSPACE
    assert L.moe_fp8_workspace_init(ctypes.byref(with_workspace(cfg(), need - 1)), None) == WORKSPACE
    for kw in (dict(x=None), dict(ids=None), dict(alpha=None), dict(out=None), dict(x=0x1008),
               dict(r=0x1004), dict(out=0x5008), dict(dt=2), dict(dt=7), dict(s_shared=None),
               dict(s_shared=0x4004), dict(w_shared=0x4008), dict(out=0x1000),
               dict(r=0x5000, out=0x5000, dt=smr.BF16)):
        assert experts(L, c, **kw) == INVALID, kw
    for i in range(6):
        for b in (bank(w=None), bank(s=None), bank(w=0x10008), bank(s=0x20004)):
            banks = [bank()] * 6
            banks[i] = b
            assert experts(L, c, banks=banks) == INVALID
    for kw in (dict(W=None), dict(W=0x2004), dict(bias=0x2004), dict(ws=None), dict(ids=None)):
        a = dict(W=0x2000, bias=None, ws=0x4000, ids=0x6000)
        a.update(kw)
        assert L.moe_fp8_layer_forward(0x1000, None, a["W"], a["bias"], *[bank()] * 6, a["ws"],
                                       ctypes.byref(c), 0x5000, 0, a["ids"], 0x7000, None) == INVALID


def test_no_tokens_enqueue_nothing(L):
    assert experts(L, with_workspace(cfg(T=0)), x=None, ids=None, alpha=None, out=None) == 0


def test_other_calls_keep_refusing_8_bit_banks(L):
    c = with_workspace(cfg())
    b = bank()
    assert L.moe_workspace_bytes(ctypes.byref(c)) == 0
    assert L.moe_experts_forward(0x1000, 0x2000, 0x3000, 0x4000, None, b, b, b, None, None, None, None,
                                 ctypes.byref(c), 0x5000, None) == INVALID


def test_layer_workspace_grows_with_tokens(L):
    a, b, c = (smr.fp8_workspace_bytes(cfg(T=t)) for t in (1, 16, 4096))
    assert 0 < a < b < c and c % 256 == 0


def test_binding_refuses_wrong_tensors(L):
    """The binding's own checks: devices, types and shapes, before the C call."""
    x = torch.zeros(4, 128)
    codes, scales = smr.fp8_empty(4, 128, device="cpu")
    with pytest.raises(ValueError):
        smr.fp8_quantize(x, codes, scales)                       # not on a GPU
    with pytest.raises(ValueError):
        smr.fp8_quantize(x, codes[:3], scales)
    with pytest.raises(ValueError):
        smr.fp8_quantize(x, codes.float(), scales)
    with pytest.raises(ValueError):
        smr.fp8_quantize(x, codes, scales.double())
    with pytest.raises(ValueError):
        smr.fp8_quantize(x.half(), codes, scales)
    with pytest.raises(ValueError):
        smr.fp8_matmul(codes, scales, codes, scales, torch.zeros(4, 5), scales)
    with pytest.raises(ValueError):
        smr.fp8_matmul(codes, scales, codes[:, :64], scales, torch.zeros(4, 4), scales)
    codes, scales = smr.fp8_empty(10, 100, 128, count=3, device="cpu")
    assert codes.shape == (3, 10, 100) and codes.stride(1) == 112 and scales.shape == (3, 1, 1)


def test_binding_refuses_wrong_layer_tensors(L):
    """Types and shapes of x, ids, weights, out, gate and residual."""
    c = cfg(T=4)
    good = dict(x=torch.zeros(4, 256, dtype=torch.bfloat16), topk_ids=torch.zeros(4, 4, dtype=torch.int32),
                weights=torch.zeros(4, 4), out=torch.zeros(4, 256), s_shared=torch.zeros(4),
                r_attn=torch.zeros(4, 256))
    smr._check_layer(c, **good)
    for name, bad in (("x", good["x"].float()), ("x", good["x"][:3]), ("topk_ids", good["topk_ids"].long()),
                      ("topk_ids", good["topk_ids"][:, :3]), ("weights", good["weights"].double()),
                      ("weights", good["weights"][:2]), ("out", good["out"][:, :128]),
                      ("s_shared", torch.zeros(3)), ("s_shared", torch.zeros(4).half()),
                      ("r_attn", good["r_attn"].bfloat16()), ("r_attn", good["r_attn"][:1])):
        with pytest.raises(ValueError):
            smr._check_layer(c, **dict(good, **{name: bad}))
    with pytest.raises(ValueError):  # the workspace on the host
        smr.fp8_experts_forward(c, torch.zeros(8, dtype=torch.uint8), good["x"], good["topk_ids"], good["weights"],
                                None, None, None, good["out"])


@pytest.mark.parametrize("kid", [16, 17, 18])
def test_failure_self_test_takes_the_new_kernels(L, kid):
    assert L.moe_inject_stall(kid, 100) == 0
    assert L.moe_inject_stall(0, 0) == 0
    for bad in (13, 14, 15, 19):
        assert L.moe_inject_stall(bad, 100) == INVALID
