"""Python binding of libmoe_route (the sparse MoE layer forward, GB300).

Argument marshalling only: every step of the layer runs in the CUDA kernels
of libmoe_route.so, called through its C ABI (include/moe_route.h). torch
supplies device memory and the current stream. There is no CPU fallback: if
the shared library is missing, importing the binding's functions raises.

Build the library with `python -m sparse_moe_routing_gb300.build`.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, replace

__all__ = [
    "MoEConfig", "MoEError", "lib", "lib_path", "abi_version", "status_string",
    "workspace_bytes", "alloc_workspace", "route", "bucket", "experts_forward",
    "layer_forward", "read_device_status", "SOFTMAX_TOPK", "SIGMOID_GROUP_TOPK",
    "F32", "BF16", "Q4_AFFINE_G64", "PATH_AUTO", "PATH_GEMV", "PATH_TC", "PATH_FUSED",
    "inject_stall", "F8_E4M3_B128", "fp8_empty", "fp8_quantize", "fp8_matmul",
    "fp8_matmul_workspace", "fp8_workspace_bytes", "fp8_alloc_workspace", "fp8_experts_forward",
    "fp8_layer_forward", "Fp8Experts", "Fp8Linear",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libmoe_route.so")

SOFTMAX_TOPK, SIGMOID_GROUP_TOPK = 0, 1
F32, BF16, Q4_AFFINE_G64, F8_E4M3_B128 = 0, 1, 2, 3
PATH_AUTO, PATH_GEMV, PATH_TC, PATH_FUSED = 0, 1, 2, 3
_STATUS = ["MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_WORKSPACE",
           "MOE_ERR_CUDA", "MOE_ERR_DEVICE_TIMEOUT", "MOE_ERR_DEVICE_CHECK"]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s" % (where, status_string(status))
        if status == 4:
            try:
                msg += " (%s)" % lib().moe_last_cuda_error().decode()
            except Exception:
                pass
        super().__init__(msg)


class _Cfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("router", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scaling", ctypes.c_float),
                ("renorm_clamp", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("expert_dtype", ctypes.c_int32), ("path", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class _Bank(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("minv", ctypes.c_void_p)]


class _Fp8Matmul(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ldo", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


_P = ctypes.c_void_p
_SIGS = {
    "moe_abi_version": (ctypes.c_int, []),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_Cfg)]),
    "moe_workspace_init": (ctypes.c_int, [ctypes.POINTER(_Cfg), _P]),
    "moe_read_device_status": (ctypes.c_int, [ctypes.POINTER(_Cfg), _P,
                                              ctypes.POINTER(ctypes.c_uint32)]),
    "moe_route": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_Cfg), _P, _P, _P, _P]),
    "moe_bucket": (ctypes.c_int, [_P, ctypes.POINTER(_Cfg), _P, _P, _P, _P, _P, _P, _P]),
    "moe_experts_forward": (ctypes.c_int, [_P, _P, _P, _P, _P, _Bank, _Bank, _Bank, _P, _P, _P,
                                           _P, ctypes.POINTER(_Cfg), _P, _P]),
    "moe_layer_forward": (ctypes.c_int, [_P, _P, _P, _P, _Bank, _Bank, _Bank, _P, _P, _P, _P,
                                         ctypes.POINTER(_Cfg), _P, _P, _P, _P]),
    "moe_launch_count": (ctypes.c_uint64, []),
    "moe_last_cuda_error": (ctypes.c_char_p, []),
    "moe_trace_kernel": (ctypes.c_int, [ctypes.c_int, _P, _P, ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_int)]),
    "moe_inject_stall": (ctypes.c_int, [ctypes.c_int, ctypes.c_uint32]),
    "moe_fp8_quantize": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 4
                         + [_P, ctypes.c_int64, _P, _P]),
    "moe_fp8_matmul": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_Fp8Matmul), _P, _P]),
    "moe_fp8_matmul_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_Fp8Matmul)]),
    "moe_fp8_matmul_init": (ctypes.c_int, [ctypes.POINTER(_Fp8Matmul), _P]),
    "moe_fp8_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_Cfg)]),
    "moe_fp8_workspace_init": (ctypes.c_int, [ctypes.POINTER(_Cfg), _P]),
    "moe_fp8_experts_forward": (ctypes.c_int, [_P] * 5 + [_Bank] * 6 + [
        _P, ctypes.POINTER(_Cfg), _P, ctypes.c_int32, _P]),
    "moe_fp8_layer_forward": (ctypes.c_int, [_P] * 4 + [_Bank] * 6 + [
        _P, ctypes.POINTER(_Cfg), _P, ctypes.c_int32, _P, _P, _P]),
}

# kernel families (moe_kernel_t)
KERNELS = {"router_logits": 1, "router_topk": 2, "shared_gate": 3, "bucket": 4,
           "gemv_gateup": 5, "gemv_down": 6, "combine": 7, "tc_gateup": 8, "tc_down": 9,
           "gather": 10, "tc_router": 11, "decode_fused": 12, "f8_quant": 13,
           "f8_few_gateup": 14, "f8_few_down": 15, "f8_tc_gateup": 16, "f8_tc_down": 17,
           "f8_matmul": 18}

_lib = None


def lib():
    """The loaded libmoe_route.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError("libmoe_route.so is not built (%s); run "
                               "`python -m sparse_moe_routing_gb300.build`" % lib_path)
        L = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def abi_version() -> int:
    return lib().moe_abi_version()


def status_string(status: int) -> str:
    try:
        return lib().moe_status_string(int(status)).decode()
    except RuntimeError:
        return _STATUS[status] if 0 <= status < len(_STATUS) else "unknown status %d" % status


@dataclass
class MoEConfig:
    """Layer configuration (moe_cfg_t without the workspace fields)."""
    T: int
    d_model: int
    n_experts: int
    top_k: int
    d_ff: int
    d_ff_shared: int = 0
    router: int = SOFTMAX_TOPK
    n_group: int = 1
    topk_group: int = 1
    routed_scaling: float = 1.0
    renorm_clamp: float = 2.0 ** -14
    act_dtype: int = BF16
    expert_dtype: int = BF16
    path: int = PATH_AUTO

    def _c(self, workspace=None) -> _Cfg:
        c = _Cfg(self.T, self.d_model, self.n_experts, self.top_k, self.d_ff, self.d_ff_shared,
                 self.router, self.n_group, self.topk_group, self.routed_scaling,
                 self.renorm_clamp, self.act_dtype, self.expert_dtype, self.path, None, 0)
        if workspace is not None:
            c.workspace = workspace.data_ptr()
            c.workspace_bytes = workspace.numel() * workspace.element_size()
        return c


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _bank(b):
    """A bank is a tensor (f32/bf16) or a (codes, scale, min) tuple (q4)."""
    if isinstance(b, (tuple, list)):
        return _Bank(_ptr(b[0]), _ptr(b[1]), _ptr(b[2]))
    return _Bank(_ptr(b), None, None)


_raw_stream = None


def _stream(stream):
    """The stream's handle; None: the current stream of the current device."""
    global _raw_stream
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        # the handle alone, where this torch gives it: making a Stream object of
        # it costs 3 us, a call of the smallest kernels 3 us in all
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            _raw_stream = lambda: raw(torch.cuda.current_device())  # noqa: E731
    return ctypes.c_void_p(_raw_stream())


def _check(status: int, where: str):
    if status != 0:
        raise MoEError(status, where)


def _empty(shape, dtype, device, stream):
    """torch.empty for a call on `stream` (None: the current one): from that
    stream's memory, so that a block handed out or given back early is used
    again in its order only; not before what the current stream has in hand at
    that time either."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device or "cuda")
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device or "cuda")
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def workspace_bytes(cfg: MoEConfig) -> int:
    n = lib().moe_workspace_bytes(ctypes.byref(cfg._c()))
    if n == 0:
        raise MoEError(1, "moe_workspace_bytes")
    return n


def alloc_workspace(cfg: MoEConfig, device=None, stream=None):
    """Allocates (with torch) and initialises a workspace for cfg on `stream`."""
    import torch
    ws = _empty(workspace_bytes(cfg), torch.uint8, device, stream)
    _check(lib().moe_workspace_init(ctypes.byref(cfg._c(ws)), _stream(stream)),
           "moe_workspace_init")
    return ws


def read_device_status(cfg: MoEConfig, workspace, stream=None):
    """Synchronises, returns (status, raw word) and clears the word."""
    info = ctypes.c_uint32(0)
    st = lib().moe_read_device_status(ctypes.byref(cfg._c(workspace)), _stream(stream),
                                      ctypes.byref(info))
    return st, info.value


def route(cfg, workspace, x, W_router, topk_ids, weights, expert_bias=None, w_shared=None,
          s_shared=None, stream=None):
    _check(lib().moe_route(_ptr(x), _ptr(W_router), _ptr(expert_bias), _ptr(w_shared),
                           ctypes.byref(cfg._c(workspace)), _ptr(topk_ids), _ptr(weights),
                           _ptr(s_shared), _stream(stream)), "moe_route")


def bucket(cfg, workspace, topk_ids, counts, offsets, active, n_active, perm, pos, stream=None):
    _check(lib().moe_bucket(_ptr(topk_ids), ctypes.byref(cfg._c(workspace)), _ptr(counts),
                            _ptr(offsets), _ptr(active), _ptr(n_active), _ptr(perm), _ptr(pos),
                            _stream(stream)), "moe_bucket")


def experts_forward(cfg, workspace, x, r_attn, topk_ids, weights, W_gate, W_up, W_down, out,
                    s_shared=None, Ws_gate=None, Ws_up=None, Ws_down=None, w_shared=None,
                    stream=None):
    _check(lib().moe_experts_forward(
        _ptr(x), _ptr(r_attn), _ptr(topk_ids), _ptr(weights), _ptr(s_shared), _bank(W_gate),
        _bank(W_up), _bank(W_down), _ptr(Ws_gate), _ptr(Ws_up), _ptr(Ws_down), _ptr(w_shared),
        ctypes.byref(cfg._c(workspace)), _ptr(out), _stream(stream)), "moe_experts_forward")


def layer_forward(cfg, workspace, x, r_attn, W_router, W_gate, W_up, W_down, out, topk_ids,
                  weights, expert_bias=None, Ws_gate=None, Ws_up=None, Ws_down=None,
                  w_shared=None, stream=None):
    _check(lib().moe_layer_forward(
        _ptr(x), _ptr(r_attn), _ptr(W_router), _ptr(expert_bias), _bank(W_gate), _bank(W_up),
        _bank(W_down), _ptr(Ws_gate), _ptr(Ws_up), _ptr(Ws_down), _ptr(w_shared),
        ctypes.byref(cfg._c(workspace)), _ptr(out), _ptr(topk_ids), _ptr(weights),
        _stream(stream)), "moe_layer_forward")


def inject_stall(kernel: str, wait_us: int):
    """Failure self-test (moe_inject_stall): the next launch of `kernel`
    ("tc_gateup", "tc_down", "decode_fused", "f8_tc_gateup", "f8_tc_down" or
    "f8_matmul") waits on a flag nothing sets and gives up after wait_us; None
    disarms."""
    _check(lib().moe_inject_stall(0 if kernel is None else KERNELS[kernel], int(wait_us)),
           "moe_inject_stall")


def launch_count() -> int:
    """Kernel launches this library has enqueued in this process."""
    return int(lib().moe_launch_count())


class KernelTrace:
    """Brackets every launch of one kernel family with CUDA events recorded on
    the stream it is launched on (moe_trace_kernel). Use as a context manager;
    `durations_ms()` returns one duration per traced launch (up to n)."""

    def __init__(self, kernel: str, n: int):
        import torch
        self.kernel = KERNELS[kernel]
        self.n = n
        self.starts = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        self.stops = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        self._count = ctypes.c_int(0)
        # torch creates the CUDA event lazily: record once to materialise it
        for e in self.starts + self.stops:
            e.record()
        self._sa = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.starts])
        self._so = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.stops])

    def __enter__(self):
        _check(lib().moe_trace_kernel(self.kernel, self._sa, self._so, self.n,
                                      ctypes.byref(self._count)), "moe_trace_kernel")
        return self

    def __exit__(self, *exc):
        lib().moe_trace_kernel(0, None, None, 0, None)
        return False

    @property
    def count(self) -> int:
        return self._count.value

    def durations_ms(self):
        import torch
        torch.cuda.synchronize()
        m = min(self.count, self.n)
        return [self.starts[i].elapsed_time(self.stops[i]) for i in range(m)]


class MoELayer:
    """One MoE layer's device weights plus its workspace: `forward` is the
    call a user makes (x, r_attn device tensors in, out/ids/weights out).

    weights: dict of device tensors named as in include/moe_route.h
    (W_router, expert_bias, W_gate, W_up, W_down or (codes, scale, min)
    tuples for 4-bit banks, Ws_gate, Ws_up, Ws_down, w_shared)."""

    def __init__(self, cfg: MoEConfig, weights: dict, device=None):
        import torch
        self.cfg = cfg
        self.w = weights
        self.device = device or torch.device("cuda", torch.cuda.current_device())
        self.ws = alloc_workspace(cfg, self.device)
        T, k, d = cfg.T, cfg.top_k, cfg.d_model
        self.out = torch.empty((T, d), dtype=torch.float32, device=self.device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=self.device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=self.device)

    def forward(self, x, r_attn, out=None, stream=None):
        w = self.w
        out = self.out if out is None else out
        def bank(name):  # a tensor, or the (codes, scale, min) of a 4-bit bank
            return w[name] if name in w else (w[name + "_q"], w[name + "_scale"], w[name + "_min"])

        layer_forward(self.cfg, self.ws, x, r_attn, w["W_router"], bank("W_gate"), bank("W_up"),
                      bank("W_down"), out, self.ids, self.weights,
                      expert_bias=w.get("expert_bias"), Ws_gate=w.get("Ws_gate"),
                      Ws_up=w.get("Ws_up"), Ws_down=w.get("Ws_down"),
                      w_shared=w.get("w_shared"), stream=stream)
        return out, self.ids, self.weights

    def device_status(self, stream=None):
        return read_device_status(self.cfg, self.ws, stream)


# ---------------------------------------------------------------------------
# 8-bit floating point: e4m3 codes and one fp32 scale per block of 128
# ---------------------------------------------------------------------------
_dt = None


def _dtypes():
    """torch dtype -> moe_dtype_t of the 8-bit calls' values."""
    global _dt
    if _dt is None:
        import torch
        _dt = {torch.float32: F32, torch.bfloat16: BF16}
    return _dt


def _dtype_of(t):
    d = (_dt or _dtypes()).get(t.dtype)
    if d is None:
        raise ValueError("expected a float32 or bfloat16 tensor, got %s" % t.dtype)
    return d


def _ld(t, shape, name):
    """Values between the rows of a matrix (or of a stack of them) on a CUDA
    device with unit column stride; the row length where there is one row."""
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    stride = t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have contiguous rows" % name)
    return stride[-2] if shape[-2] > 1 else max(stride[-2], shape[-1])


def _codes_dtype(t, name):
    if t.dtype not in (_codes_types or _code_types()):
        raise ValueError("%s must be float8_e4m3fn (or its bytes as uint8)" % name)


_codes_types = None


def _code_types():
    global _codes_types
    import torch
    _codes_types = (torch.float8_e4m3fn, torch.uint8)
    return _codes_types


def _shape_is(t, shape, name):
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _scales_ok(t, shape, name):
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if (_dt or _dtypes()).get(t.dtype) != F32:
        raise ValueError("%s must be float32" % name)


def fp8_empty(rows, cols, block_rows=1, count=None, device=None):
    """(codes, scales) tensors for a rows x cols matrix (a stack of `count` of
    them): codes' rows are padded to 16 bytes, as the products take them."""
    import torch
    lead = () if count is None else (count,)
    pitch = -(-cols // 16) * 16
    codes = torch.empty(lead + (rows, pitch), dtype=torch.float8_e4m3fn, device=device or "cuda")
    scales = torch.empty(lead + (-(-rows // block_rows), -(-cols // 128)), dtype=torch.float32,
                         device=device or "cuda")
    return codes[..., :cols], scales


def fp8_quantize(x, codes, scales, block_rows=1, stream=None):
    """moe_fp8_quantize: x [rows, cols] or [count, rows, cols] (float32 or
    bfloat16) into codes (float8_e4m3fn, same shape) and scales."""
    shape = x.shape
    n = len(shape)
    if n not in (2, 3):
        raise ValueError("x must have two or three dimensions")
    _codes_dtype(codes, "codes")
    _shape_is(codes, shape, "codes")
    rows, cols = shape[-2], shape[-1]
    nb = (-(-rows // block_rows) if block_rows > 0 else 0, -(-cols // 128))
    _scales_ok(scales, nb if n == 2 else (shape[0],) + nb, "scales")
    dtype = _dtype_of(x)
    ldx, ldq = _ld(x, shape, "x"), _ld(codes, shape, "codes")
    count = 1
    if n == 3:
        count = shape[0]
        if count > 1 and (x.stride(0) != rows * ldx or codes.stride(0) != rows * ldq):
            raise ValueError("stacked matrices must follow one another at rows * row stride")
    _check(lib().moe_fp8_quantize(x.data_ptr(), dtype, ldx, count, rows, cols, block_rows,
                                  codes.data_ptr(), ldq, _ptr(scales), _stream(stream)),
           "moe_fp8_quantize")


def _matmul_args(M, N, K, out_dtype=BF16, lda=0, ldb=0, ldo=0, workspace=None):
    p = -(-max(K, 1) // 16) * 16
    m = _Fp8Matmul(M, N, K, out_dtype, lda or p, ldb or p, ldo or N, None, 0)
    if workspace is not None:
        m.workspace = workspace.data_ptr()
        m.workspace_bytes = workspace.numel() * workspace.element_size()
    return m


def fp8_matmul_workspace(M, N, K, device=None, stream=None):
    """Allocates (with torch) and initialises the workspace of an M x N x K
    product on `stream`."""
    import torch
    n = lib().moe_fp8_matmul_workspace_bytes(ctypes.byref(_matmul_args(M, N, K)))
    if n == 0:
        raise MoEError(1, "moe_fp8_matmul_workspace_bytes")
    ws = _empty(n, torch.uint8, device, stream)
    _check(lib().moe_fp8_matmul_init(ctypes.byref(_matmul_args(M, N, K, workspace=ws)),
                                     _stream(stream)), "moe_fp8_matmul_init")
    return ws


def fp8_matmul(a, a_scale, b, b_scale, out, workspace, stream=None):
    """moe_fp8_matmul: out [M, N] = a [M, K] b [N, K]^T, codes with scales per
    1 x 128 (a) and 128 x 128 (b); out float32 or bfloat16."""
    (M, K), N = a.shape, b.shape[0]
    _codes_dtype(a, "a")
    _codes_dtype(b, "b")
    _shape_is(b, (N, K), "b")
    _shape_is(out, (M, N), "out")
    kb = -(-K // 128)
    _scales_ok(a_scale, (M, kb), "a_scale")
    _scales_ok(b_scale, (-(-N // 128), kb), "b_scale")
    m = _Fp8Matmul(M, N, K, _dtype_of(out), _ld(a, (M, K), "a"), _ld(b, (N, K), "b"),
                   _ld(out, (M, N), "out"), _ptr(workspace),
                   workspace.numel() * workspace.element_size())
    _check(lib().moe_fp8_matmul(a.data_ptr(), _ptr(a_scale), b.data_ptr(), _ptr(b_scale),
                                ctypes.byref(m), out.data_ptr(), _stream(stream)), "moe_fp8_matmul")


class Fp8Linear:
    """y = x W^T with W [N, K] held in 8 bits and x quantised on the way:
    fp8_quantize, then fp8_matmul, for up to max_rows rows. The quantised x and
    the workspace belong to the object: calls on several streams are ordered by
    the caller."""

    def __init__(self, weight, max_rows, device=None):
        if device is not None:
            weight = weight.to(device)
        N, K = weight.shape
        self.N, self.K, self.max_rows = N, K, max_rows
        self.codes, self.scales = fp8_empty(N, K, 128, device=weight.device)
        fp8_quantize(weight, self.codes, self.scales, block_rows=128)
        self.x, self.x_scales = fp8_empty(max_rows, K, 1, device=weight.device)
        # One workspace for every number of rows. What a product needs depends on
        # its row blocks only and does not grow with them alone (fewer tiles are
        # split more), but past 152 of them k is not split.
        size = lambda M: lib().moe_fp8_matmul_workspace_bytes(  # noqa: E731
            ctypes.byref(_matmul_args(M, N, K)))
        most = max((1, *range(128, min(max_rows, 152 * 128) + 1, 128), max_rows), key=size)
        self.ws = fp8_matmul_workspace(most, N, K, weight.device)

    def __call__(self, x, out, stream=None):
        M = x.shape[0]
        if M > self.max_rows:
            raise ValueError("x has %d rows, made for %d" % (M, self.max_rows))
        xq, xs = self.x[:M], self.x_scales[:M]
        fp8_quantize(x, xq, xs, stream=stream)
        fp8_matmul(xq, xs, self.codes, self.scales, out, self.ws, stream)
        return out

    def device_status(self, stream=None):
        """(status, raw word) of the products since the last call, as read_device_status."""
        return read_device_status(MoEConfig(T=1, d_model=128, n_experts=1, top_k=1, d_ff=128), self.ws, stream)


def fp8_workspace_bytes(cfg: MoEConfig) -> int:
    c = cfg._c()
    n = lib().moe_fp8_workspace_bytes(ctypes.byref(c))
    if n == 0:
        raise MoEError(1, "moe_fp8_workspace_bytes")
    return n


def fp8_alloc_workspace(cfg: MoEConfig, device=None, stream=None):
    """Allocates (with torch) and initialises a workspace of the 8-bit layer on
    `stream`. It serves other T of the same layer too, where it is large enough."""
    import torch
    ws = _empty(fp8_workspace_bytes(cfg), torch.uint8, device, stream)
    _check(lib().moe_fp8_workspace_init(ctypes.byref(cfg._c(ws)), _stream(stream)),
           "moe_fp8_workspace_init")
    return ws


def _bank8(b, shape):
    """An 8-bit bank from (codes, scales); None stands for no shared expert. A bank
    of one matrix may come without its first dimension."""
    if b is None:
        return _Bank(None, None, None)
    codes, scales = b
    _codes_dtype(codes, "a bank's codes")
    if tuple(codes.shape) not in (tuple(shape), tuple(shape)[1:] if shape[0] == 1 else None):
        raise ValueError("a bank's codes have shape %s, expected %s" % (tuple(codes.shape), tuple(shape)))
    want = (shape[0], -(-shape[1] // 128), -(-shape[2] // 128))
    _scales_ok(scales, want[1:] if shape[0] == 1 and scales.dim() == 2 else want, "a bank's scales")
    return _Bank(_ptr(codes), _ptr(scales), None)


def _banks8(cfg, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down):
    E, d, I, Is = cfg.n_experts, cfg.d_model, cfg.d_ff, cfg.d_ff_shared
    sh = (lambda b, s: _bank8(b, s)) if Is else (lambda b, s: _Bank(None, None, None))
    return (_bank8(W_gate, (E, I, d)), _bank8(W_up, (E, I, d)), _bank8(W_down, (E, d, I)),
            sh(Ws_gate, (1, Is, d)), sh(Ws_up, (1, Is, d)), sh(Ws_down, (1, d, Is)))


_layer_types = None


def _check_layer(cfg, x, topk_ids, weights, out, s_shared, r_attn):
    """Types and shapes of the 8-bit layer's tensors; cfg a MoEConfig or the
    structure that the call gets."""
    global _layer_types
    if _layer_types is None:
        import torch
        _layer_types = torch.bfloat16, torch.int32, torch.float32
    bf16, i32, f32 = _layer_types
    xs, ks = (cfg.T, cfg.d_model), (cfg.T, cfg.top_k)
    if x.dtype != bf16 or x.shape != xs or out.shape != xs:
        raise ValueError("x must be bfloat16 [%d, %d], and out as large" % xs)
    if topk_ids.dtype != i32 or topk_ids.shape != ks or weights.dtype != f32 or weights.shape != ks:
        raise ValueError("topk_ids must be int32 and weights float32 [%d, %d]" % ks)
    if r_attn is not None and (r_attn.dtype != f32 or r_attn.shape != xs):
        raise ValueError("r_attn must be float32 [%d, %d]" % xs)
    if s_shared is not None and (s_shared.dtype != f32 or s_shared.numel() != cfg.T):
        raise ValueError("s_shared must be float32 [%d]" % cfg.T)


def _check_routing(cfg, W_router, expert_bias, w_shared):
    """Types and shapes of the 8-bit layer's routing tensors, where given."""
    import torch
    E, d = cfg.n_experts, cfg.d_model
    if W_router is not None and (W_router.dtype != torch.bfloat16 or W_router.shape != (E, d)):
        raise ValueError("W_router must be bfloat16 [%d, %d]" % (E, d))
    if expert_bias is not None and (expert_bias.dtype != torch.float32 or expert_bias.numel() != E):
        raise ValueError("expert_bias must be float32 [%d]" % E)
    if w_shared is not None and (w_shared.dtype != torch.bfloat16 or w_shared.numel() != d):
        raise ValueError("w_shared must be bfloat16 [%d]" % d)


def fp8_experts_forward(cfg, workspace, x, topk_ids, weights, W_gate, W_up, W_down, out,
                        s_shared=None, r_attn=None, Ws_gate=None, Ws_up=None, Ws_down=None,
                        w_shared=None, stream=None):
    """moe_fp8_experts_forward: banks are (codes, scales) pairs; out float32 or
    bfloat16 [T, d_model]; r_attn optional."""
    _check_layer(cfg, x, topk_ids, weights, out, s_shared, r_attn)
    _check_routing(cfg, None, None, w_shared)
    _ptr(workspace)
    b = _banks8(cfg, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down)
    _check(lib().moe_fp8_experts_forward(
        _ptr(x), _ptr(r_attn), _ptr(topk_ids), _ptr(weights), _ptr(s_shared), *b, _ptr(w_shared),
        ctypes.byref(cfg._c(workspace)), _ptr(out), _dtype_of(out), _stream(stream)),
        "moe_fp8_experts_forward")


def fp8_layer_forward(cfg, workspace, x, W_router, W_gate, W_up, W_down, out, topk_ids, weights,
                      r_attn=None, expert_bias=None, Ws_gate=None, Ws_up=None, Ws_down=None,
                      w_shared=None, stream=None):
    """moe_fp8_layer_forward: the whole layer with 8-bit banks."""
    _check_layer(cfg, x, topk_ids, weights, out, None, r_attn)
    _check_routing(cfg, W_router, expert_bias, w_shared)
    _ptr(workspace)
    b = _banks8(cfg, W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down)
    _check(lib().moe_fp8_layer_forward(
        _ptr(x), _ptr(r_attn), _ptr(W_router), _ptr(expert_bias), *b, _ptr(w_shared),
        ctypes.byref(cfg._c(workspace)), _ptr(out), _dtype_of(out), _ptr(topk_ids), _ptr(weights),
        _stream(stream)), "moe_fp8_layer_forward")


class Fp8Experts:
    """One layer's 8-bit banks plus its workspace; `forward` runs the expert
    half for given routing, `layer` routing and experts.

    weights: dict of (codes, scales) pairs W_gate, W_up, W_down and, with a
    shared expert, Ws_gate, Ws_up, Ws_down; for `layer` also W_router,
    expert_bias and w_shared tensors. `from_bf16` quantises a bf16 layer's.

    Calls run on `stream` (None: the current one), after what is on it: a caller
    who changes streams orders them, the object's making and its calls among
    themselves (they share a workspace). A result that a call allocates (out not
    given) belongs to the call's stream."""

    def __init__(self, cfg: MoEConfig, weights: dict, device=None):
        import torch
        self.cfg = replace(cfg)
        self.w = dict(weights)  # (the calls go by the banks' addresses)
        _check_routing(cfg, weights.get("W_router"), weights.get("expert_bias"), weights.get("w_shared"))
        self.device = device or torch.device("cuda", torch.cuda.current_device())
        self.ws = fp8_alloc_workspace(cfg, self.device)
        self._banks = _banks8(cfg, weights["W_gate"], weights["W_up"], weights["W_down"],
                              weights.get("Ws_gate"), weights.get("Ws_up"), weights.get("Ws_down"))
        self._c = cfg._c(self.ws)
        self._cp = ctypes.byref(self._c)
        self._x_shape = (cfg.T, cfg.d_model)
        self._w_shared = _ptr(weights.get("w_shared"))

    @staticmethod
    def from_bf16(cfg: MoEConfig, weights: dict, device=None):
        """Quantises the banks of a layer's weight dict (128 x 128 blocks)."""
        w = dict(weights)
        for name in ("W_gate", "W_up", "W_down", "Ws_gate", "Ws_up", "Ws_down"):
            m = weights.get(name)
            if m is None:
                continue
            codes, scales = fp8_empty(m.shape[-2], m.shape[-1], 128,
                                      m.shape[0] if m.dim() == 3 else None, m.device)
            fp8_quantize(m, codes, scales, block_rows=128)
            w[name] = (codes, scales)
        return Fp8Experts(cfg, w, device)

    def forward(self, x, topk_ids, weights, s_shared=None, r_attn=None, out=None, stream=None):
        import torch
        if out is None:
            out = _empty(self._x_shape, torch.bfloat16, self.device, stream)
        _check_layer(self._c, x, topk_ids, weights, out, s_shared, r_attn)
        _check(lib().moe_fp8_experts_forward(
            _ptr(x), _ptr(r_attn), _ptr(topk_ids), _ptr(weights), _ptr(s_shared), *self._banks,
            self._w_shared, self._cp, _ptr(out), _dtype_of(out), _stream(stream)),
            "moe_fp8_experts_forward")
        return out

    def layer(self, x, topk_ids, weights, r_attn=None, out=None, stream=None):
        import torch
        if out is None:
            out = _empty(self._x_shape, torch.bfloat16, self.device, stream)
        _check_layer(self._c, x, topk_ids, weights, out, None, r_attn)
        _check(lib().moe_fp8_layer_forward(
            _ptr(x), _ptr(r_attn), _ptr(self.w["W_router"]), _ptr(self.w.get("expert_bias")),
            *self._banks, self._w_shared, self._cp, _ptr(out), _dtype_of(out),
            _ptr(topk_ids), _ptr(weights), _stream(stream)), "moe_fp8_layer_forward")
        return out

    def device_status(self, stream=None):
        return read_device_status(self.cfg, self.ws, stream)
