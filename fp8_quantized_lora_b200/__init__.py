"""B200 (sm_100a) hot path of FALQON's melded FP8 linear layer.

A thin ctypes binding over ``libfalqon.so`` (C ABI declared in
``include/falqon.h``).  Each Python function has the name of the C entry
point it marshals to and only turns torch tensors into device pointers and
the current CUDA stream into a ``void*``; all computation runs in the
library's CUDA kernels.  There is no CPU path: importing this package without
the built library raises.
"""

from __future__ import annotations

import ctypes as C
import os

import torch

__all__ = [
    "FalqonError", "lib", "falqon_quantize", "falqon_linear_fwd", "falqon_linear_bwd",
    "falqon_proxy_update", "falqon_workspace_size", "falqon_status_string", "falqon_version",
    "falqon_linear_bwd_noalloc", "falqon_proxy_update_topk", "falqon_linear_fwd_folded",
    "falqon_linear_bwd_folded", "folded_t_planes", "falqon_selftest_bounded_waits", "falqon_workspace_init",
    "workspace", "falqon_lora_separate_fwd", "falqon_lora_separate_bwd", "separate_saved_views",
    "separate_bwd_views", "falqon_linear_fwd_grouped",
    "falqon_norm_fwd", "falqon_norm_bwd", "falqon_linear_fwd_epilogue", "falqon_linear_epilogue_bwd",
    "falqon_clip_grads", "GradList", "NORM_LAYER", "NORM_RMS", "ACT_NONE", "ACT_RELU", "ACT_GELU_ERF",
    "ACT_GELU_TANH", "ACT_SILU", "OP_NORM_BWD", "OP_LINEAR_EPILOGUE_BWD", "OP_CLIP_GRADS",
    "SEPARATE_BF16", "SEPARATE_FP8", "OP_QUANTIZE",
    "OP_LINEAR_FWD",
    "OP_LINEAR_BWD", "OP_PROXY_UPDATE", "OP_PROXY_UPDATE_TOPK", "OP_FOLDED_T", "OP_LINEAR_BWD_FOLDED",
    "PROXY_ACCUMULATE", "PROXY_SELECT", "PROXY_KEEP_RESIDUAL", "PROXY_STRICT", "PROXY_TENSOR", "PROXY_DEFER_CLEAR", "DEV_NONFINITE", "DEV_SCALE_OVERFLOW", "DEV_TIMEOUT",
    "LIB_PATH", "EXPORTED_SYMBOLS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfalqon.so")

OP_QUANTIZE, OP_LINEAR_FWD, OP_LINEAR_BWD, OP_PROXY_UPDATE, OP_PROXY_UPDATE_TOPK = 0, 1, 2, 3, 4
OP_FOLDED_T, OP_LINEAR_BWD_FOLDED = 5, 6
OP_SEPARATE_SAVED_BF16, OP_SEPARATE_SAVED_FP8, OP_SEPARATE_FWD_FP8 = 7, 8, 9
OP_SEPARATE_BWD_BF16, OP_SEPARATE_BWD_FP8 = 10, 11
OP_NORM_BWD, OP_LINEAR_EPILOGUE_BWD, OP_CLIP_GRADS = 12, 13, 14
SEPARATE_BF16, SEPARATE_FP8 = 0, 1
NORM_LAYER, NORM_RMS = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU_ERF, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
DTYPE_BF16, DTYPE_F32 = 0, 1
PROXY_ACCUMULATE, PROXY_SELECT, PROXY_KEEP_RESIDUAL, PROXY_STRICT, PROXY_TENSOR = 1, 2, 4, 8, 16
PROXY_DEFER_CLEAR = 32  # with ACCUMULATE | SELECT: row_mask carries the clear to the next call
DEV_NONFINITE, DEV_SCALE_OVERFLOW, DEV_TIMEOUT = 1, 2, 4
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE", 4: "CUDA"}

EXPORTED_SYMBOLS = (
    "falqon_quantize", "falqon_linear_fwd", "falqon_linear_bwd", "falqon_proxy_update",
    "falqon_workspace_size", "falqon_status_string", "falqon_version",
    "falqon_linear_bwd_noalloc", "falqon_proxy_update_topk", "falqon_quantize_e5m2",
    "falqon_linear_bwd_e5m2", "falqon_linear_fwd_folded", "falqon_linear_bwd_folded",
    "falqon_selftest_bounded_waits", "falqon_workspace_init", "falqon_lora_separate_fwd",
    "falqon_lora_separate_bwd", "falqon_linear_fwd_grouped", "falqon_norm_fwd", "falqon_norm_bwd",
    "falqon_linear_fwd_epilogue", "falqon_linear_epilogue_bwd", "falqon_clip_grads",
)


class FalqonError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.status, self.status)} "
                         f"({falqon_status_string(self.status)})")


_LIB = None


def lib():
    """The loaded C library (ctypes), with argument types declared."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m fp8_quantized_lora_b200.build` "
            "(there is no CPU fallback)")
    L = C.CDLL(LIB_PATH)
    p, i64, u32, sz = C.c_void_p, C.c_int64, C.c_uint32, C.c_size_t
    L.falqon_quantize.argtypes = [p, C.c_int, i64, i64, p, p, p, p, p, p, sz, p]
    L.falqon_quantize_e5m2.argtypes = [p, C.c_int, i64, i64, p, p, p, p, p, sz, p]
    L.falqon_linear_fwd.argtypes = [p, p, p, p, i64, i64, i64, p, p, p, sz, p]
    L.falqon_linear_bwd.argtypes = [p, p, p, p, p, p, p, p, i64, i64, i64, i64, p, p, p, p, p, sz, p]
    L.falqon_linear_bwd_e5m2.argtypes = [p, p, p, p, p, p, p, p, i64, i64, i64, i64, p, p, p, p, p, sz, p]
    L.falqon_proxy_update.argtypes = [p, p, p, p, p, i64, i64, i64, u32, p, p, p, p, sz, p]
    L.falqon_proxy_update_topk.argtypes = [p, p, p, p, p, i64, i64, i64, i64, u32, p, p, p, p, sz, p]
    L.falqon_linear_bwd_noalloc.argtypes = [p, p, p, p, p, p, p, p, i64, i64, i64, i64, p, p, p, p, p]
    L.falqon_linear_fwd_folded.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, p, p, sz, p, p]
    L.falqon_selftest_bounded_waits.argtypes = [p, p, p, p]
    L.falqon_linear_bwd_folded.argtypes = [p, p, p, p, p, p, p, p, p, sz, i64, i64, i64, i64, p, p, p, p, p,
                                           sz, p]
    for f in ("falqon_quantize", "falqon_linear_fwd", "falqon_linear_bwd", "falqon_proxy_update",
              "falqon_linear_bwd_noalloc"):
        getattr(L, f).restype = C.c_int
    L.falqon_lora_separate_fwd.argtypes = [C.c_int, p, p, p, p, p, p, p, i64, i64, i64, i64, p, p, sz, p, p, sz, p]
    L.falqon_lora_separate_bwd.argtypes = [C.c_int, p, p, p, p, p, p, p, p, p, p, p, sz, i64, i64, i64, i64, p, p,
                                           p, p, p, sz, p]
    L.falqon_linear_fwd_grouped.argtypes = [p, p, C.c_int, p, p, p, p, i64, i64, p, p]
    L.falqon_linear_fwd_grouped.restype = C.c_int
    f32 = C.c_float
    L.falqon_norm_fwd.argtypes = [p, C.c_int, p, p, C.c_int, C.c_int, i64, i64, f32, p, p, p, p, p]
    L.falqon_norm_bwd.argtypes = [p, p, C.c_int, p, C.c_int, C.c_int, p, p, p, i64, i64, p, p, p, p, p, sz, p]
    L.falqon_linear_fwd_epilogue.argtypes = [p, p, p, p, p, C.c_int, C.c_int, p, i64, i64, i64, p, p, p, p]
    L.falqon_linear_epilogue_bwd.argtypes = [p, p, C.c_int, i64, i64, p, p, p, sz, p]
    L.falqon_clip_grads.argtypes = [C.c_int, p, p, p, f32, f32, p, p, p, p, p, sz, p]
    for f in ("falqon_norm_fwd", "falqon_norm_bwd", "falqon_linear_fwd_epilogue", "falqon_linear_epilogue_bwd",
              "falqon_clip_grads"):
        getattr(L, f).restype = C.c_int
    L.falqon_workspace_init.argtypes = [p, sz, p]
    L.falqon_workspace_init.restype = C.c_int
    L.falqon_workspace_size.argtypes = [C.c_int, i64, i64, i64, i64]
    L.falqon_workspace_size.restype = sz
    L.falqon_status_string.argtypes = [C.c_int]
    L.falqon_status_string.restype = C.c_char_p
    L.falqon_version.restype = C.c_char_p
    _LIB = L
    return L


def falqon_status_string(status: int) -> str:
    return lib().falqon_status_string(int(status)).decode()


def falqon_version() -> str:
    return lib().falqon_version().decode()


def falqon_workspace_size(op: int, M: int = 0, N: int = 0, K: int = 0, r: int = 0) -> int:
    return int(lib().falqon_workspace_size(int(op), int(M), int(N), int(K), int(r)))


# ------------------------------------------------------------------ marshalling helpers
def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("falqon tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("falqon tensors must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise FalqonError(status, where)


def falqon_workspace_init(workspace, stream=None):
    """Zero-fills a workspace (uint8 tensor, 256-byte aligned) on the stream:
    required once for a quantize workspace before its first use."""
    st = lib().falqon_workspace_init(_ptr(workspace), workspace.numel(), _stream(stream, workspace.device))
    _check(st, "falqon_workspace_init")
    return workspace


def workspace(op, M=0, N=0, K=0, r=0, device="cuda", stream=None):
    """A 256-byte-aligned workspace for `op` at these sizes, initialised
    (falqon_workspace_init), or None when the op needs none."""
    need = falqon_workspace_size(op, M, N, K, r)
    if need == 0:
        return None
    raw = torch.empty(need + 256, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 256
    return falqon_workspace_init(raw[off:off + need], stream)


def _workspace(op, M, N, K, r, device, workspace):
    need = falqon_workspace_size(op, M, N, K, r)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = globals()["workspace"](op, M, N, K, r, device)
    return workspace, workspace.numel()


def _u8(t):
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


# ------------------------------------------------------------------ entry points
def falqon_quantize(x, codes=None, scale=None, amax=None, residual=None, dev_status=None,
                    workspace=None, stream=None, fmt="e4m3"):
    """Per-tensor FP8 quantization of a 2-D bf16/fp32 tensor (E4M3, or E5M2
    for gradients: fmt="e5m2", no residual); returns (codes, scale, amax)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    dt = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(x.dtype)
    if dt is None:
        raise ValueError("x must be bfloat16 or float32")
    dev = x.device
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if codes is None else codes
    scale = torch.empty(1, dtype=torch.float32, device=dev) if scale is None else scale
    amax = torch.empty(1, dtype=torch.float32, device=dev) if amax is None else amax
    ws, wsb = _workspace(OP_QUANTIZE, rows, cols, 0, 0, dev, workspace)
    if fmt == "e5m2":
        if residual is not None:
            raise ValueError("the residual is defined for E4M3 only")
        st = lib().falqon_quantize_e5m2(_ptr(x), dt, rows, cols, _ptr(_u8(codes)), _ptr(scale), _ptr(amax),
                                        _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
        _check(st, "falqon_quantize_e5m2")
        return codes, scale, amax
    if fmt != "e4m3":
        raise ValueError("fmt must be 'e4m3' or 'e5m2'")
    st = lib().falqon_quantize(_ptr(x), dt, rows, cols, _ptr(_u8(codes)), _ptr(scale), _ptr(amax),
                               _ptr(residual), _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_quantize")
    return codes, scale, amax


def falqon_linear_fwd(xq, s_x, wq, s_w, y=None, dev_status=None, stream=None):
    """Y = Xq . Wq^T / (s_x s_w) in bf16."""
    M, K = xq.shape
    N = wq.shape[0]
    dev = xq.device
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    st = lib().falqon_linear_fwd(_ptr(_u8(xq)), _ptr(s_x), _ptr(_u8(wq)), _ptr(s_w), M, N, K,
                                 _ptr(y), _ptr(dev_status), None, 0, _stream(stream, dev))
    _check(st, "falqon_linear_fwd")
    return y


def falqon_linear_fwd_grouped(xq, s_x, wqs, s_ws, ys=None, dev_status=None, stream=None):
    """Y_s = Xq . Wq_s^T / (s_x s_w_s) for up to three backbones that read the
    same Xq, in one launch; returns the list of outputs."""
    M, K = xq.shape
    n = len(wqs)
    dev = xq.device
    if ys is None:
        ys = [torch.empty((M, w.shape[0]), dtype=torch.bfloat16, device=dev) for w in wqs]
    wp = (C.c_void_p * n)(*[_ptr(_u8(w)) for w in wqs])
    sp = (C.c_void_p * n)(*[_ptr(sw) for sw in s_ws])
    yp = (C.c_void_p * n)(*[_ptr(y) for y in ys])
    Ns = (C.c_int64 * n)(*[int(w.shape[0]) for w in wqs])
    st = lib().falqon_linear_fwd_grouped(_ptr(_u8(xq)), _ptr(s_x), n, wp, sp, Ns, yp, M, K, _ptr(dev_status),
                                         _stream(stream, dev))
    _check(st, "falqon_linear_fwd_grouped")
    return ys


def falqon_linear_bwd(dyq, s_dy, wq, s_w, xq, s_x, A, B, dx=True, dA=True, dB=True,
                      dev_status=None, workspace=None, stream=None, dy_fmt="e4m3"):
    """Backward of the melded layer; each output may be True (allocate), a tensor, or None.
    dy_fmt="e5m2": dyq holds E5M2 codes (falqon_quantize(..., fmt="e5m2"))."""
    M, N = dyq.shape
    K = wq.shape[1] if wq is not None else xq.shape[1]
    r = A.shape[0] if A is not None else 0
    dev = dyq.device

    def out(v, shape):
        if v is True:
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return v if v is not None and v is not False else None

    dx_t, dA_t, dB_t = out(dx, (M, K)), out(dA, (r, K)), out(dB, (N, r))
    ws, wsb = (None, 0)
    if dA_t is not None or dB_t is not None:
        ws, wsb = _workspace(OP_LINEAR_BWD, M, N, K, r, dev, workspace)
    if dy_fmt not in ("e4m3", "e5m2"):
        raise ValueError("dy_fmt must be 'e4m3' or 'e5m2'")
    fn = lib().falqon_linear_bwd_e5m2 if dy_fmt == "e5m2" else lib().falqon_linear_bwd
    st = fn(_ptr(_u8(dyq)), _ptr(s_dy), _ptr(None if wq is None else _u8(wq)),
            _ptr(s_w), _ptr(None if xq is None else _u8(xq)), _ptr(s_x),
            _ptr(A), _ptr(B), M, N, K, r, _ptr(dx_t), _ptr(dA_t), _ptr(dB_t),
            _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_linear_bwd_e5m2" if dy_fmt == "e5m2" else "falqon_linear_bwd")
    return dx_t, dA_t, dB_t


def falqon_proxy_update(wq, s_w, proxy, dB_inc, A, flags=PROXY_ACCUMULATE | PROXY_SELECT,
                        row_mask=None, n_selected=None, dev_status=None, workspace=None,
                        stream=None):
    """Row-wise proxy update in place on (wq, proxy); returns (row_mask, n_selected).
    With PROXY_DEFER_CLEAR, row_mask is the caller's: zeros before the first
    call, then the previous call's output (rows it marks read as +0)."""
    N, K = proxy.shape
    r = A.shape[0] if A is not None else 0
    dev = proxy.device
    if flags & PROXY_DEFER_CLEAR and row_mask is None:
        raise ValueError("PROXY_DEFER_CLEAR reads the previous selection: pass row_mask")
    if flags & PROXY_SELECT:
        row_mask = torch.empty(N, dtype=torch.uint8, device=dev) if row_mask is None else row_mask
        n_selected = torch.empty(1, dtype=torch.int32, device=dev) if n_selected is None else n_selected
    ws, wsb = _workspace(OP_PROXY_UPDATE, 0, N, K, r, dev, workspace)
    st = lib().falqon_proxy_update(_ptr(None if wq is None else _u8(wq)), _ptr(s_w), _ptr(proxy),
                                   _ptr(dB_inc), _ptr(A), N, K, r, int(flags), _ptr(row_mask),
                                   _ptr(n_selected), _ptr(dev_status), _ptr(ws), wsb,
                                   _stream(stream, dev))
    _check(st, "falqon_proxy_update")
    return row_mask, n_selected


def falqon_proxy_update_topk(wq, s_w, proxy_q, dB_inc, A, k, flags=PROXY_ACCUMULATE | PROXY_SELECT,
                             comp_mask=None, n_selected=None, dev_status=None, workspace=None, stream=None):
    """Top-k proxy update over the r rank components, in place on (wq, proxy_q);
    proxy_q is float32 [r, N].  Returns (comp_mask, n_selected) (None, None
    without PROXY_SELECT)."""
    r, N = proxy_q.shape
    K = wq.shape[1] if wq is not None else (A.shape[1] if A is not None else 0)
    dev = proxy_q.device
    ws, wsb = (None, 0)
    if flags & PROXY_SELECT:
        comp_mask = torch.empty(r, dtype=torch.uint8, device=dev) if comp_mask is None else comp_mask
        n_selected = torch.empty(1, dtype=torch.int32, device=dev) if n_selected is None else n_selected
        ws, wsb = _workspace(OP_PROXY_UPDATE_TOPK, 0, N, K, r, dev, workspace)
    st = lib().falqon_proxy_update_topk(_ptr(None if wq is None else _u8(wq)), _ptr(s_w), _ptr(proxy_q),
                                        _ptr(dB_inc), _ptr(A), N, K, r, int(k), int(flags), _ptr(comp_mask),
                                        _ptr(n_selected), _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_proxy_update_topk")
    return comp_mask, n_selected


def falqon_linear_bwd_noalloc(dyq, s_dy, wq, s_w, xq, s_x, A, B, dx=True, dA=True, dB=True,
                              dev_status=None, stream=None):
    """falqon_linear_bwd without a workspace: the library's built-in scratch
    array holds the intermediates (for callers that cannot allocate device
    memory).  Outputs follow falqon_linear_bwd; only the outputs themselves
    are allocated here when passed as True."""
    M, N = dyq.shape
    K = wq.shape[1] if wq is not None else xq.shape[1]
    r = A.shape[0] if A is not None else 0
    dev = dyq.device

    def out(v, shape):
        if v is True:
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return v if v is not None and v is not False else None

    dx_t, dA_t, dB_t = out(dx, (M, K)), out(dA, (r, K)), out(dB, (N, r))
    st = lib().falqon_linear_bwd_noalloc(
        _ptr(_u8(dyq)), _ptr(s_dy), _ptr(None if wq is None else _u8(wq)), _ptr(s_w),
        _ptr(None if xq is None else _u8(xq)), _ptr(s_x), _ptr(A), _ptr(B), M, N, K, r,
        _ptr(dx_t), _ptr(dA_t), _ptr(dB_t), _ptr(dev_status), _stream(stream, dev))
    _check(st, "falqon_linear_bwd_noalloc")
    return dx_t, dA_t, dB_t


def falqon_linear_fwd_folded(xq, s_x, wq, s_w, aq, s_a, y=None, t_saved=None, dev_status=None, stream=None):
    """[Y | T] = Xq . [Wq ; A~q]^T in one GEMM (quantized adapter folded into
    the backbone); returns (y, t_saved), t_saved being the uint8 buffer that
    holds T for falqon_linear_bwd_folded (see folded_t_planes)."""
    M, K = xq.shape
    N = wq.shape[0]
    r = aq.shape[0]
    dev = xq.device
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    if t_saved is None:
        t_saved, _ = _workspace(OP_FOLDED_T, M, 0, 0, r, dev, None)
    st = lib().falqon_linear_fwd_folded(_ptr(_u8(xq)), _ptr(s_x), _ptr(_u8(wq)), _ptr(s_w), _ptr(_u8(aq)),
                                        _ptr(s_a), M, N, K, r, _ptr(y), _ptr(t_saved), t_saved.numel(),
                                        _ptr(dev_status), _stream(stream, dev))
    _check(st, "falqon_linear_fwd_folded")
    return y, t_saved


def folded_t_planes(t_saved, M, r):
    """(hi, lo) bfloat16 views [r, ld] of a folded T (or U) buffer: T[m, i] = hi[i, m] + lo[i, m]."""
    ld = (M + 7) // 8 * 8
    plane = (ld * r * 2 + 255) // 256 * 256
    hi = t_saved[:ld * r * 2].view(torch.bfloat16).view(r, ld)
    lo = t_saved[plane:plane + ld * r * 2].view(torch.bfloat16).view(r, ld)
    return hi, lo


def falqon_linear_bwd_folded(dyq, s_dy, wq, s_w, bq, s_b, xq, s_x, t_saved, r, dx=True, dA=True, dB=True,
                             dev_status=None, workspace=None, stream=None):
    """[dX | U] = dYq . [Wq | B~q] in one GEMM, then dB from the forward's T
    and dA from U in one launch; each output may be True (allocate), a
    tensor, or None.  Returns (dx, dA, dB)."""
    M, N = dyq.shape
    K = wq.shape[1] if wq is not None else xq.shape[1]
    dev = dyq.device

    def out(v, shape):
        if v is True:
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return v if v is not None and v is not False else None

    dx_t, dA_t, dB_t = out(dx, (M, K)), out(dA, (r, K)), out(dB, (N, r))
    ws, wsb = (None, 0)
    if dA_t is not None:
        ws, wsb = _workspace(OP_LINEAR_BWD_FOLDED, M, N, K, r, dev, workspace)
    st = lib().falqon_linear_bwd_folded(
        _ptr(_u8(dyq)), _ptr(s_dy), _ptr(None if wq is None else _u8(wq)), _ptr(s_w),
        _ptr(None if bq is None else _u8(bq)), _ptr(s_b), _ptr(None if xq is None else _u8(xq)), _ptr(s_x),
        _ptr(t_saved), 0 if t_saved is None else t_saved.numel(), M, N, K, r, _ptr(dx_t), _ptr(dA_t),
        _ptr(dB_t), _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_linear_bwd_folded")
    return dx_t, dA_t, dB_t


def falqon_selftest_bounded_waits(flag, dev_status, which, stream=None):
    """Launches the library's self-test of its bounded waits (about one
    second): see include/falqon.h."""
    st = lib().falqon_selftest_bounded_waits(_ptr(flag), _ptr(dev_status), _ptr(which),
                                             _stream(stream, flag.device))
    _check(st, "falqon_selftest_bounded_waits")


# ------------------------------------------------------------------ separate LoRA paths (the comparison)
def _a256(v):
    return (v + 255) // 256 * 256


def separate_saved_views(saved, precision, M, N, K, r):
    """Views of the forward's saved buffer: {"S": bf16 [M, r]} and, for the
    FP8 path, "sq" [M, r], "aq" [r, K], "bq" [N, r] codes and "scales" (s_S,
    s_A, s_B) as float32 [3]."""
    o = 0
    v = {"S": saved[o:o + M * r * 2].view(torch.bfloat16).view(M, r)}
    o += _a256(M * r * 2)
    if precision == SEPARATE_FP8:
        v["sq"] = saved[o:o + M * r].view(M, r)
        o += _a256(M * r)
        v["aq"] = saved[o:o + r * K].view(r, K)
        o += _a256(r * K)
        v["bq"] = saved[o:o + N * r].view(N, r)
        o += _a256(N * r)
        v["scales"] = saved[o:o + 12].view(torch.float32)
    return v


def separate_bwd_views(workspace, precision, M, N, r, quantize_ws_bytes):
    """Views of the backward's workspace: "G" bf16 [M, r] and, for the FP8
    path, "gq" [M, r] codes and "s_g" float32 [1]."""
    o = _a256(quantize_ws_bytes)
    v = {"G": workspace[o:o + M * r * 2].view(torch.bfloat16).view(M, r)}
    o += _a256(M * r * 2)
    if precision == SEPARATE_FP8:
        v["gq"] = workspace[o:o + M * r].view(M, r)
        o += _a256(M * r)
    ldt = (M + 15) // 16 * 16
    o += 2 * _a256(ldt * r * (1 if precision == SEPARATE_FP8 else 2)) + _a256(N * r * 2)
    v["s_g"] = workspace[o:o + 4].view(torch.float32)
    return v


def falqon_lora_separate_fwd(precision, xq, s_x, x, wq, s_w, A, B, y=None, saved=None, dev_status=None,
                             workspace=None, stream=None):
    """Separate LoRA path forward (bf16 or FP8 adapter products beside the FP8
    backbone); returns (y, saved)."""
    M, K = xq.shape
    N = wq.shape[0]
    r = A.shape[0]
    dev = xq.device
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    sop = OP_SEPARATE_SAVED_FP8 if precision == SEPARATE_FP8 else OP_SEPARATE_SAVED_BF16
    if saved is None:
        saved, _ = _workspace(sop, M, N, K, r, dev, None)
    ws, wsb = (None, 0)
    if precision == SEPARATE_FP8:
        ws, wsb = _workspace(OP_SEPARATE_FWD_FP8, M, N, K, r, dev, workspace)
    st = lib().falqon_lora_separate_fwd(int(precision), _ptr(_u8(xq)), _ptr(s_x), _ptr(x), _ptr(_u8(wq)), _ptr(s_w),
                                        _ptr(A), _ptr(B), M, N, K, r, _ptr(y), _ptr(saved), saved.numel(),
                                        _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_lora_separate_fwd")
    return y, saved


def falqon_lora_separate_bwd(precision, dyq, s_dy, dy, wq, s_w, xq, s_x, x, A, B, saved, dx=True, dA=True, dB=True,
                             dev_status=None, workspace=None, stream=None):
    """Separate LoRA path backward; each output may be True (allocate), a
    tensor, or None.  Returns (dx, dA, dB)."""
    M, N = dyq.shape
    r, K = A.shape
    dev = dyq.device

    def out(v, shape):
        if v is True:
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return v if v is not None and v is not False else None

    dx_t, dA_t, dB_t = out(dx, (M, K)), out(dA, (r, K)), out(dB, (N, r))
    bop = OP_SEPARATE_BWD_FP8 if precision == SEPARATE_FP8 else OP_SEPARATE_BWD_BF16
    ws, wsb = _workspace(bop, M, N, K, r, dev, workspace)
    st = lib().falqon_lora_separate_bwd(
        int(precision), _ptr(_u8(dyq)), _ptr(s_dy), _ptr(dy), _ptr(None if wq is None else _u8(wq)), _ptr(s_w),
        _ptr(None if xq is None else _u8(xq)), _ptr(s_x), _ptr(x), _ptr(A), _ptr(B), _ptr(saved), saved.numel(),
        M, N, K, r, _ptr(dx_t), _ptr(dA_t), _ptr(dB_t), _ptr(dev_status), _ptr(ws), wsb, _stream(stream, dev))
    _check(st, "falqon_lora_separate_bwd")
    return dx_t, dA_t, dB_t


# ------------------------------------------------------------------ around the linear layer
# Small calls take the GPU two to five microseconds, so these bindings are
# written to spend little more on the host: one check per tensor, integers for
# pointers, no context managers where the tensors' device and stream are
# current.
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _elsewhere(dev, stream):
    """A scope that makes `dev` and the caller's stream current, or None where
    they are: what is allocated then belongs to the stream that the call runs on."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is of {stream.device}, the tensors are on {dev}")
        return torch.cuda.stream(stream)  # also selects the stream's device
    return None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _addr(t, name, shape, dtypes, dev):
    """The address of a tensor that the call takes `shape` elements of `dtypes` at; None for None."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_F32, _BF16, _EITHER, _I32 = (torch.float32,), (torch.bfloat16,), (torch.bfloat16, torch.float32), (torch.int32,)


def _scalar(t, name, dev):
    """The address of one float (a scale), of any shape."""
    return _addr(t, name, t.shape if t.numel() == 1 else (1,), _F32, dev)


def _device_of(t, name, dtypes):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError("falqon tensors must live on a CUDA device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.device


def _like(v, name, t, dev):
    """(tensor, address) of an output with the shape and type of `t`: True
    (allocate), a tensor, or None (not wanted)."""
    if v is True:
        v = torch.empty_like(t)
        return v, v.data_ptr()
    return (None, None) if v is None or v is False else (v, _addr(v, name, t.shape, (t.dtype,), dev))


def _vector(v, name, n, t, dev):
    """The same for `n` float32 beside `t`."""
    if v is True:
        v = t.new_empty((n,), dtype=torch.float32)
        return v, v.data_ptr()
    return (None, None) if v is None or v is False else (v, _addr(v, name, (n,), _F32, dev))


def _scratch(op, M, N, K, dev, workspace):
    """(tensor, address, bytes) of a workspace that needs no initialisation: the caller's, or one of this call."""
    if workspace is None:
        need = falqon_workspace_size(op, M, N, K, 0)
        raw = torch.empty(need + 256, dtype=torch.uint8, device=dev)
        return raw, raw.data_ptr() + (-raw.data_ptr()) % 256, need
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _status(dev_status, dev):
    return None if dev_status is None else _addr(dev_status, "dev_status", dev_status.shape, _I32, dev)


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev.index)


def falqon_norm_fwd(x, gamma=None, beta=None, eps=1e-5, kind=NORM_LAYER, y=True, mean=True, rstd=True,
                    dev_status=None, stream=None):
    """Layer norm (or RMS norm: kind=NORM_RMS, no beta) of each row of x [rows,
    cols], bf16 or fp32; returns (y, mean, rstd).  mean and rstd (float32
    [rows], what falqon_norm_bwd reads) may be True (allocate), a tensor, or
    None; mean is None for NORM_RMS."""
    dev = _device_of(x, "x", _EITHER)
    scope = _elsewhere(dev, stream)
    if scope is not None:
        with scope:
            return falqon_norm_fwd(x, gamma, beta, eps, kind, y, mean, rstd, dev_status)
    shape = x.shape
    rows, cols = shape
    dtype = x.dtype
    param = gamma if gamma is not None else beta
    pdtypes = _EITHER if param is None else (param.dtype,)
    if param is not None and param.dtype not in _DTYPES:
        raise ValueError(f"gamma and beta must be bfloat16 or float32, got {param.dtype}")
    xp = _addr(x, "x", shape, (dtype,), dev)
    y, yp = _like(True if y is None else y, "y", x, dev)
    mean, mp = _vector(None if kind == NORM_RMS and mean is True else mean, "mean", rows, x, dev)
    rstd, rp = _vector(rstd, "rstd", rows, x, dev)
    st = lib().falqon_norm_fwd(
        xp, _DTYPES[dtype], _addr(gamma, "gamma", (cols,), pdtypes, dev),
        _addr(beta, "beta", (cols,), pdtypes, dev), DTYPE_BF16 if param is None else _DTYPES[param.dtype], kind, rows,
        cols, eps, yp, mp, rp, _status(dev_status, dev), _raw_stream(dev))
    _check(st, "falqon_norm_fwd")
    return y, mean, rstd


def falqon_norm_bwd(dy, x, gamma, mean, rstd, kind=NORM_LAYER, dres=None, dx=True, dgamma=True, dbeta=True,
                    dev_status=None, workspace=None, stream=None):
    """Backward of falqon_norm_fwd; dres (nullable) joins dx.  Each output may
    be True (allocate), a tensor, or None; dgamma and dbeta are float32 sums,
    dbeta is None for NORM_RMS.  Returns (dx, dgamma, dbeta)."""
    dev = _device_of(x, "x", _EITHER)
    scope = _elsewhere(dev, stream)
    if scope is not None:
        with scope:
            return falqon_norm_bwd(dy, x, gamma, mean, rstd, kind, dres, dx, dgamma, dbeta, dev_status, workspace)
    shape = x.shape
    rows, cols = shape
    dtype = x.dtype
    own = (dtype,)
    xp = _addr(x, "x", shape, own, dev)
    dx, dxp = _like(dx, "dx", x, dev)
    dgamma, dgp = _vector(dgamma, "dgamma", cols, x, dev)
    dbeta, dbp = _vector(None if kind == NORM_RMS and dbeta is True else dbeta, "dbeta", cols, x, dev)
    ws, wsp, wsb = (None, None, 0)
    if dgamma is not None or dbeta is not None:
        ws, wsp, wsb = _scratch(OP_NORM_BWD, rows, 0, cols, dev, workspace)
    st = lib().falqon_norm_bwd(
        _addr(dy, "dy", shape, own, dev), xp, _DTYPES[dtype],
        _addr(gamma, "gamma", (cols,), _EITHER, dev), DTYPE_BF16 if gamma is None else _DTYPES[gamma.dtype], kind,
        _addr(mean, "mean", (rows,), _F32, dev), _addr(rstd, "rstd", (rows,), _F32, dev),
        _addr(dres, "dres", shape, own, dev), rows, cols, dxp, dgp, dbp, _status(dev_status, dev), wsp, wsb,
        _raw_stream(dev))
    _check(st, "falqon_norm_bwd")
    return dx, dgamma, dbeta


def falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias=None, act=ACT_NONE, residual=None, z=None, y=True,
                               dev_status=None, stream=None):
    """Y = act(Xq . Wq^T / (s_x s_w) + bias) + residual in bf16; returns (y, z).
    z, the pre-activation in bf16 for falqon_linear_epilogue_bwd, may be True
    (allocate), a tensor, or None."""
    dev = _device_of(xq, "xq", _CODES)
    scope = _elsewhere(dev, stream)
    if scope is not None:
        with scope:
            return falqon_linear_fwd_epilogue(xq, s_x, wq, s_w, bias, act, residual, z, y, dev_status)
    if wq.dim() != 2:
        raise ValueError("wq must be 2-D")
    M, K = xq.shape
    N = wq.shape[0]
    out = (M, N)
    if y is True or y is None:
        y = xq.new_empty(out, dtype=torch.bfloat16)
        yp = y.data_ptr()
    else:
        yp = _addr(y, "y", out, _BF16, dev)
    z, zp = _like(z, "z", y, dev)
    st = lib().falqon_linear_fwd_epilogue(
        _addr(xq, "xq", (M, K), _CODES, dev), _scalar(s_x, "s_x", dev), _addr(wq, "wq", (N, K), _CODES, dev),
        _scalar(s_w, "s_w", dev), _addr(bias, "bias", (N,), _EITHER, dev),
        DTYPE_BF16 if bias is None else _DTYPES[bias.dtype], act, _addr(residual, "residual", out, _BF16, dev), M, N, K,
        zp, yp, _status(dev_status, dev), _raw_stream(dev))
    _check(st, "falqon_linear_fwd_epilogue")
    return y, z


def falqon_linear_epilogue_bwd(dy, z, act, dz=True, dbias=True, workspace=None, stream=None):
    """dZ = dY act'(Z) in bf16 and dbias, its column sums in float32; each may
    be True (allocate), a tensor, or None.  z may be None for ACT_NONE, whose
    dZ is dY.  Returns (dz, dbias)."""
    dev = _device_of(dy, "dy", _BF16)
    scope = _elsewhere(dev, stream)
    if scope is not None:
        with scope:
            return falqon_linear_epilogue_bwd(dy, z, act, dz, dbias, workspace)
    shape = dy.shape
    M, N = shape
    dyp = _addr(dy, "dy", shape, _BF16, dev)
    dz, dzp = _like(dz, "dz", dy, dev)
    dbias, dbp = _vector(dbias, "dbias", N, dy, dev)
    ws, wsp, wsb = (None, None, 0)
    if dbias is not None:
        ws, wsp, wsb = _scratch(OP_LINEAR_EPILOGUE_BWD, M, N, 0, dev, workspace)
    st = lib().falqon_linear_epilogue_bwd(
        dyp, _addr(z, "z", shape, _BF16, dev), act, M, N, dzp, dbp, wsp, wsb, _raw_stream(dev))
    _check(st, "falqon_linear_epilogue_bwd")
    return dz, dbias


class _Tensors:
    """Tensors (bf16 or float32, contiguous, on one device) marshalled for one call."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("no tensors")
        self.device = self.tensors[0].device
        for t in self.tensors:
            if t.dtype not in _DTYPES:
                raise ValueError(f"gradients must be bfloat16 or float32, got {t.dtype}")
            if t.device != self.device:
                raise ValueError(f"gradients on {self.device} and {t.device}")
        n = len(self.tensors)
        self.pointers = (C.c_void_p * n)(*[_ptr(t) for t in self.tensors])
        self.numel = (C.c_int64 * n)(*[t.numel() for t in self.tensors])
        self.dtypes = (C.c_int * n)(*[_DTYPES[t.dtype] for t in self.tensors])

    def current(self):
        return self

    def __len__(self):
        return len(self.tensors)

    def __iter__(self):
        return iter(self.tensors)


class GradList(_Tensors):
    """Tensors (bf16 or float32, contiguous, on one device) marshalled once for
    many calls of falqon_clip_grads: a training loop whose gradient buffers stay
    where they are builds it at its start.

    The list stands for the memory that the tensors have when it is built, and
    keeps it: gradients that get other memory later (a new .grad every step,
    `data =`, set_) need a new list, as they need a new CUDA graph.  Memory that
    resize_ moves is followed, memory that it gives back is refused
    (ValueError); each call looks at the address of every storage, of which a
    flat buffer is one."""

    def __init__(self, tensors):
        super().__init__(tensors)
        at = {}  # storage -> its place in _storages
        self._storages, self._where = [], []
        for t in self.tensors:
            s = t.untyped_storage()
            k = at.setdefault(s._cdata, len(at))
            if k == len(self._storages):
                self._storages.append(s)
            # (storage, first byte, end) of each tensor; one without elements has no memory
            first = t.storage_offset() * t.element_size()
            self._where.append((k, first, first + t.numel() * t.element_size()) if t.numel() else None)
        self._bases = [s.data_ptr() for s in self._storages]

    def current(self):
        """This list, with the addresses that its memory has now."""
        bases = [s.data_ptr() for s in self._storages]
        if bases != self._bases:
            sizes = [s.nbytes() for s in self._storages]
            if any(w and w[2] > sizes[w[0]] for w in self._where):
                raise ValueError("memory of a GradList has been given back")
            for i, w in enumerate(self._where):
                self.pointers[i] = bases[w[0]] + w[1] if w else None
            self._bases = bases
        return self


def falqon_clip_grads(grads, max_norm, factor=1.0, out=None, norm=None, coef=None, dev_status=None, workspace=None,
                      stream=None):
    """The global norm of `grads` (tensors, or a GradList of them), and, where
    `out` is wanted, the gradients times factor * min(1, max_norm / norm).
    out: None (the norm alone), True (allocate), or tensors / a GradList of the
    same sizes and types, which may be `grads` itself (in place).  Returns
    (out, norm, coef), norm and coef being float32 [1]."""
    g = grads.current() if isinstance(grads, _Tensors) else _Tensors(grads)
    dev = g.device
    scope = _elsewhere(dev, stream)
    if scope is not None:
        with scope:
            return falqon_clip_grads(g, max_norm, factor, g if out is grads else out, norm, coef, dev_status, workspace)
    o = out
    if out is True:
        o = _Tensors(torch.empty_like(t) for t in g)
    elif out is grads:
        o = g
    elif out is not None:
        o = out.current() if isinstance(out, _Tensors) else _Tensors(out)
    if o is not None and o is not g:
        if len(o) != len(g) or o.device != dev or bytes(o.numel) != bytes(g.numel) or \
                bytes(o.dtypes) != bytes(g.dtypes):
            raise ValueError("out must match grads in number, sizes, types and device")
    norm, np_ = _vector(True if norm is None else norm, "norm", 1, g.tensors[0], dev)
    coef, cp = _vector(True if coef is None else coef, "coef", 1, g.tensors[0], dev)
    ws, wsp, wsb = _scratch(OP_CLIP_GRADS, 0, 0, 0, dev, workspace)
    st = lib().falqon_clip_grads(len(g), g.pointers, g.dtypes, g.numel, max_norm, factor,
                                 None if o is None else o.pointers, np_, cp, _status(dev_status, dev), wsp, wsb,
                                 _raw_stream(dev))
    _check(st, "falqon_clip_grads")
    return (None if o is None else o.tensors), norm, coef
