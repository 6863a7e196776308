"""Binding of libmoe.so (include/moe.h).

Argument marshalling only: tensors are checked for device/dtype/shape and
handed over as raw pointers together with torch's current HIP stream; every
step of the layer runs in the library's kernels.  The checks and the calls
themselves are native (csrc/marshal.cpp, _marshal.so), the rest is ctypes.
There is no fallback: if a library is missing or a call fails, an exception
says so.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")
MARSHAL_PATH = os.path.join(HERE, "_marshal.so")

MOE_OK = 0
F32, BF16, FP8_E4M3, MXFP4 = 0, 1, 2, 3
ROUTE_DEFAULT, ROUTE_RENORMALIZE, ROUTE_DEEPSEEKV3, ROUTE_RENORMALIZE_NAIVE = 0, 1, 2, 4
ROUTE_FLAG_RENORMALIZE = 1
KERNEL_IDS = ["route", "permute_count", "permute_scan", "permute_scatter", "fc1", "fc2",
              "finalize", "quantize", "ffn_fused", "permute_one", "rmsnorm", "rmsnorm_backward",
              "rmsnorm_dweight", "dispatch", "dispatch_backward", "finalize_backward",
              "route_backward", "swiglu", "swiglu_backward", "quantize_mxfp4",
              "dequantize_mxfp4", "few_fc1", "few_fc2"]
FUSED_MAX_I = 2048
NOALLOC_SCRATCH_BYTES = 64 << 20
FEW_MAX_T = 32

# The 4-bit types; None in a torch that has none of these names.
_CODES, _SCALES = getattr(torch, "float4_e2m1fn_x2", None), getattr(torch, "float8_e8m0fnu", None)
_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: FP8_E4M3}
if _CODES is not None:
    _DT[_CODES] = MXFP4
_lib = None
_marshal = None
_loading = threading.Lock()


class MoeError(RuntimeError):
    def __init__(self, fn, status, reason):
        super().__init__(f"{fn} failed: {status_string(status)} ({reason})")
        self.status = status


def lib():
    """The loaded libmoe.so with argument types set (raises if not built)."""
    if _lib is None:
        with _loading:  # threads that make their first call together load once
            if _lib is None:
                _load()
    return _lib


def _load():
    global _lib, _marshal, _dev
    for path in (LIB_PATH, MARSHAL_PATH):
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run "
                               "`python -m mixture_experts_layer_07_amd.build`")
    L = C.CDLL(LIB_PATH)
    P, i, u, f, z = C.c_void_p, C.c_int, C.c_uint, C.c_float, C.c_size_t
    L.moe_route.argtypes = [P, i, i, i, i, i, i, P, f, u, P, P, P]
    L.moe_permute.argtypes = [P, i, i, i, i, P, P, P, P, z, P]
    L.moe_expert_ffn.argtypes = [P, i, i, i, i, i, i, i, P, P, P, P, i, P, P, P, P, z, P]
    L.moe_finalize.argtypes = [P, i, P, P, i, i, i, i, P, i, P]
    L.moe_quantize_fp8.argtypes = [P, i, i, i, P, P, P]
    L.moe_expert_ffn_fp8.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P, P, P, P, P, z, P]
    L.moe_expert_ffn_noalloc.argtypes = [P, i, i, i, i, i, i, i, P, P, P, P, i, P, P, P, P]
    L.moe_expert_ffn_fused.argtypes = [P, i, i, i, i, i, i, i, P, P, P, P, i, P, P, i, P, P]
    L.moe_expert_ffn_fp8_fused.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P, P, P, i, P, P]
    L.moe_rmsnorm.argtypes = [P, P, P, i, i, i, f, P, P, P, P, P]
    L.moe_rmsnorm_backward.argtypes = [P, P, P, P, i, i, i, f, P, P, P, z, P]
    L.moe_rmsnorm_backward_workspace_size.argtypes = [i, i]
    L.moe_rmsnorm_backward_workspace_size.restype = z
    L.moe_dispatch.argtypes = [P, P, i, i, i, i, i, P, P, P, P]
    L.moe_dispatch_backward.argtypes = [P, i, P, i, i, i, i, P, i, P]
    L.moe_finalize_backward.argtypes = [P, i, P, i, P, P, i, i, i, i, P, P, P]
    L.moe_route_backward.argtypes = [P, P, P, i, i, i, i, f, u, P, P]
    L.moe_swiglu.argtypes = [P, i, i, i, P, P, P, P, P, P]
    L.moe_swiglu_backward.argtypes = [P, i, P, P, i, i, P, P, P]
    L.moe_quantize_mxfp4.argtypes = [P, i, i, i, P, P, P]
    L.moe_dequantize_mxfp4.argtypes = [P, P, i, i, i, P, P]
    L.moe_expert_ffn_mxfp4.argtypes = [P, P, i, i, i, i, i, i, P, P, P, P, P, P, P, P, z, P]
    L.moe_layer_few.argtypes = [P, i, P, i, i, i, i, i, i, i, i, P, f, u, i, P, P, i, P, P, P, P, P, P, z, P]
    L.moe_layer_few_workspace_size.argtypes = [i, i, i, i, i, i, i]
    L.moe_layer_few_workspace_size.restype = z
    L.moe_workspace_size.argtypes = [i, i, i, i, i, i, i]
    L.moe_workspace_size.restype = z
    L.moe_status_string.argtypes = [i]
    L.moe_status_string.restype = C.c_char_p
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = C.c_char_p
    L.moe_timing_enable.argtypes = [i]
    L.moe_kernel_times.argtypes = [P, P, i]
    for fn in ("moe_route", "moe_permute", "moe_expert_ffn", "moe_expert_ffn_noalloc", "moe_finalize",
               "moe_quantize_fp8", "moe_expert_ffn_fp8", "moe_expert_ffn_fused",
               "moe_expert_ffn_fp8_fused", "moe_rmsnorm", "moe_rmsnorm_backward",
               "moe_dispatch", "moe_dispatch_backward", "moe_finalize_backward",
               "moe_route_backward", "moe_swiglu", "moe_swiglu_backward", "moe_quantize_mxfp4",
               "moe_dequantize_mxfp4", "moe_expert_ffn_mxfp4", "moe_layer_few",
               "moe_timing_enable", "moe_kernel_times"):
        getattr(L, fn).restype = C.c_int
    from . import _marshal as native
    native.setup(lambda fn: C.cast(getattr(L, fn), C.c_void_p).value, _failed, _refuse)
    _marshal, _dev = native, native.check
    _lib = L  # last: where it is set, the rest is


def status_string(st: int) -> str:
    return lib().moe_status_string(int(st)).decode()


def last_error() -> str:
    return lib().moe_last_error().decode()


def _failed(fn: str, st: int):
    raise MoeError(fn, st, last_error())


def _check(fn: str, st: int):
    if st != MOE_OK:
        _failed(fn, st)


def _call(fn: str, device, *args):
    """Calls library entry `fn` with `device` current and its current stream
    appended; tensor arguments become device pointers and must all live on
    `device` (the kernels run on the current device)."""
    if _lib is None:
        lib()
    _marshal.call(fn, device if isinstance(device, torch.device) else torch.device(device), *args)


def _refuse(t, name, dtype, shape):
    """Says what _dev found."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None):
    """t if it is a contiguous GPU tensor of that dtype (or one of a tuple of
    dtypes) and shape.  lib() puts the native form in this one's place."""
    lib()
    return _marshal.check(t, name, dtype, shape)


def dtype_code(dt: torch.dtype) -> int:
    return _DT[dt]


def workspace_size(T, k, E, n_shared, H, I, act_dtype) -> int:
    """act_dtype torch.float8_e4m3fn sizes the workspace of expert_ffn_fp8, torch.float4_e2m1fn_x2
    that of expert_ffn_mxfp4."""
    return int(lib().moe_workspace_size(T, k, E, n_shared, H, I, _DT[act_dtype]))


def alloc_workspace(T, k, E, n_shared, H, I, act_dtype, device="cuda") -> torch.Tensor:
    n = workspace_size(T, k, E, n_shared, H, I, act_dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------- calls
def route(logits, k, method, n_group=1, topk_group=1, bias=None, scaling=1.0,
          renormalize=False, out=None):
    """moe_route -> (ids int32 [T,k], scales fp32 [T,k])."""
    _dev(logits, "logits", torch.float32)
    T, E = logits.shape
    if bias is not None:
        _dev(bias, "bias", torch.float32, (E,))
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        scales = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    else:
        ids, scales = out
        _dev(ids, "ids", torch.int32, (T, k))
        _dev(scales, "scales", torch.float32, (T, k))
    flags = ROUTE_FLAG_RENORMALIZE if renormalize else 0
    _call("moe_route", logits.device, logits, T, E, method, k, n_group, topk_group, bias,
          float(scaling), flags, ids, scales)
    return ids, scales


def permute(ids, E, n_shared=0, ws=None, out=None):
    """moe_permute -> (expert_offsets [E+n_shared+1], permuted_pair [T*k], unpermute [T*k])."""
    _dev(ids, "ids", torch.int32)
    T, k = ids.shape
    d = ids.device
    if out is None:
        off = torch.empty(E + n_shared + 1, dtype=torch.int32, device=d)
        pp = torch.empty(T * k, dtype=torch.int32, device=d)
        up = torch.empty(T * k, dtype=torch.int32, device=d)
    else:
        off, pp, up = out
        _dev(off, "expert_offsets", torch.int32, (E + n_shared + 1,))
        _dev(pp, "permuted_pair", torch.int32, (T * k,))
        _dev(up, "unpermute", torch.int32, (T * k,))
    if ws is None:
        ws = alloc_workspace(T, k, E, n_shared, 128, 128, torch.bfloat16, d)
    _dev(ws, "ws", torch.uint8)
    _call("moe_permute", d, ids, T, k, E, n_shared, off, pp, up, ws, ws.numel())
    return off, pp, up


def expert_ffn(x, expert_offsets, permuted_pair, w13, w2, k, E, n_shared=0, w13_scale=None,
               w2_scale=None, ws=None, out=None):
    """moe_expert_ffn -> fc2_out [T*k + n_shared*T, H] in x's dtype."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, H = x.shape
    G = E + n_shared
    _dev(w13, "w13", (torch.float32, torch.bfloat16, torch.float8_e4m3fn))
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, H))
    _dev(w2, "w2", w13.dtype, (G, H, I))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    if w13.dtype == torch.float8_e4m3fn:
        _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
        _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    R = T * k + n_shared * T
    if out is None:
        out = torch.empty((R, H), dtype=x.dtype, device=x.device)
    else:
        _dev(out, "fc2_out", x.dtype, (R, H))
    if ws is None:
        ws = alloc_workspace(T, k, E, n_shared, H, I, x.dtype, x.device)
    _dev(ws, "ws", torch.uint8)
    _call("moe_expert_ffn", x.device, x, _DT[x.dtype], T, H, I, k, E, n_shared, expert_offsets,
          permuted_pair, w13, w2, _DT[w13.dtype], w13_scale, w2_scale, out, ws, ws.numel())
    return out


def expert_ffn_noalloc(x, expert_offsets, permuted_pair, w13, w2, k, E, n_shared=0,
                       w13_scale=None, w2_scale=None, out=None):
    """moe_expert_ffn_noalloc: expert_ffn with h in the library's static device
    scratch (no workspace; MOE_NOALLOC_SCRATCH_BYTES bounds h) -> fc2_out."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    T, H = x.shape
    G = E + n_shared
    _dev(w13, "w13", (torch.float32, torch.bfloat16, torch.float8_e4m3fn))
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, H))
    _dev(w2, "w2", w13.dtype, (G, H, I))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    if w13.dtype == torch.float8_e4m3fn:
        _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
        _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    R = T * k + n_shared * T
    if out is None:
        out = torch.empty((R, H), dtype=x.dtype, device=x.device)
    else:
        _dev(out, "fc2_out", x.dtype, (R, H))
    _call("moe_expert_ffn_noalloc", x.device, x, _DT[x.dtype], T, H, I, k, E, n_shared,
          expert_offsets, permuted_pair, w13, w2, _DT[w13.dtype], w13_scale, w2_scale, out)
    return out


def quantize_fp8(x, out=None):
    """moe_quantize_fp8 -> (xq float8_e4m3fn [rows, cols], x_scale fp32 [rows, cols/128])."""
    _dev(x, "x", (torch.float32, torch.bfloat16))
    rows, cols = x.shape
    if out is None:
        xq = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=x.device)
        xs = torch.empty((rows, cols // 128), dtype=torch.float32, device=x.device)
    else:
        xq, xs = out
        _dev(xq, "xq", torch.float8_e4m3fn, (rows, cols))
        _dev(xs, "x_scale", torch.float32, (rows, cols // 128))
    _call("moe_quantize_fp8", x.device, x, _DT[x.dtype], rows, cols, xq, xs)
    return xq, xs


def expert_ffn_fp8(xq, x_scale, expert_offsets, permuted_pair, w13, w2, w13_scale, w2_scale, k, E,
                   n_shared=0, ws=None, out=None):
    """moe_expert_ffn_fp8 -> fc2_out bf16 [T*k + n_shared*T, H]."""
    _dev(xq, "xq", torch.float8_e4m3fn)
    T, H = xq.shape
    _dev(x_scale, "x_scale", torch.float32, (T, H // 128))
    G = E + n_shared
    _dev(w13, "w13", torch.float8_e4m3fn)
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, H))
    _dev(w2, "w2", torch.float8_e4m3fn, (G, H, I))
    _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
    _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    R = T * k + n_shared * T
    if out is None:
        out = torch.empty((R, H), dtype=torch.bfloat16, device=xq.device)
    else:
        _dev(out, "fc2_out", torch.bfloat16, (R, H))
    if ws is None:
        ws = alloc_workspace(T, k, E, n_shared, H, I, torch.float8_e4m3fn, xq.device)
    _dev(ws, "ws", torch.uint8)
    _call("moe_expert_ffn_fp8", xq.device, xq, x_scale, T, H, I, k, E, n_shared, expert_offsets,
          permuted_pair, w13, w2, w13_scale, w2_scale, out, ws, ws.numel())
    return out


def expert_ffn_fused(x, expert_offsets, permuted_pair, w13, w2, k, E, n_shared=0, w13_scale=None,
                     w2_scale=None, split=0, out=None):
    """moe_expert_ffn_fused (one kernel, h kept on chip) -> fc2_out bf16
    [T*k + n_shared*T, H]; same results as expert_ffn, no workspace."""
    _dev(x, "x", torch.bfloat16)
    T, H = x.shape
    G = E + n_shared
    _dev(w13, "w13", (torch.bfloat16, torch.float8_e4m3fn))
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, H))
    _dev(w2, "w2", w13.dtype, (G, H, I))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    if w13.dtype == torch.float8_e4m3fn:
        _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
        _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    R = T * k + n_shared * T
    if out is None:
        out = torch.empty((R, H), dtype=torch.bfloat16, device=x.device)
    else:
        _dev(out, "fc2_out", torch.bfloat16, (R, H))
    _call("moe_expert_ffn_fused", x.device, x, BF16, T, H, I, k, E, n_shared, expert_offsets,
          permuted_pair, w13, w2, _DT[w13.dtype], w13_scale, w2_scale, int(split), out)
    return out


def expert_ffn_fp8_fused(xq, x_scale, expert_offsets, permuted_pair, w13, w2, w13_scale, w2_scale,
                         k, E, n_shared=0, split=0, out=None):
    """moe_expert_ffn_fp8_fused -> fc2_out bf16 [T*k + n_shared*T, H]; same results as
    expert_ffn_fp8, no workspace."""
    _dev(xq, "xq", torch.float8_e4m3fn)
    T, H = xq.shape
    _dev(x_scale, "x_scale", torch.float32, (T, H // 128))
    G = E + n_shared
    _dev(w13, "w13", torch.float8_e4m3fn)
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, H))
    _dev(w2, "w2", torch.float8_e4m3fn, (G, H, I))
    _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
    _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    R = T * k + n_shared * T
    if out is None:
        out = torch.empty((R, H), dtype=torch.bfloat16, device=xq.device)
    else:
        _dev(out, "fc2_out", torch.bfloat16, (R, H))
    _call("moe_expert_ffn_fp8_fused", xq.device, xq, x_scale, T, H, I, k, E, n_shared,
          expert_offsets, permuted_pair, w13, w2, w13_scale, w2_scale, int(split), out)
    return out


def finalize(fc2_out, unpermute, scales, n_shared=0, out_dtype=None, out=None):
    """moe_finalize -> y [T, H]."""
    _dev(fc2_out, "fc2_out", (torch.float32, torch.bfloat16))
    _dev(scales, "scales", torch.float32)
    T, k = scales.shape
    _dev(unpermute, "unpermute", torch.int32, (T * k,))
    R, H = fc2_out.shape
    if R != T * k + n_shared * T:
        raise ValueError(f"fc2_out has {R} rows, expected {T * k + n_shared * T}")
    ydt = out_dtype or fc2_out.dtype
    if out is None:
        out = torch.empty((T, H), dtype=ydt, device=fc2_out.device)
    else:
        _dev(out, "y", ydt, (T, H))
    _call("moe_finalize", fc2_out.device, fc2_out, _DT[fc2_out.dtype], unpermute, scales, T, k, H,
          n_shared, out, _DT[ydt])
    return out


# ----------------------------------------------------------- row operators
# None of them records a graph.  With gradients enabled, rmsnorm, dispatch and swiglu warn
# (UserWarning) of a tensor that requires grad: their results are constants to autograd.  A training
# program calls the backward functions itself, for example from a torch.autograd.Function, whose
# forward and backward run with gradients disabled.
def _out(t, name, shape, dtype, device):
    """The caller's output buffer `t`, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _dev(t, name, dtype, shape)


def _rows_of(x, name, dtype):
    _dev(x, name, dtype)
    if x.dim() != 2:
        raise ValueError(f"{name} must be [rows, columns] (got {tuple(x.shape)})")
    return x.shape


def _places(unpermute, k):
    """T of a moe_permute result."""
    _dev(unpermute, "unpermute", torch.int32)
    if k < 1 or unpermute.dim() != 1 or unpermute.numel() % k:
        raise ValueError(f"unpermute must be [T * k] (got {tuple(unpermute.shape)}, k = {k})")
    return unpermute.numel() // k


def _unused(names, given):
    for name, t in zip(names, given):
        if t is not None:
            raise ValueError(f"out: {name} is not an output of this call")


_ACT = (torch.float32, torch.bfloat16)


def rmsnorm(x, weight, eps=1e-6, residual=None, quantize=False, want_y=True, out=None):
    """moe_rmsnorm -> (y, total, yq, y_scale): y = rmsnorm(total) * weight with total = x + residual
    (None without a residual), and with quantize the e4m3 codes and 1x128 scales of y that
    expert_ffn_fp8 takes (else None, None).  want_y=False writes the codes alone (y None).
    `out` is the same tuple of buffers; out's total may be x or residual."""
    T, H = _rows_of(x, "x", _ACT)
    dt, d = x.dtype, x.device
    _dev(weight, "weight", dt, (H,))
    if residual is not None:
        _dev(residual, "residual", dt, (T, H))
    y, total, yq, ys = (None,) * 4 if out is None else out
    if want_y:
        y = _out(y, "y", (T, H), dt, d)
    else:
        _unused(("y",), (y,))
    if residual is not None:
        total = _out(total, "total", (T, H), dt, d)
    else:
        _unused(("total",), (total,))
    if quantize:
        yq = _out(yq, "yq", (T, H), torch.float8_e4m3fn, d)
        ys = _out(ys, "y_scale", (T, H // 128), torch.float32, d)
    else:
        _unused(("yq", "y_scale"), (yq, ys))
    _call("moe_rmsnorm", d, x, residual, weight, _DT[dt], T, H, float(eps), total, y, yq, ys)
    return y, total, yq, ys


def rmsnorm_backward_workspace(T, H, device="cuda") -> torch.Tensor:
    n = int(lib().moe_rmsnorm_backward_workspace_size(T, H))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def rmsnorm_backward(dy, z, weight, eps=1e-6, dsum=None, ws=None, out=None):
    """moe_rmsnorm_backward -> (dz [T, H], dweight fp32 [H]): z is rmsnorm's total (x without a
    residual), dz the gradient of x and of the residual alike, dsum the gradient that reaches z
    through the residual stream.  out's dz may be dy or dsum."""
    T, H = _rows_of(z, "z", _ACT)
    dt, d = z.dtype, z.device
    _dev(dy, "dy", dt, (T, H))
    _dev(weight, "weight", dt, (H,))
    if dsum is not None:
        _dev(dsum, "dsum", dt, (T, H))
    dz, dw = (None, None) if out is None else out
    dz = _out(dz, "dz", (T, H), dt, d)
    dw = _out(dw, "dweight", (H,), torch.float32, d)
    if ws is None:
        ws = rmsnorm_backward_workspace(T, H, d)
    _dev(ws, "ws", torch.uint8)
    _call("moe_rmsnorm_backward", d, dy, z, weight, dsum, _DT[dt], T, H, float(eps), dz, dw, ws, ws.numel())
    return dz, dw


def dispatch(x, unpermute, k, n_shared=0, x_scale=None, out=None):
    """moe_dispatch -> rows [T*k + n_shared*T, H] in expert order; for e4m3 codes x with their
    x_scale -> (rows, rows_scale), and `out` is such a pair.  Rows that no pair names (unpermute
    entries outside [0, T*k) are dropped) are not written: a new tensor holds anything there."""
    T, H = _rows_of(x, "x", (torch.float32, torch.bfloat16, torch.float8_e4m3fn))
    d, fp8 = x.device, x.dtype == torch.float8_e4m3fn
    if _places(unpermute, k) != T:
        raise ValueError(f"unpermute has {unpermute.numel()} pairs, expected {T * k}")
    R = T * k + n_shared * T
    if fp8 != (x_scale is not None):
        raise ValueError("x_scale goes with float8_e4m3fn x, and only with it")
    scale = None
    if fp8:
        _dev(x_scale, "x_scale", torch.float32, (T, H // 128))
        out, scale = (None, None) if out is None else out
        scale = _out(scale, "rows_scale", (R, H // 128), torch.float32, d)
    out = _out(out, "rows", (R, H), x.dtype, d)
    _call("moe_dispatch", d, x, x_scale, _DT[x.dtype], T, H, k, n_shared, unpermute, out, scale)
    return (out, scale) if fp8 else out


def dispatch_backward(d_rows, unpermute, k, n_shared=0, out_dtype=None, out=None):
    """moe_dispatch_backward -> dx [T, H]: each token's rows summed."""
    R, H = _rows_of(d_rows, "d_rows", _ACT)
    T = _places(unpermute, k)
    if R != T * k + n_shared * T:
        raise ValueError(f"d_rows has {R} rows, expected {T * k + n_shared * T}")
    dt = out_dtype or d_rows.dtype
    out = _out(out, "dx", (T, H), dt, d_rows.device)
    _call("moe_dispatch_backward", d_rows.device, d_rows, _DT[d_rows.dtype], unpermute, T, k, H,
          n_shared, out, _DT[dt])
    return out


def finalize_backward(dy, fc2_out, unpermute, scales, n_shared=0, out=None):
    """moe_finalize_backward -> (d_fc2 [T*k + n_shared*T, H] in fc2_out's dtype, d_scales fp32 [T, k]).
    out's d_fc2 may be fc2_out.  Rows that no pair names are not written, as in dispatch."""
    _dev(scales, "scales", torch.float32)
    T, k = scales.shape
    R, H = _rows_of(fc2_out, "fc2_out", _ACT)
    _dev(dy, "dy", _ACT, (T, H))
    _dev(unpermute, "unpermute", torch.int32, (T * k,))
    if R != T * k + n_shared * T:
        raise ValueError(f"fc2_out has {R} rows, expected {T * k + n_shared * T}")
    d = fc2_out.device
    d_fc2, d_scales = (None, None) if out is None else out
    d_fc2 = _out(d_fc2, "d_fc2", (R, H), fc2_out.dtype, d)
    d_scales = _out(d_scales, "d_scales", (T, k), torch.float32, d)
    _call("moe_finalize_backward", d, dy, _DT[dy.dtype], fc2_out, _DT[fc2_out.dtype], unpermute, scales,
          T, k, H, n_shared, d_fc2, d_scales)
    return d_fc2, d_scales


def route_backward(logits, ids, d_scales, method, scaling=1.0, renormalize=False, out=None):
    """moe_route_backward -> d_logits fp32 [T, E] from the gradient of route's scales."""
    T, E = _rows_of(logits, "logits", torch.float32)
    _dev(ids, "ids", torch.int32)
    k = ids.shape[1] if ids.dim() == 2 else 0
    _dev(ids, "ids", shape=(T, k))
    _dev(d_scales, "d_scales", torch.float32, (T, k))
    out = _out(out, "d_logits", (T, E), torch.float32, logits.device)
    _call("moe_route_backward", logits.device, logits, ids, d_scales, T, E, method, k, float(scaling),
          ROUTE_FLAG_RENORMALIZE if renormalize else 0, out)
    return out


def swiglu(gu, quantize=False, checkpoint=False, want_h=None, out=None):
    """moe_swiglu -> (h, hq, h_scale, guq, gu_scale) of FC1 rows gu [rows, 2I] (gate, then up):
    h in gu's dtype, with quantize its e4m3 codes and 1x128 scales instead (want_h=True: both),
    with checkpoint the codes and scales of gu for swiglu_backward; the others None.  `out` is the
    same tuple of buffers."""
    rows, I2 = _rows_of(gu, "gu", _ACT)
    if I2 % 2:
        raise ValueError(f"gu must be [rows, 2I] (got {tuple(gu.shape)})")
    I, dt, d = I2 // 2, gu.dtype, gu.device
    want_h = not quantize if want_h is None else want_h
    h, hq, hs, q, qs = (None,) * 5 if out is None else out
    if want_h:
        h = _out(h, "h", (rows, I), dt, d)
    else:
        _unused(("h",), (h,))
    if quantize:
        hq = _out(hq, "hq", (rows, I), torch.float8_e4m3fn, d)
        hs = _out(hs, "h_scale", (rows, I // 128), torch.float32, d)
    else:
        _unused(("hq", "h_scale"), (hq, hs))
    if checkpoint:
        q = _out(q, "guq", (rows, I2), torch.float8_e4m3fn, d)
        qs = _out(qs, "gu_scale", (rows, I2 // 128), torch.float32, d)
    else:
        _unused(("guq", "gu_scale"), (q, qs))
    _call("moe_swiglu", d, gu, _DT[dt], rows, I, h, hq, hs, q, qs)
    return h, hq, hs, q, qs


def swiglu_backward(dh, guq, gu_scale, want_h=False, out=None):
    """moe_swiglu_backward -> (d_gu [rows, 2I], h [rows, I] or None) from swiglu's checkpoint;
    with want_h the checkpoint's h again, for FC2's weight gradient (out's h may be dh)."""
    rows, I = _rows_of(dh, "dh", _ACT)
    dt, d = dh.dtype, dh.device
    _dev(guq, "guq", torch.float8_e4m3fn, (rows, 2 * I))
    _dev(gu_scale, "gu_scale", torch.float32, (rows, 2 * I // 128))
    d_gu, h = (None, None) if out is None else out
    d_gu = _out(d_gu, "d_gu", (rows, 2 * I), dt, d)
    if want_h:
        h = _out(h, "h", (rows, I), dt, d)
    else:
        _unused(("h",), (h,))
    _call("moe_swiglu_backward", d, dh, _DT[dt], guq, gu_scale, rows, I, d_gu, h)
    return d_gu, h


# ------------------------------------------------------------------- MXFP4
# Codes are torch.float4_e2m1fn_x2 [.., cols/2] (two a byte, the even column low) and scales
# torch.float8_e8m0fnu [.., cols/32]; bytes of a checkpoint become them by .view(dtype).
# These calls, and layer_few, have no gradient: they warn (UserWarning) of a tensor that requires grad
# while gradients are enabled.
def need_mxfp4_types():
    """Refuses where torch lacks the types of codes or scales."""
    if _CODES is None or _SCALES is None:
        raise NotImplementedError("MXFP4 needs a torch with float4_e2m1fn_x2 and float8_e8m0fnu")


def quantize_mxfp4(x, out=None):
    """moe_quantize_mxfp4 -> (codes float4_e2m1fn_x2 [rows, cols/2], scale float8_e8m0fnu
    [rows, cols/32]) of x [rows, cols]; weights [.., N, K] go as x.view(-1, K)."""
    need_mxfp4_types()
    rows, cols = _rows_of(x, "x", _ACT)
    q, scale = (None, None) if out is None else out
    q = _out(q, "codes", (rows, cols // 2), _CODES, x.device)
    scale = _out(scale, "scale", (rows, cols // 32), _SCALES, x.device)
    _call("moe_quantize_mxfp4", x.device, x, _DT[x.dtype], rows, cols, q, scale)
    return q, scale


def dequantize_mxfp4(codes, scale, dtype=torch.bfloat16, out=None):
    """moe_dequantize_mxfp4 -> the values [rows, cols] of quantize_mxfp4's codes and scales."""
    need_mxfp4_types()
    rows, half = _rows_of(codes, "codes", _CODES)
    if half % 16:
        raise ValueError(f"codes must be [rows, cols/2] with cols a multiple of 32 (got {tuple(codes.shape)})")
    _dev(scale, "scale", _SCALES, (rows, half // 16))
    if dtype not in _ACT:
        raise ValueError(f"dtype must be one of {_ACT} (got {dtype})")
    out = _out(out, "x", (rows, 2 * half), dtype, codes.device)
    _call("moe_dequantize_mxfp4", codes.device, codes, scale, rows, 2 * half, _DT[dtype], out)
    return out


def expert_ffn_mxfp4(xq, x_scale, expert_offsets, permuted_pair, w13, w2, w13_scale, w2_scale, k, E,
                     n_shared=0, ws=None, out=None):
    """moe_expert_ffn_mxfp4 -> fc2_out bf16 [T*k + n_shared*T, H]; w13 [G, 2I, H/2] and w2 [G, H, I/2]
    codes with scales [G, 2I, H/32] and [G, H, I/32]."""
    need_mxfp4_types()
    T, half = _rows_of(xq, "xq", _CODES)
    H, G, d = 2 * half, E + n_shared, xq.device
    _dev(x_scale, "x_scale", _SCALES, (T, H // 32))
    _dev(w13, "w13", _CODES)
    if w13.dim() != 3:
        raise ValueError(f"w13 must be [G, 2I, H/2] (got {tuple(w13.shape)})")
    I = w13.shape[1] // 2
    _dev(w13, "w13", shape=(G, 2 * I, half))
    _dev(w2, "w2", _CODES, (G, H, I // 2))
    _dev(w13_scale, "w13_scale", _SCALES, (G, 2 * I, H // 32))
    _dev(w2_scale, "w2_scale", _SCALES, (G, H, I // 32))
    _dev(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    _dev(permuted_pair, "permuted_pair", torch.int32, (T * k,))
    R = T * k + n_shared * T
    out = _out(out, "fc2_out", (R, H), torch.bfloat16, d)
    if ws is None:
        ws = alloc_workspace(T, k, E, n_shared, H, I, _CODES, d)
    _dev(ws, "ws", torch.uint8)
    _call("moe_expert_ffn_mxfp4", d, xq, x_scale, T, H, I, k, E, n_shared, expert_offsets, permuted_pair,
          w13, w2, w13_scale, w2_scale, out, ws, ws.numel())
    return out


# ------------------------------------------------------------ a few tokens
def layer_few_workspace(T, H, I, E, k, n_shared=0, act_dtype=torch.bfloat16, device="cuda") -> torch.Tensor:
    n = int(lib().moe_layer_few_workspace_size(T, H, I, E, k, n_shared, _DT[act_dtype]))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def layer_few(x, logits, w13, w2, k, method, w13_scale=None, w2_scale=None, n_group=1, topk_group=1, bias=None,
              scaling=1.0, renormalize=False, n_shared=0, ws=None, out=None):
    """moe_layer_few, the whole layer for at most FEW_MAX_T tokens -> (y [T, H] in x's dtype, ids int32
    [T, k], scales fp32 [T, k]).  Weights as expert_ffn takes them, or as expert_ffn_mxfp4 does (by
    w13's dtype); `out` is the same tuple of buffers."""
    T, H = _rows_of(x, "x", _ACT)
    d = x.device
    if _rows_of(logits, "logits", torch.float32)[0] != T:
        raise ValueError(f"logits has {logits.shape[0]} rows, expected {T}")
    E = logits.shape[1]
    G = E + n_shared
    if bias is not None:
        _dev(bias, "bias", torch.float32, (E,))
    _dev(w13, "w13", (torch.float32, torch.bfloat16, torch.float8_e4m3fn, _CODES))
    if w13.dim() != 3:
        raise ValueError(f"w13 must be [G, 2I, H] (got {tuple(w13.shape)})")
    I, mx = w13.shape[1] // 2, w13.dtype == _CODES
    _dev(w13, "w13", shape=(G, 2 * I, H // 2 if mx else H))
    _dev(w2, "w2", w13.dtype, (G, H, I // 2 if mx else I))
    if mx:
        need_mxfp4_types()
        _dev(w13_scale, "w13_scale", _SCALES, (G, 2 * I, H // 32))
        _dev(w2_scale, "w2_scale", _SCALES, (G, H, I // 32))
    elif w13.dtype == torch.float8_e4m3fn:
        _dev(w13_scale, "w13_scale", torch.float32, (G, 2 * I // 128, H // 128))
        _dev(w2_scale, "w2_scale", torch.float32, (G, H // 128, I // 128))
    y, ids, scales = (None,) * 3 if out is None else out
    y = _out(y, "y", (T, H), x.dtype, d)
    ids = _out(ids, "ids", (T, k), torch.int32, d)
    scales = _out(scales, "scales", (T, k), torch.float32, d)
    if ws is None:
        ws = layer_few_workspace(T, H, I, E, k, n_shared, x.dtype, d)
    _dev(ws, "ws", torch.uint8)
    _call("moe_layer_few", d, x, _DT[x.dtype], logits, T, H, I, E, method, k, n_group, topk_group, bias,
          float(scaling), ROUTE_FLAG_RENORMALIZE if renormalize else 0, n_shared, w13, w2, _DT[w13.dtype],
          w13_scale, w2_scale, ids, scales, y, ws, ws.numel())
    return y, ids, scales


def timing_enable(on: bool = True):
    _check("moe_timing_enable", lib().moe_timing_enable(1 if on else 0))


def kernel_times(reset: bool = True):
    """{kernel: (total_ms, launches)} since the last reset (waits for the events)."""
    ms = (C.c_double * len(KERNEL_IDS))()
    n = (C.c_int64 * len(KERNEL_IDS))()
    _check("moe_kernel_times", lib().moe_kernel_times(C.cast(ms, C.c_void_p),
                                                      C.cast(n, C.c_void_p), int(reset)))
    return {name: (ms[i], n[i]) for i, name in enumerate(KERNEL_IDS)}
