"""Python binding of the gfx950 GPTQ layer-quantization library.

Thin ctypes layer over include/gptq.h: it checks tensor placement and dtypes,
allocates the outputs and the workspace with torch on the tensors' device,
passes raw device pointers and the current HIP stream, and raises on any
non-OK status.  Every step of the computation runs in the HIP library; there
is no host fallback.  The names match the C entry points.
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "GPTQError", "lib_path", "load_library", "gptq_hessian_accumulate",
    "gptq_cholesky_inverse", "gptq_quantize_layer", "gptq_workspace_bytes",
    "gptq_hessian_workspace_bytes", "gptq_factor_workspace_bytes",
    "gptq_hessian_accumulate_noalloc", "gptq_dequant_matmul", "gptq_dequant_matmul_t",
    "gptq_lora_matmul", "gptq_lora_backward", "gptq_lora_workspace_bytes",
    "gptq_lora_backward_workspace_bytes", "gptq_dequant_matmul_t_workspace_bytes",
    "gptq_distill_loss", "gptq_distill_backward", "gptq_quantize_stack",
    "gptq_mx_quantize", "gptq_mx_matmul", "gptq_mx_matmul_t", "gptq_mx_gated",
    "gptq_mx_gated_backward", "gptq_mx_matmul_workspace_bytes",
    "gptq_mx_matmul_t_workspace_bytes", "gptq_mx_gated_workspace_bytes",
    "gptq_mx_gated_backward_workspace_bytes", "gptq_token_logprobs",
    "gptq_token_logprobs_backward", "gptq_token_logprobs_workspace_bytes",
    "gptq_trace_enable", "gptq_trace_read", "TRACE_PHASES",
    "EXPORTED_SYMBOLS", "GRIDS", "ACTIVATIONS", "GPTQ_OK", "GPTQ_ERR_INVALID_ARG", "GPTQ_ERR_NOT_SPD",
    "GPTQ_ERR_WORKSPACE", "GPTQ_ERR_HIP",
]

GPTQ_OK, GPTQ_ERR_INVALID_ARG, GPTQ_ERR_NOT_SPD, GPTQ_ERR_WORKSPACE, GPTQ_ERR_HIP = range(5)
GPTQ_BF16, GPTQ_F32, GPTQ_F16 = 0, 1, 2
GPTQ_NOALLOC_SCRATCH_BYTES = 256 << 20      # include/gptq.h

EXPORTED_SYMBOLS = (
    "gptq_status_string", "gptq_hessian_workspace_bytes",
    "gptq_hessian_accumulate", "gptq_factor_workspace_bytes",
    "gptq_cholesky_inverse", "gptq_workspace_bytes", "gptq_quantize_layer",
    "gptq_hessian_accumulate_noalloc", "gptq_dequant_matmul",
    "gptq_stack_workspace_bytes", "gptq_quantize_stack", "gptq_trace_enable",
    "gptq_trace_read", "gptq_dequant_matmul_t_workspace_bytes", "gptq_dequant_matmul_t",
    "gptq_lora_workspace_bytes", "gptq_lora_matmul", "gptq_lora_backward_workspace_bytes",
    "gptq_lora_backward", "gptq_distill_loss", "gptq_distill_backward",
    "gptq_mx_quantize", "gptq_mx_matmul_workspace_bytes", "gptq_mx_matmul",
    "gptq_mx_matmul_t_workspace_bytes", "gptq_mx_matmul_t",
    "gptq_mx_gated_workspace_bytes", "gptq_mx_gated",
    "gptq_mx_gated_backward_workspace_bytes", "gptq_mx_gated_backward",
    "gptq_token_logprobs_workspace_bytes", "gptq_token_logprobs", "gptq_token_logprobs_backward",
)
TRACE_PHASES = ("stats", "factor", "chain", "lazy", "other")
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().gptq_status_string(status).decode() if _LIB else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


GRIDS = {"minmax": 0, "symmetric": 1, "fixed": 2}


class _Params(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("blocksize", ctypes.c_int32), ("percdamp", ctypes.c_float),
                ("act_order", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("static_groups", ctypes.c_int32), ("fixed_scales", ctypes.c_void_p),
                ("fixed_zeros", ctypes.c_void_p)]


class _StackLayer(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("w_dtype", ctypes.c_int), ("m", ctypes.c_int64),
                ("d", ctypes.c_int64), ("ldw", ctypes.c_int64), ("params", _Params),
                ("qweight", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("g_idx", ctypes.c_void_p)]


class _Adapters(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("row", ctypes.c_void_p), ("n_adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32)]


def lib_path() -> str:
    return os.path.join(_HERE, "libgptq_hip.so")


def load_library():
    """Load libgptq_hip.so (built in-tree by build.py).  Raises if absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: the HIP library has not been built "
                          "(run post_weight_quantization_15_amd.build.build())")
    lib = ctypes.CDLL(path)
    vp, i64, sz, f32, i32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float, ctypes.c_int32)
    pp = ctypes.POINTER(_Params)
    lib.gptq_status_string.restype = ctypes.c_char_p
    lib.gptq_status_string.argtypes = [ctypes.c_int]
    lib.gptq_hessian_workspace_bytes.restype = sz
    lib.gptq_hessian_workspace_bytes.argtypes = [i64, i64]
    lib.gptq_hessian_accumulate.restype = ctypes.c_int
    lib.gptq_hessian_accumulate.argtypes = [vp, i64, vp, ctypes.c_int, i64, i64, vp, sz, vp]
    lib.gptq_hessian_accumulate_noalloc.restype = ctypes.c_int
    lib.gptq_hessian_accumulate_noalloc.argtypes = [vp, i64, vp, ctypes.c_int, i64, i64, vp]
    lib.gptq_dequant_matmul.restype = ctypes.c_int
    lib.gptq_dequant_matmul.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, vp, ctypes.c_int,
                                        vp, vp, i64, i32, i32, i32, vp, i64, vp]
    ap = ctypes.POINTER(_Adapters)
    dt = ctypes.c_int
    lib.gptq_dequant_matmul_t_workspace_bytes.restype = sz
    lib.gptq_dequant_matmul_t_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gptq_dequant_matmul_t.restype = ctypes.c_int
    lib.gptq_dequant_matmul_t.argtypes = [vp, dt, i64, i64, i64, vp, vp, dt, vp, vp, i64, i32, i32,
                                          i32, vp, i64, vp, sz, vp]
    lib.gptq_lora_workspace_bytes.restype = sz
    lib.gptq_lora_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.gptq_lora_matmul.restype = ctypes.c_int
    lib.gptq_lora_matmul.argtypes = [vp, dt, i64, i64, i64, vp, vp, dt, vp, vp, i64, i32, i32, i32,
                                     ap, vp, vp, dt, i64, vp, sz, vp]
    lib.gptq_lora_backward_workspace_bytes.restype = sz
    lib.gptq_lora_backward_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.gptq_lora_backward.restype = ctypes.c_int
    lib.gptq_lora_backward.argtypes = [vp, dt, i64, i64, i64, vp, i64, vp, vp, vp, dt, vp, vp, i64,
                                       i32, i32, i32, ap, vp, i64, vp, vp, i32, vp, sz, vp]
    lib.gptq_distill_loss.restype = ctypes.c_int
    lib.gptq_distill_loss.argtypes = [vp, dt, i64, i64, i64, vp, vp, i64, f32, vp, vp, vp, vp, vp,
                                      i64, vp]
    lib.gptq_distill_backward.restype = ctypes.c_int
    lib.gptq_distill_backward.argtypes = [vp, dt, i64, i64, i64, vp, vp, vp, i64, f32, vp, vp, vp,
                                          vp, i64, vp]
    lib.gptq_mx_quantize.restype = ctypes.c_int
    lib.gptq_mx_quantize.argtypes = [vp, dt, i64, i64, i64, vp, vp, vp, i64, vp]
    lib.gptq_mx_matmul_workspace_bytes.restype = sz
    lib.gptq_mx_matmul_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.gptq_mx_matmul.restype = ctypes.c_int
    lib.gptq_mx_matmul.argtypes = [vp, i32, vp, i64, i64, i64, vp, vp, i64, vp, dt, i64, vp, sz,
                                      vp]
    lib.gptq_mx_matmul_t_workspace_bytes.restype = sz
    lib.gptq_mx_matmul_t_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gptq_mx_matmul_t.restype = ctypes.c_int
    lib.gptq_mx_matmul_t.argtypes = [vp, dt, i64, i64, i64, vp, vp, i64, vp, i64, vp, sz, vp]
    lib.gptq_mx_gated_workspace_bytes.restype = sz
    lib.gptq_mx_gated_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.gptq_mx_gated.restype = ctypes.c_int
    lib.gptq_mx_gated.argtypes = [vp, i32, vp, i64, i64, i64, vp, vp, vp, vp, i64, i32, vp, i64,
                                     vp, vp, i64, vp, sz, vp]
    lib.gptq_mx_gated_backward_workspace_bytes.restype = sz
    lib.gptq_mx_gated_backward_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gptq_mx_gated_backward.restype = ctypes.c_int
    lib.gptq_mx_gated_backward.argtypes = [vp, dt, i64, i64, i64, vp, vp, i64, vp, vp, vp, vp, i64,
                                              i32, vp, i64, vp, vp, sz, vp]
    lib.gptq_token_logprobs_workspace_bytes.restype = sz
    lib.gptq_token_logprobs_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gptq_token_logprobs.restype = ctypes.c_int
    lib.gptq_token_logprobs.argtypes = [vp, dt, i64, i64, i64, vp, f32, i64, vp, vp, vp, vp, vp, vp,
                                        vp, sz, vp]
    lib.gptq_token_logprobs_backward.restype = ctypes.c_int
    lib.gptq_token_logprobs_backward.argtypes = [vp, dt, i64, i64, i64, vp, vp, f32, vp, vp, vp, i64,
                                                 vp]
    sp = ctypes.POINTER(_StackLayer)
    lib.gptq_stack_workspace_bytes.restype = sz
    lib.gptq_stack_workspace_bytes.argtypes = [sp, i32, i64]
    lib.gptq_quantize_stack.restype = ctypes.c_int
    lib.gptq_quantize_stack.argtypes = [sp, i32, vp, i64, i32, vp,
                                        ctypes.POINTER(ctypes.c_double), vp, sz, vp]
    lib.gptq_trace_enable.restype = ctypes.c_int
    lib.gptq_trace_enable.argtypes = [i32]
    lib.gptq_trace_read.restype = ctypes.c_int
    lib.gptq_trace_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_int64), i32]
    lib.gptq_factor_workspace_bytes.restype = sz
    lib.gptq_factor_workspace_bytes.argtypes = [i64]
    lib.gptq_cholesky_inverse.restype = ctypes.c_int
    lib.gptq_cholesky_inverse.argtypes = [vp, i64, i64, f32, i32, vp, vp, vp,
                                          ctypes.POINTER(f32), vp, sz, vp]
    lib.gptq_workspace_bytes.restype = sz
    lib.gptq_workspace_bytes.argtypes = [i64, i64, pp, i32]
    lib.gptq_quantize_layer.restype = ctypes.c_int
    lib.gptq_quantize_layer.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64,
                                        pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    _LIB = lib
    return lib


def _lib():
    return load_library()


def _dev_ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU (no host path exists)")
    return ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return GPTQ_BF16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _params(bits, group_size, blocksize, percdamp, act_order, grid="minmax",
            static_groups=False, fixed_scales=None, fixed_zeros=None):
    if grid not in GRIDS:
        raise ValueError(f"grid must be one of {sorted(GRIDS)}")
    return _Params(int(bits), int(group_size), int(blocksize), float(percdamp),
                   int(bool(act_order)), GRIDS[grid], int(bool(static_groups)),
                   fixed_scales.data_ptr() if fixed_scales is not None else None,
                   fixed_zeros.data_ptr() if fixed_zeros is not None else None)


def _check(status, where):
    if status != GPTQ_OK:
        raise GPTQError(status, where)


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _row_stride(t, name):
    """Leading dimension of a row-major [rows, cols] tensor with unit column
    stride.  Rows that overlap (stride(0) < cols, e.g. an expanded view)
    cannot be described by one leading dimension and are rejected."""
    rows, cols = t.shape
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name} rows overlap (stride(0) = {t.stride(0)} < {cols})")
    return t.stride(0) if rows > 1 else cols


def _expect(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def gptq_hessian_workspace_bytes(d: int, n_tok: int) -> int:
    return int(_lib().gptq_hessian_workspace_bytes(d, n_tok))


def gptq_factor_workspace_bytes(d: int) -> int:
    return int(_lib().gptq_factor_workspace_bytes(d))


def gptq_workspace_bytes(m, d, bits=4, group_size=-1, blocksize=128,
                         percdamp=0.01, act_order=False, factor_inside=True,
                         grid="minmax", static_groups=False, fixed_scales=None,
                         fixed_zeros=None) -> int:
    p = _params(bits, group_size, blocksize, percdamp, act_order, grid,
                static_groups, fixed_scales, fixed_zeros)
    return int(_lib().gptq_workspace_bytes(m, d, ctypes.byref(p), int(factor_inside)))


def gptq_hessian_accumulate(S: torch.Tensor, X: torch.Tensor, ws=None) -> torch.Tensor:
    """S [d, d] fp32 += X^T X for token-major X [n_tok, d] (bf16 or fp32)."""
    if S.dim() != 2 or S.shape[0] != S.shape[1]:
        raise ValueError("S must be a [d, d] tensor")
    d = S.shape[0]
    _expect(S, "S", torch.float32, (d, d), S.device)
    if X.dim() != 2 or X.shape[1] != d:
        raise ValueError("X must be [n_tok, d]")
    if X.device != S.device:
        raise ValueError("X and S must be on the same device")
    ldx = _row_stride(X, "X")
    dtc = _dtype_code(X)
    lib = _lib()
    n_tok = X.shape[0]
    need = lib.gptq_hessian_workspace_bytes(d, n_tok)
    if ws is None or ws.numel() < need:
        ws = _workspace(need, S.device)
    st = lib.gptq_hessian_accumulate(_dev_ptr(S), d, _dev_ptr(X), dtc,
                                     n_tok, ldx, _dev_ptr(ws),
                                     ws.numel(), _stream(S.device))
    _check(st, "gptq_hessian_accumulate")
    return S


def gptq_hessian_accumulate_noalloc(S: torch.Tensor, X: torch.Tensor) -> torch.Tensor:
    """As gptq_hessian_accumulate, with the library's static scratch instead
    of a workspace (no device allocation anywhere in the call)."""
    if S.dim() != 2 or S.shape[0] != S.shape[1]:
        raise ValueError("S must be a [d, d] tensor")
    d = S.shape[0]
    _expect(S, "S", torch.float32, (d, d), S.device)
    if X.dim() != 2 or X.shape[1] != d:
        raise ValueError("X must be [n_tok, d]")
    if X.device != S.device:
        raise ValueError("X and S must be on the same device")
    ldx = _row_stride(X, "X")
    dtc = _dtype_code(X)
    st = _lib().gptq_hessian_accumulate_noalloc(_dev_ptr(S), d, _dev_ptr(X), dtc,
                                                X.shape[0], ldx, _stream(S.device))
    _check(st, "gptq_hessian_accumulate_noalloc")
    return S


def gptq_cholesky_inverse(S: torch.Tensor, n: int, percdamp: float = 0.01,
                          act_order: bool = False, ws=None):
    """Returns (R [d, d] fp32 upper, perm [d] int32, dead [d] uint8, damp)."""
    if S.dim() != 2 or S.shape[0] != S.shape[1]:
        raise ValueError("S must be a [d, d] tensor")
    d = S.shape[0]
    dev = S.device
    _expect(S, "S", torch.float32, (d, d), dev)
    lib = _lib()
    R = torch.empty(d, d, dtype=torch.float32, device=dev)
    perm = torch.empty(d, dtype=torch.int32, device=dev)
    dead = torch.empty(d, dtype=torch.uint8, device=dev)
    need = lib.gptq_factor_workspace_bytes(d)
    if ws is None or ws.numel() < need:
        ws = _workspace(need, dev)
    damp = ctypes.c_float(0.0)
    st = lib.gptq_cholesky_inverse(_dev_ptr(S), int(n), d, float(percdamp),
                                   int(bool(act_order)), _dev_ptr(R), _dev_ptr(perm),
                                   _dev_ptr(dead), ctypes.byref(damp), _dev_ptr(ws),
                                   ws.numel(), _stream(dev))
    _check(st, "gptq_cholesky_inverse")
    return R, perm, dead, float(damp.value)


def gptq_quantize_layer(W: torch.Tensor, S: torch.Tensor = None, n: int = 0,
                        bits: int = 4, group_size: int = -1, blocksize: int = 128,
                        percdamp: float = 0.01, act_order: bool = False,
                        R=None, perm=None, dead=None, want_w_hat: bool = False,
                        ws=None, grid: str = "minmax", static_groups: bool = False,
                        fixed_scales=None, fixed_zeros=None) -> dict:
    """Quantize W [m, d]; returns qweight, scales, zeros, g_idx (and w_hat).

    grid: "minmax", "symmetric" (signed codes; ternary at bits=2) or
    "fixed" (fixed_scales fp32 / fixed_zeros uint8, [m, n_g] on W's device).
    static_groups: fit the groups on the original contiguous columns."""
    if W.dim() != 2:
        raise ValueError("W must be [m, d]")
    m, d = W.shape
    dev = W.device
    ldw = _row_stride(W, "W")
    dtc = _dtype_code(W)
    given = [t is not None for t in (R, perm, dead)]
    if any(given) and not all(given):
        raise ValueError("pass R, perm and dead together (or none of them)")
    if all(given):
        _expect(R, "R", torch.float32, (d, d), dev)
        _expect(perm, "perm", torch.int32, (d,), dev)
        _expect(dead, "dead", torch.uint8, (d,), dev)
    else:
        if S is None:
            raise ValueError("S is required when no factor is given")
        _expect(S, "S", torch.float32, (d, d), dev)
    ng = 1 if group_size == -1 else -(-d // group_size)
    if grid == "fixed":
        _expect(fixed_scales, "fixed_scales", torch.float32, (m, ng), dev)
        _expect(fixed_zeros, "fixed_zeros", torch.uint8, (m, ng), dev)
    elif fixed_scales is not None or fixed_zeros is not None:
        raise ValueError("fixed_scales / fixed_zeros need grid='fixed'")
    lib = _lib()
    p = _params(bits, group_size, blocksize, percdamp, act_order, grid,
                static_groups, fixed_scales, fixed_zeros)
    factor_inside = R is None
    need = lib.gptq_workspace_bytes(m, d, ctypes.byref(p), int(factor_inside))
    if need == 0:
        raise GPTQError(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes")
    if ws is None or ws.numel() < need:
        ws = _workspace(need, dev)
    words = -(-d * bits // 32)
    out = dict(
        qweight=torch.empty(m, words, dtype=torch.int32, device=dev),
        scales=torch.empty(m, ng, dtype=torch.float32, device=dev),
        zeros=torch.empty(m, ng, dtype=torch.uint8, device=dev),
        g_idx=torch.empty(d, dtype=torch.int32, device=dev),
    )
    w_hat = torch.empty(m, d, dtype=torch.float32, device=dev) if want_w_hat else None
    st = lib.gptq_quantize_layer(
        _dev_ptr(W), dtc, m, d, ldw,
        _dev_ptr(S) if S is not None and not all(given) else None, int(n), ctypes.byref(p),
        _dev_ptr(R), _dev_ptr(perm), _dev_ptr(dead),
        _dev_ptr(out["qweight"]), _dev_ptr(out["scales"]), _dev_ptr(out["zeros"]),
        _dev_ptr(out["g_idx"]), _dev_ptr(w_hat), _dev_ptr(ws), ws.numel(), _stream(dev))
    _check(st, "gptq_quantize_layer")
    if want_w_hat:
        out["w_hat"] = w_hat
    return out


def gptq_dequant_matmul(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                        zeros: torch.Tensor, g_idx: torch.Tensor, bits: int,
                        group_size: int, signed: bool = False, Y=None) -> torch.Tensor:
    """Y [n, m] fp32 = X W_hat^T for bf16 activations X [n, d] and the stored
    format of gptq_quantize_layer (qweight, scales, zeros, g_idx); scales
    may be float32 or the compact float16 storage."""
    if X.dim() != 2:
        raise ValueError("X must be [n, d]")
    n, d = X.shape
    m = qweight.shape[0]
    dev = X.device
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    ldx = _row_stride(X, "X")
    words = -(-d * bits // 32)
    ng = 1 if group_size == -1 else -(-d // group_size)
    if qweight.dtype not in (torch.int32, torch.uint32):
        raise TypeError("qweight must be int32/uint32")
    if tuple(qweight.shape) != (m, words) or not qweight.is_contiguous():
        raise ValueError(f"qweight must be contiguous [{m}, {words}]")
    if scales.dtype not in (torch.float32, torch.float16):
        raise TypeError("scales must be float32 or float16")
    _expect(scales, "scales", scales.dtype, (m, ng), dev)
    _expect(zeros, "zeros", torch.uint8, (m, ng), dev)
    _expect(g_idx, "g_idx", torch.int32, (d,), dev)
    if qweight.device != dev:
        raise ValueError("qweight must be on X's device")
    if Y is None:
        Y = torch.empty(n, m, dtype=torch.float32, device=dev)
    else:
        _expect(Y, "Y", torch.float32, (n, m), dev)
    sdt = GPTQ_F16 if scales.dtype == torch.float16 else GPTQ_F32
    st = _lib().gptq_dequant_matmul(_dev_ptr(X), GPTQ_BF16, n, d, ldx, _dev_ptr(qweight),
                                    _dev_ptr(scales), sdt, _dev_ptr(zeros), _dev_ptr(g_idx),
                                    m, int(bits), int(group_size), int(bool(signed)),
                                    _dev_ptr(Y), m, _stream(dev))
    _check(st, "gptq_dequant_matmul")
    return Y


# ---------------------------------------------------------------------------
# Adapters beside the packed weights, and the loss that trains them
# ---------------------------------------------------------------------------

_F32, _BF16 = torch.float32, torch.bfloat16

# The current device and its stream as an integer.  A call for one token is as
# long on the host as on the GPU; these are torch's own accessors without the
# objects around them (0.2 us instead of 5).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _like(t, name, dtype, shape, dev):
    """_expect, with the usual answer first."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev:
            return
    except AttributeError:
        pass
    _expect(t, name, dtype, shape, dev)


def _gpu_rows(t, name, cols=None, dtypes=(_BF16,)):
    """Checks a [rows, cols] tensor on the GPU; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [rows, {'cols' if cols is None else cols}], "
                         f"got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.shape[1]
    return _row_stride(t, name) if t.shape[0] else t.shape[1]


def _gpu_device(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU (no host path exists)")
    return t.device


def _check_packed(qweight, scales, zeros, g_idx, bits, group_size, m, d, dev):
    """Checks the stored format of an [m, d] layer; returns the scales' type code."""
    if bits not in (2, 3, 4, 8) or not (group_size == -1 or group_size > 0):
        raise GPTQError(GPTQ_ERR_INVALID_ARG, "bits / group_size")
    ng = 1 if group_size == -1 else -(-d // group_size)
    if qweight.dtype not in (torch.int32, torch.uint32):
        raise TypeError("qweight must be int32/uint32")
    _like(qweight, "qweight", qweight.dtype, (m, -(-d * bits // 32)), dev)
    if scales.dtype not in (_F32, torch.float16):
        raise TypeError("scales must be float32 or float16")
    _like(scales, "scales", scales.dtype, (m, ng), dev)
    _like(zeros, "zeros", torch.uint8, (m, ng), dev)
    _like(g_idx, "g_idx", torch.int32, (d,), dev)
    return GPTQ_F16 if scales.dtype == torch.float16 else GPTQ_F32


def _check_adapters(A, B, adapter, alpha, n, m, d, dev):
    """Checks a set of adapters; returns its descriptor."""
    if A.dim() != 3 or A.shape[2] != d:
        raise ValueError(f"A must be [n_adapters, rank, {d}], got {tuple(A.shape)}")
    count, rank = A.shape[0], A.shape[1]
    _like(A, "A", _BF16, (count, rank, d), dev)
    _like(B, "B", _BF16, (count, m, rank), dev)
    _like(adapter, "adapter", torch.int32, (n,), dev)
    _like(alpha, "alpha", _F32, (count,), dev)
    return _Adapters(A.data_ptr(), B.data_ptr(), alpha.data_ptr(), adapter.data_ptr(), count, rank)


def _out(t, name, dtype, shape, dev):
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _like(t, name, dtype, shape, dev)
    return t


def _enough(ws, need, dev):
    if ws is None:
        return torch.empty(need or 1, dtype=torch.uint8, device=dev)
    if ws.numel() * ws.element_size() < need:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if ws.device != dev or not ws.is_contiguous() or ws.data_ptr() % 16:
        raise ValueError(f"ws must be contiguous, 16-byte aligned, on {dev}")
    return ws


def _scratch(ws, need, dev):
    """A workspace (none where none is needed), its address and its size."""
    if ws is None and not need:
        return None, None, 0
    ws = _enough(ws, need, dev)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _launch(dev, where, fn, *args):
    """Calls a library function with the stream of `dev` last, `dev` being the
    current device for the launch."""
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev.index))
    else:
        st = fn(*args, _raw_stream(dev.index))
    if st != GPTQ_OK:
        raise GPTQError(st, where)


def gptq_lora_workspace_bytes(n: int, m: int, d: int, group_size: int, rank: int) -> int:
    return int(_lib().gptq_lora_workspace_bytes(n, m, d, group_size, rank))


def gptq_lora_backward_workspace_bytes(n: int, m: int, d: int, rank: int, n_adapters: int) -> int:
    return int(_lib().gptq_lora_backward_workspace_bytes(n, m, d, rank, n_adapters))


def gptq_dequant_matmul_t_workspace_bytes(n: int, m: int, d: int) -> int:
    return int(_lib().gptq_dequant_matmul_t_workspace_bytes(n, m, d))


def gptq_lora_matmul(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                     zeros: torch.Tensor, g_idx: torch.Tensor, bits: int, group_size: int,
                     A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor,
                     alpha: torch.Tensor, signed: bool = False, Y=None, H=None,
                     want_h: bool = False, out_dtype=torch.float32, ws=None):
    """Y [n, m] = X W_hat^T + alpha_a (X A_a^T) B_a^T, a = adapter[row].

    X bf16 [n, d] and the stored format as in gptq_dequant_matmul; A bf16
    [n_adapters, rank, d], B bf16 [n_adapters, m, rank], alpha fp32
    [n_adapters], adapter int32 [n] (an id outside [0, n_adapters), e.g. -1:
    the shared product alone).  Y is float32 or bfloat16 (out_dtype, or the
    given Y's).  Returns Y, or (Y, H) with H = X A_a^T fp32 [n, rank] when
    want_h is set or H is given (gptq_lora_backward needs it)."""
    ldx = _gpu_rows(X, "X")
    dev = _gpu_device(X)
    n, d = X.shape
    m = qweight.shape[0]
    sdt = _check_packed(qweight, scales, zeros, g_idx, bits, group_size, m, d, dev)
    ad = _check_adapters(A, B, adapter, alpha, n, m, d, dev)
    if Y is not None:
        out_dtype = Y.dtype
    if out_dtype is not _F32 and out_dtype is not _BF16:
        raise TypeError(f"Y must be float32 or bfloat16, got {out_dtype}")
    lib = _lib()
    need = lib.gptq_lora_workspace_bytes(n, m, d, group_size, ad.rank)
    ws = _enough(ws, need, dev)
    Y = _out(Y, "Y", out_dtype, (n, m), dev)
    if want_h or H is not None:
        H = _out(H, "H", _F32, (n, ad.rank), dev)
    _launch(dev, "gptq_lora_matmul", lib.gptq_lora_matmul, X.data_ptr(), GPTQ_BF16, n, d, ldx,
            qweight.data_ptr(), scales.data_ptr(), sdt, zeros.data_ptr(), g_idx.data_ptr(), m, bits,
            group_size, 1 if signed else 0, ctypes.byref(ad), None if H is None else H.data_ptr(),
            Y.data_ptr(), GPTQ_F32 if out_dtype is _F32 else GPTQ_BF16, m, ws.data_ptr(),
            ws.numel() * ws.element_size())
    return Y if H is None else (Y, H)


def gptq_lora_backward(dY: torch.Tensor, X: torch.Tensor, H, qweight: torch.Tensor,
                       scales: torch.Tensor, zeros: torch.Tensor, g_idx: torch.Tensor, bits: int,
                       group_size: int, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor,
                       alpha: torch.Tensor, signed: bool = False, need_dx: bool = True,
                       need_dab: bool = True, dX=None, dA=None, dB=None, accumulate: bool = False,
                       ws=None):
    """Gradients of gptq_lora_matmul from dY bf16 [n, m]: (dX bf16 [n, d], dA
    fp32 like A, dB fp32 like B), None for those not needed.  H as the
    forward call returned it (only read for dB).  accumulate adds to the given
    dA and dB instead of overwriting them."""
    ldy = _gpu_rows(dY, "dY")
    dev = _gpu_device(dY)
    n, m = dY.shape
    d = A.shape[-1]
    sdt = _check_packed(qweight, scales, zeros, g_idx, bits, group_size, m, d, dev)
    ad = _check_adapters(A, B, adapter, alpha, n, m, d, dev)
    ldx = d
    if need_dab:
        ldx = _gpu_rows(X, "X", d)
        if X.shape[0] != n or X.device != dev:
            raise ValueError(f"X must be [{n}, {d}] on {dev}")
        _like(H, "H", _F32, (n, ad.rank), dev)
        if accumulate and (dA is None or dB is None):
            raise ValueError("accumulate needs dA and dB")
        dA = _out(dA, "dA", _F32, tuple(A.shape), dev)
        dB = _out(dB, "dB", _F32, tuple(B.shape), dev)
    else:
        dA = dB = None
    dX = _out(dX, "dX", _BF16, (n, d), dev) if need_dx else None
    lib = _lib()
    need = lib.gptq_lora_backward_workspace_bytes(n, m, d, ad.rank, ad.n_adapters)
    ws = _enough(ws, need, dev)
    _launch(dev, "gptq_lora_backward", lib.gptq_lora_backward, dY.data_ptr(), GPTQ_BF16, n, m, ldy,
            X.data_ptr() if need_dab else None, ldx, H.data_ptr() if need_dab else None,
            qweight.data_ptr(), scales.data_ptr(), sdt, zeros.data_ptr(), g_idx.data_ptr(), d, bits,
            group_size, 1 if signed else 0, ctypes.byref(ad),
            dX.data_ptr() if need_dx else None, d, dA.data_ptr() if need_dab else None,
            dB.data_ptr() if need_dab else None, 1 if accumulate else 0, ws.data_ptr(),
            ws.numel() * ws.element_size())
    return dX, dA, dB


def gptq_dequant_matmul_t(dY: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                          zeros: torch.Tensor, g_idx: torch.Tensor, bits: int, group_size: int,
                          signed: bool = False, dX=None, ws=None) -> torch.Tensor:
    """dX bf16 [n, d] = dY W_hat for dY bf16 [n, m]: the gradient of
    gptq_dequant_matmul with respect to its activations."""
    ldy = _gpu_rows(dY, "dY")
    dev = _gpu_device(dY)
    n, m = dY.shape
    d = g_idx.shape[0]
    sdt = _check_packed(qweight, scales, zeros, g_idx, bits, group_size, m, d, dev)
    lib = _lib()
    ws = _enough(ws, lib.gptq_dequant_matmul_t_workspace_bytes(n, m, d), dev)
    dX = _out(dX, "dX", _BF16, (n, d), dev)
    _launch(dev, "gptq_dequant_matmul_t", lib.gptq_dequant_matmul_t, dY.data_ptr(), GPTQ_BF16, n, m,
            ldy, qweight.data_ptr(), scales.data_ptr(), sdt, zeros.data_ptr(), g_idx.data_ptr(), d,
            bits, group_size, 1 if signed else 0, dX.data_ptr(), d, ws.data_ptr(),
            ws.numel() * ws.element_size())
    return dX


_LOGITS = {torch.bfloat16: GPTQ_BF16, torch.float16: GPTQ_F16, torch.float32: GPTQ_F32}


def _check_distill(logits, t_idx, t_logits, t_lse, weight):
    ldl = _gpu_rows(logits, "logits", None, tuple(_LOGITS))
    dev = _gpu_device(logits)
    n = logits.shape[0]
    if t_idx.dim() != 2:
        raise ValueError("t_idx must be [n, k]")
    k = t_idx.shape[1]
    _like(t_idx, "t_idx", torch.int32, (n, k), dev)
    _like(t_logits, "t_logits", _F32, (n, k), dev)
    if t_lse is not None:
        _like(t_lse, "t_lse", _F32, (n,), dev)
    if weight is not None:
        _like(weight, "weight", _F32, (n,), dev)
    return ldl, dev, n, k


def _dlogits(t, logits, dev):
    """The gradient's tensor (the logits' own is allowed) and its row stride."""
    if t is None:
        t = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    ldd = _gpu_rows(t, "dlogits", logits.shape[1], (logits.dtype,))
    if t.shape != logits.shape or t.device != dev:
        raise ValueError(f"dlogits must be {tuple(logits.shape)} on {dev}")
    return t, ldd


def gptq_distill_loss(logits: torch.Tensor, t_idx: torch.Tensor, t_logits: torch.Tensor,
                      temperature: float = 1.0, t_lse=None, weight=None, want_grad: bool = False,
                      dlogits=None) -> dict:
    """Divergence of the student's logits [n, vocab] (bfloat16, float16 or
    float32) from a teacher known by the logits t_logits fp32 [n, k] at the ids
    t_idx int32 [n, k] (outside [0, vocab): padding), per row, times weight and
    temperature^2.  t_lse fp32 [n], the teacher's log-sum-exp of its logits /
    temperature, makes what the known ids leave one more class; without it
    the known ids are renormalised.  Returns {"loss": fp32 [n], "stats": fp32
    [n, 2] (for gptq_distill_backward), "dlogits": the gradient of
    sum(loss), or None}; dlogits may be the logits' own tensor."""
    ldl, dev, n, k = _check_distill(logits, t_idx, t_logits, t_lse, weight)
    ldd = 0
    if want_grad or dlogits is not None:
        dlogits, ldd = _dlogits(dlogits, logits, dev)
    loss = torch.empty(n, dtype=_F32, device=dev)
    stats = torch.empty(n, 2, dtype=_F32, device=dev)
    _launch(dev, "gptq_distill_loss", _lib().gptq_distill_loss, logits.data_ptr(),
            _LOGITS[logits.dtype], n, logits.shape[1], ldl, t_idx.data_ptr(), t_logits.data_ptr(), k,
            temperature, None if t_lse is None else t_lse.data_ptr(),
            None if weight is None else weight.data_ptr(), loss.data_ptr(), stats.data_ptr(),
            None if dlogits is None else dlogits.data_ptr(), ldd)
    return dict(loss=loss, stats=stats, dlogits=dlogits)


def gptq_distill_backward(logits: torch.Tensor, stats: torch.Tensor, t_idx: torch.Tensor,
                          t_logits: torch.Tensor, grad: torch.Tensor, temperature: float = 1.0,
                          t_lse=None, weight=None, dlogits=None) -> torch.Tensor:
    """dlogits = grad[row] d loss[row] / d logits from the stats of
    gptq_distill_loss on the same arguments; grad fp32 [n]."""
    ldl, dev, n, k = _check_distill(logits, t_idx, t_logits, t_lse, weight)
    _like(stats, "stats", _F32, (n, 2), dev)
    _like(grad, "grad", _F32, (n,), dev)
    dlogits, ldd = _dlogits(dlogits, logits, dev)
    _launch(dev, "gptq_distill_backward", _lib().gptq_distill_backward, logits.data_ptr(),
            _LOGITS[logits.dtype], n, logits.shape[1], ldl, stats.data_ptr(), t_idx.data_ptr(),
            t_logits.data_ptr(), k, temperature, None if t_lse is None else t_lse.data_ptr(),
            None if weight is None else weight.data_ptr(), grad.data_ptr(), dlogits.data_ptr(), ldd)
    return dlogits


# ---------------------------------------------------------------------------
# Given tokens of rows of logits
# ---------------------------------------------------------------------------

def gptq_token_logprobs_workspace_bytes(n: int, vocab: int, k: int) -> int:
    return int(_lib().gptq_token_logprobs_workspace_bytes(n, vocab, k))


def gptq_token_logprobs(logits: torch.Tensor, tokens=None, k: int = 0, temperature: float = 1.0,
                        ws=None) -> dict:
    """Statistics of the rows of logits [n, vocab] (bfloat16, float16 or
    float32) at a temperature: {"logp": the log probability of tokens int32
    [n] (outside [0, vocab): 0; None without tokens), "entropy", "lse": fp32
    [n], "stats": fp32 [n, 3] (for gptq_token_logprobs_backward), "top_logits":
    fp32 [n, k], "top_idx": int32 [n, k]: the k largest logits, equal ones by
    lower id (None with k = 0)}.  top_idx, top_logits and lse are a teacher's
    t_idx, t_logits and t_lse in gptq_distill_loss."""
    ldl = _gpu_rows(logits, "logits", None, tuple(_LOGITS))
    dev = _gpu_device(logits)
    n, vocab = logits.shape
    if tokens is not None:
        _like(tokens, "tokens", torch.int32, (n,), dev)
    lib = _lib()
    ws, at_ws, ws_bytes = _scratch(ws, lib.gptq_token_logprobs_workspace_bytes(n, vocab, k), dev)
    # (new tensors cost the host half of what views of one cost)
    logp = None if tokens is None else torch.empty(n, dtype=_F32, device=dev)
    entropy, lse = torch.empty(n, dtype=_F32, device=dev), torch.empty(n, dtype=_F32, device=dev)
    stats = torch.empty(n, 3, dtype=_F32, device=dev)
    top = torch.empty(n, k, dtype=_F32, device=dev) if k > 0 else None
    idx = torch.empty(n, k, dtype=torch.int32, device=dev) if k > 0 else None
    _launch(dev, "gptq_token_logprobs", lib.gptq_token_logprobs, logits.data_ptr(),
            _LOGITS[logits.dtype], n, vocab, ldl, None if tokens is None else tokens.data_ptr(),
            temperature, k, None if logp is None else logp.data_ptr(), entropy.data_ptr(),
            lse.data_ptr(), stats.data_ptr(), None if top is None else top.data_ptr(),
            None if idx is None else idx.data_ptr(), at_ws, ws_bytes)
    return dict(logp=logp, entropy=entropy, lse=lse, stats=stats, top_logits=top, top_idx=idx)


def gptq_token_logprobs_backward(logits: torch.Tensor, stats: torch.Tensor, tokens=None,
                                 grad_logp=None, grad_entropy=None, temperature: float = 1.0,
                                 dlogits=None) -> torch.Tensor:
    """The gradient of sum(grad_logp logp + grad_entropy entropy), both fp32
    [n] or None, with respect to the logits, in their dtype, from the stats of
    gptq_token_logprobs on the same arguments; dlogits may be the logits' own
    tensor."""
    ldl = _gpu_rows(logits, "logits", None, tuple(_LOGITS))
    dev = _gpu_device(logits)
    n, vocab = logits.shape
    _like(stats, "stats", _F32, (n, 3), dev)
    if tokens is not None:
        _like(tokens, "tokens", torch.int32, (n,), dev)
    elif grad_logp is not None:
        raise ValueError("grad_logp needs tokens")
    if grad_logp is not None:
        _like(grad_logp, "grad_logp", _F32, (n,), dev)
    if grad_entropy is not None:
        _like(grad_entropy, "grad_entropy", _F32, (n,), dev)
    dlogits, ldd = _dlogits(dlogits, logits, dev)
    _launch(dev, "gptq_token_logprobs_backward", _lib().gptq_token_logprobs_backward,
            logits.data_ptr(), _LOGITS[logits.dtype], n, vocab, ldl, stats.data_ptr(),
            None if tokens is None else tokens.data_ptr(), temperature,
            None if grad_logp is None else grad_logp.data_ptr(),
            None if grad_entropy is None else grad_entropy.data_ptr(), dlogits.data_ptr(), ldd)
    return dlogits


# ---------------------------------------------------------------------------
# Layers and activations in 4-bit floating point
# ---------------------------------------------------------------------------

_MX_BF16, _MX_ROUND, _MX_CODES = range(3)


def _check_mx(codes, scales, name, blocks, dev):
    """Checks a matrix [rows, 32 blocks] in the stored format; returns its rows."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError(f"{name} codes must be [rows, 16 blocks]")
    rows = codes.shape[0]
    _like(codes, f"{name} codes", torch.uint8, (rows, 16 * blocks), dev)
    _like(scales, f"{name} scales", torch.uint8, (rows, blocks), dev)
    return rows


def _mx_input(X, x_scales, quantize_x, blocks):
    """Checks the activations of a product with layers of `blocks` blocks (None:
    as X has); returns (form, row stride, scales' pointer, n, d, device)."""
    if isinstance(X, torch.Tensor) and X.dtype is torch.uint8:
        if x_scales is None or quantize_x:
            raise ValueError("X as codes needs x_scales, and is quantized already")
        dev = _gpu_device(X)
        n = _check_mx(X, x_scales, "X", blocks, dev)
        # the fewest columns with these blocks, which alone count here: the widest layers end
        # inside their last one
        return _MX_CODES, 0, x_scales.data_ptr(), n, 32 * blocks - 31, dev
    if x_scales is not None:
        raise ValueError("x_scales belongs to X as codes (uint8)")
    ldx = _gpu_rows(X, "X")
    dev = _gpu_device(X)
    n, d = X.shape
    if -(-d // 32) != blocks:
        raise ValueError(f"X has {d} columns, the layer {blocks} blocks of 32")
    return (_MX_ROUND if quantize_x else _MX_BF16), ldx, None, n, d, dev


def gptq_mx_matmul_workspace_bytes(n: int, m: int, d: int, x_form: int) -> int:
    return int(_lib().gptq_mx_matmul_workspace_bytes(n, m, d, x_form))


def gptq_mx_matmul_t_workspace_bytes(n: int, m: int, d: int) -> int:
    return int(_lib().gptq_mx_matmul_t_workspace_bytes(n, m, d))


def gptq_mx_gated_workspace_bytes(n: int, m: int, d: int, x_form: int) -> int:
    return int(_lib().gptq_mx_gated_workspace_bytes(n, m, d, x_form))


def gptq_mx_gated_backward_workspace_bytes(n: int, m: int, d: int) -> int:
    return int(_lib().gptq_mx_gated_backward_workspace_bytes(n, m, d))


def gptq_mx_quantize(X: torch.Tensor, want_hat: bool = False, codes=None, scales=None,
                        hat=None) -> dict:
    """X [n, d] (bfloat16, float16 or float32) in 4-bit floating point: {"codes":
    uint8 [n, 16 ceil(d / 32)], two values a byte, the even column's in the
    lower half, "scales": uint8 [n, ceil(d / 32)], 127 + the power of two of
    each block of 32 columns (255: a block with a value that is not finite),
    and with want_hat (or hat given) "hat": the values that the codes stand
    for, in X's dtype}."""
    ldx = _gpu_rows(X, "X", None, tuple(_LOGITS))
    dev = _gpu_device(X)
    n, d = X.shape
    blocks = -(-d // 32)
    codes = _out(codes, "codes", torch.uint8, (n, 16 * blocks), dev)
    scales = _out(scales, "scales", torch.uint8, (n, blocks), dev)
    if want_hat or hat is not None:
        hat = _out(hat, "hat", X.dtype, (n, d), dev)
    _launch(dev, "gptq_mx_quantize", _lib().gptq_mx_quantize, X.data_ptr(), _LOGITS[X.dtype],
            n, d, ldx, codes.data_ptr(), scales.data_ptr(), None if hat is None else hat.data_ptr(),
            d)
    out = dict(codes=codes, scales=scales)
    if hat is not None:
        out["hat"] = hat
    return out


def gptq_mx_matmul(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      quantize_x: bool = False, x_scales=None, Y=None, out_dtype=torch.float32,
                      ws=None) -> torch.Tensor:
    """Y [n, m] = X W^T for a layer W [m, d] as gptq_mx_quantize stores it.

    X is bfloat16 [n, d], taken as it is or (quantize_x) rounded to 4 bits as
    gptq_mx_quantize does, or the codes of that call with their x_scales.
    Y is float32 or bfloat16 (out_dtype, or the given Y's)."""
    if scales.dim() != 2:
        raise ValueError("scales must be [m, blocks]")
    form, ldx, xs, n, d, dev = _mx_input(X, x_scales, quantize_x, scales.shape[1])
    m = _check_mx(codes, scales, "layer", scales.shape[1], dev)
    if Y is not None:
        out_dtype = Y.dtype
    if out_dtype is not _F32 and out_dtype is not _BF16:
        raise TypeError(f"Y must be float32 or bfloat16, got {out_dtype}")
    lib = _lib()
    ws, at_ws, ws_bytes = _scratch(ws, lib.gptq_mx_matmul_workspace_bytes(n, m, d, form), dev)
    Y = _out(Y, "Y", out_dtype, (n, m), dev)
    _launch(dev, "gptq_mx_matmul", lib.gptq_mx_matmul, X.data_ptr(), form, xs, n, d, ldx,
            codes.data_ptr(), scales.data_ptr(), m, Y.data_ptr(),
            GPTQ_F32 if out_dtype is _F32 else GPTQ_BF16, m, at_ws, ws_bytes)
    return Y


def gptq_mx_matmul_t(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, d: int,
                        dX=None, ws=None) -> torch.Tensor:
    """dX bf16 [n, d] = dY W for dY bf16 [n, m]: the gradient of
    gptq_mx_matmul with respect to its activations."""
    ldy = _gpu_rows(dY, "dY")
    dev = _gpu_device(dY)
    n, m = dY.shape
    if _check_mx(codes, scales, "layer", -(-d // 32), dev) != m:
        raise ValueError(f"the layer must have {m} rows")
    lib = _lib()
    ws = _enough(ws, lib.gptq_mx_matmul_t_workspace_bytes(n, m, d), dev)
    dX = _out(dX, "dX", _BF16, (n, d), dev)
    _launch(dev, "gptq_mx_matmul_t", lib.gptq_mx_matmul_t, dY.data_ptr(), GPTQ_BF16, n, m, ldy,
            codes.data_ptr(), scales.data_ptr(), d, dX.data_ptr(), d, ws.data_ptr(),
            ws.numel() * ws.element_size())
    return dX


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def gptq_mx_gated(X: torch.Tensor, gate_codes: torch.Tensor, gate_scales: torch.Tensor,
                     up_codes: torch.Tensor, up_scales: torch.Tensor, activation: str = "silu",
                     quantize_x: bool = False, x_scales=None, want_parts: bool = False, Y=None,
                     ws=None):
    """Y bf16 [n, m] = act(G) * U with G = X W_gate^T and U = X W_up^T, for two
    layers [m, d] as gptq_mx_quantize stores them; X, quantize_x and
    x_scales as in gptq_mx_matmul.  Returns Y, or (Y, G, U) with both
    factors in bf16 where want_parts is set (gptq_mx_gated_backward needs
    them)."""
    act = _activation(activation)
    if gate_scales.dim() != 2:
        raise ValueError("gate_scales must be [m, blocks]")
    blocks = gate_scales.shape[1]
    form, ldx, xs, n, d, dev = _mx_input(X, x_scales, quantize_x, blocks)
    m = _check_mx(gate_codes, gate_scales, "gate", blocks, dev)
    if _check_mx(up_codes, up_scales, "up", blocks, dev) != m:
        raise ValueError("gate and up must have the same shape")
    lib = _lib()
    ws, at_ws, ws_bytes = _scratch(ws, lib.gptq_mx_gated_workspace_bytes(n, m, d, form), dev)
    Y = _out(Y, "Y", _BF16, (n, m), dev)
    G = U = None
    if want_parts:
        G = torch.empty(n, m, dtype=_BF16, device=dev)
        U = torch.empty(n, m, dtype=_BF16, device=dev)
    _launch(dev, "gptq_mx_gated", lib.gptq_mx_gated, X.data_ptr(), form, xs, n, d, ldx,
            gate_codes.data_ptr(), gate_scales.data_ptr(), up_codes.data_ptr(), up_scales.data_ptr(),
            m, act, Y.data_ptr(), m, None if G is None else G.data_ptr(),
            None if U is None else U.data_ptr(), m, at_ws, ws_bytes)
    return (Y, G, U) if want_parts else Y


def gptq_mx_gated_backward(dY: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                              gate_codes: torch.Tensor, gate_scales: torch.Tensor,
                              up_codes: torch.Tensor, up_scales: torch.Tensor, d: int,
                              activation: str = "silu", need_dx: bool = True, dX=None, ws=None):
    """Gradients of gptq_mx_gated from dY bf16 [n, m] and the G and U it
    returned: (dX bf16 [n, d] or None, dG, dU bf16 [n, m]: views of one
    buffer, with a row stride beyond m)."""
    act = _activation(activation)
    ldy = _gpu_rows(dY, "dY")
    dev = _gpu_device(dY)
    n, m = dY.shape
    ldg = _gpu_rows(G, "G", m)
    if _gpu_rows(U, "U", m) != ldg or G.shape != dY.shape or U.shape != dY.shape or \
            G.device != dev or U.device != dev:
        raise ValueError(f"G and U must be {tuple(dY.shape)} with one row stride, on {dev}")
    lib = _lib()
    if need_dx:
        blocks = -(-d // 32)
        if _check_mx(gate_codes, gate_scales, "gate", blocks, dev) != m or \
                _check_mx(up_codes, up_scales, "up", blocks, dev) != m:
            raise ValueError(f"gate and up must have {m} rows")
        ws = _enough(ws, lib.gptq_mx_gated_backward_workspace_bytes(n, m, d), dev)
        dX = _out(dX, "dX", _BF16, (n, d), dev)
    else:
        dX = ws = None
    mp = -(-m // 64) * 64
    grads = torch.empty(n, 2 * mp, dtype=_BF16, device=dev)
    _launch(dev, "gptq_mx_gated_backward", lib.gptq_mx_gated_backward, dY.data_ptr(),
            GPTQ_BF16, n, m, ldy, G.data_ptr(), U.data_ptr(), ldg,
            gate_codes.data_ptr() if need_dx else None, gate_scales.data_ptr() if need_dx else None,
            up_codes.data_ptr() if need_dx else None, up_scales.data_ptr() if need_dx else None, d,
            act, None if dX is None else dX.data_ptr(), d, grads.data_ptr(),
            None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size())
    return dX, grads[:, :m], grads[:, mp:mp + m]


def gptq_quantize_stack(Ws, X: torch.Tensor, params, activation: str = "none",
                        ws=None) -> dict:
    """Quantize the linear layers Ws[0], Ws[1], ... in order, each on the
    bf16 outputs of the quantized layer before it (X feeds the first).
    params: one dict of gptq_quantize_layer settings per layer (or one dict
    for all).  Returns {"layers": [outputs per layer], "layer_err": [floats],
    "X_out": bf16 [n, m_last] (the next layer's inputs)}."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if isinstance(params, dict):
        params = [params] * len(Ws)
    if len(params) != len(Ws) or not Ws:
        raise ValueError("one params dict per layer")
    if X.dim() != 2 or X.dtype != torch.bfloat16 or not X.is_contiguous():
        raise ValueError("X must be a contiguous bf16 [n, d] tensor")
    dev = X.device
    n = X.shape[0]
    arr = (_StackLayer * len(Ws))()
    outs = []
    for i, (W, p) in enumerate(zip(Ws, params)):
        if W.dim() != 2 or W.device != dev:
            raise ValueError("each W must be [m, d] on X's device")
        m, d = W.shape
        ldw = _row_stride(W, "W")
        g = p.get("group_size", -1)
        bits = p.get("bits", 4)
        ng = 1 if g == -1 else -(-d // g)
        o = dict(qweight=torch.empty(m, -(-d * bits // 32), dtype=torch.int32, device=dev),
                 scales=torch.empty(m, ng, dtype=torch.float32, device=dev),
                 zeros=torch.empty(m, ng, dtype=torch.uint8, device=dev),
                 g_idx=torch.empty(d, dtype=torch.int32, device=dev))
        outs.append(o)
        grid = p.get("grid", "minmax")
        fs, fz = p.get("fixed_scales"), p.get("fixed_zeros")
        if grid == "fixed":
            _expect(fs, "fixed_scales", torch.float32, (m, ng), dev)
            _expect(fz, "fixed_zeros", torch.uint8, (m, ng), dev)
        pp = _params(bits, g, p.get("blocksize", 128), p.get("percdamp", 0.01),
                     p.get("act_order", False), grid, p.get("static_groups", False),
                     fs, fz)
        arr[i] = _StackLayer(W.data_ptr(), _dtype_code(W), m, d, ldw, pp,
                             o["qweight"].data_ptr(), o["scales"].data_ptr(),
                             o["zeros"].data_ptr(), o["g_idx"].data_ptr())
    lib = _lib()
    need = lib.gptq_stack_workspace_bytes(arr, len(Ws), n)
    if need == 0:
        raise GPTQError(GPTQ_ERR_INVALID_ARG, "gptq_stack_workspace_bytes")
    if ws is None or ws.numel() < need:
        ws = _workspace(need, dev)
    X_out = torch.empty(n, Ws[-1].shape[0], dtype=torch.bfloat16, device=dev)
    errs = (ctypes.c_double * len(Ws))()
    st = lib.gptq_quantize_stack(arr, len(Ws), _dev_ptr(X), n, ACTIVATIONS[activation],
                                 _dev_ptr(X_out), errs, _dev_ptr(ws), ws.numel(),
                                 _stream(dev))
    _check(st, "gptq_quantize_stack")
    return dict(layers=outs, layer_err=[float(e) for e in errs], X_out=X_out)


def gptq_trace_enable(enable: bool = True) -> None:
    """Record per-phase GPU time (hipEvents around each launch group)."""
    _check(_lib().gptq_trace_enable(int(bool(enable))), "gptq_trace_enable")


def gptq_trace_read(reset: bool = True) -> dict:
    """{phase: (milliseconds, launch groups)} since the last reset."""
    ms = (ctypes.c_double * len(TRACE_PHASES))()
    n = (ctypes.c_int64 * len(TRACE_PHASES))()
    _check(_lib().gptq_trace_read(ms, n, int(bool(reset))), "gptq_trace_read")
    return {p: (float(ms[i]), int(n[i])) for i, p in enumerate(TRACE_PHASES)}
