"""Block-quantized matrix x vector products for AMD MI355X (gfx950).

Python binding of ``libqmv.so`` (hand-written HIP, C ABI in
``include/qmv.h``).  This module only marshals arguments: it checks tensor
devices, dtypes and shapes, passes raw device pointers and the current HIP
stream to the library, and turns a non-OK return code into ``QmvError``.
Every step of the computation runs in the library's kernels; there is no
fallback of any kind, and importing this package fails loudly when the
library has not been built.

A call runs on `stream`, or on the current stream.  The tensors that it makes
(outputs, workspaces) come from that stream's pool.  As for any work on
another stream, the caller has it wait for what makes the inputs, waits for
it before the outputs are read, and keeps the inputs until it is done.

Entry points (same names as the C ABI):
  qmv_q8_0 / qmv_q4_0 / qmv_q4_1   float block-quantized matvec, batch 1..8
  qmv_q4_k                         the same for Q4_K super-blocks (256 weights, 144 bytes)
  qmv_q6_k                         the same for Q6_K super-blocks (256 weights, 210 bytes)
  qmv_matvec_path                  the same with the kernel family chosen
                                   (PATH_AUTO / PATH_FMA / PATH_MFMA)
  qmv_matvec_xt                    the same with fp32, fp16 or bf16 activations
  qmv_i8_requant                   int8 matvec + per-channel gemmlowp requant
  qmv_i8_requant_lut               the same through a frozen int8 lookup table
  qmv_moe                          grouped MoE expert matvec
  qmv_moe_xt                       the same with fp32, fp16 or bf16 activations
  qmv_moe_swiglu                   MoE gate||up with the SwiGLU step fused
  qmv_moe_swiglu_xt                the same with fp32, fp16 or bf16 activations
  qmv_moe_combine                  MoE down with the router-weighted combine
  qmv_group_plan                   items sorted by group: the plan of the grouped products
  qmv_moe_grouped                  expert products grouped by expert, any number of tokens
  qmv_moe_grouped_swiglu           gate||up with the SwiGLU step fused, grouped by expert
  qmv_moe_weighted_sum             router-weighted sum over a token's slots
  qmv_lora                         shared projection with a low-rank adapter per token
  qmv_spec_verify                  drafted tokens against the target's probabilities
  qmv_cache_write / qmv_cache_read    keys and values into the pages of a quantized cache, and back (serving.py)
  qmv_cache_attention              attention of new tokens over such a cache (serving.py)
  qmv_logprobs                     log probabilities, entropy, most probable tokens (serving.py)
  qmv_dequant                      stored blocks -> fp32 (test/inspection aid)
  qmv_stream_read                  stream-read ceiling of the device (measurement aid)
  qmv_chain                        batch-1 matvec stages in one persistent launch
  qmv_chain_noalloc                the same with library-held barrier words (no workspace)
"""
import ctypes
import os

__all__ = ["QmvError", "qmv_q8_0", "qmv_q4_0", "qmv_q4_1", "qmv_q4_k", "qmv_q6_k", "qmv_matvec_path", "qmv_matvec_xt", "PATH_AUTO",
           "PATH_FMA", "PATH_MFMA", "X_F32", "X_F16", "X_BF16", "qmv_i8_requant", "qmv_i8_requant_lut",
           "qmv_moe", "qmv_moe_xt", "qmv_moe_swiglu", "qmv_moe_swiglu_xt", "qmv_moe_combine",
           "GroupPlan", "qmv_group_plan", "qmv_moe_grouped", "qmv_moe_grouped_swiglu", "qmv_moe_weighted_sum",
           "qmv_lora", "qmv_spec_verify",
           "qmv_dequant", "qmv_stream_read", "qmv_chain", "qmv_chain_noalloc", "ChainStage", "CHAIN_WORKSPACE_BYTES", "abi_version", "last_error",
           "library_path", "lib", "Q8_0", "Q4_0", "Q4_1", "Q4_K", "Q6_K", "FORMATS", "BLOCK_BYTES", "row_bytes",
           "KVCache", "Logprobs", "cache_page_bytes", "serving"]      # serving's own __all__ has its entry points

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libqmv.so")

Q8_0, Q4_0, Q4_1, Q4_K, Q6_K = 0, 1, 2, 3, 4
FORMATS = {"q8_0": Q8_0, "q4_0": Q4_0, "q4_1": Q4_1, "q4_k": Q4_K, "q6_k": Q6_K}
BLOCK_BYTES = {Q8_0: 34, Q4_0: 18, Q4_1: 20}      # per 32 weights
SUPER_BLOCK = {Q4_K: (256, 144), Q6_K: (256, 210)}   # (weights, bytes) per super-block


def row_bytes(fmt, n_cols):
    """Stored bytes of one row of n_cols weights (0 for an unknown format)."""
    f = FORMATS.get(fmt, fmt)
    if f in SUPER_BLOCK:
        w, b = SUPER_BLOCK[f]
        return n_cols // w * b
    return n_cols // 32 * BLOCK_BYTES.get(f, 0)


PATH_AUTO, PATH_FMA, PATH_MFMA = 0, 1, 2
X_F32, X_F16, X_BF16 = 0, 1, 2
_ERRORS = {1: "QMV_EINVAL", 2: "QMV_EALIGN", 3: "QMV_EUNSUPPORTED", 4: "QMV_EHIP"}
CHAIN_WORKSPACE_BYTES = 40960


class ChainStage(ctypes.Structure):
    """qmv_chain_stage of include/qmv.h."""
    _fields_ = [("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int64),
                ("wait", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QmvError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{_ERRORS.get(code, code)}: {msg}")
        self.code = code


def library_path():
    return _LIB_PATH


def _open():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built: run __graft_entry__.build() "
                          "(hipcc --offload-arch=gfx950) first")
    L = ctypes.CDLL(_LIB_PATH)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    for name in ("qmv_q8_0", "qmv_q4_0", "qmv_q4_1", "qmv_q4_k", "qmv_q6_k"):
        f = getattr(L, name)
        f.argtypes = [P, i64, i64, P, i64, i32, P, i64, P]
        f.restype = i32
    L.qmv_matvec_path.argtypes = [ctypes.c_int, P, i64, i64, P, i64, i32, P, i64, i32, P]
    L.qmv_matvec_path.restype = i32
    L.qmv_matvec_xt.argtypes = [ctypes.c_int, P, i64, i64, P, i32, i64, i32, P, i64, i32, P]
    L.qmv_matvec_xt.restype = i32
    L.qmv_i8_requant.argtypes = [P, i64, i64, P, i64, i32, P, P, P, i64, P]
    L.qmv_i8_requant.restype = i32
    L.qmv_i8_requant_lut.argtypes = [P, i64, i64, P, i64, i32, P, P, P, P, i64, P]
    L.qmv_i8_requant_lut.restype = i32
    L.qmv_moe.argtypes = [ctypes.c_int, P, i64, i32, i64, i64, P, i32, i32, P, i64, i64, P, P]
    L.qmv_moe.restype = i32
    L.qmv_moe_swiglu.argtypes = [ctypes.c_int, P, i64, i32, i64, i64, P, i32, i32, P, i64, i64, P, P]
    L.qmv_moe_swiglu.restype = i32
    for name in ("qmv_moe_xt", "qmv_moe_swiglu_xt"):
        f = getattr(L, name)
        f.argtypes = [ctypes.c_int, P, i64, i32, i64, i64, P, i32, i32, P, i32, i64, i64, P, P]
        f.restype = i32
    L.qmv_moe_combine.argtypes = [ctypes.c_int, P, i64, i32, i64, i64, P, P, i32, i32, P, i64, i64, P, P]
    L.qmv_moe_combine.restype = i32
    sz = ctypes.c_size_t
    L.qmv_group_plan_bytes.argtypes = [i64, i32]
    L.qmv_lora_workspace_bytes.argtypes = [i64, i32, i32]
    L.qmv_spec_verify_workspace_bytes.argtypes = [i64, i32, i64]
    for name in ("qmv_group_plan_bytes", "qmv_lora_workspace_bytes", "qmv_spec_verify_workspace_bytes"):
        getattr(L, name).restype = sz
    L.qmv_group_plan.argtypes = [P, i64, i32, P, sz, P]
    L.qmv_group_plan.restype = i32
    for name in ("qmv_moe_grouped", "qmv_moe_grouped_swiglu"):
        f = getattr(L, name)
        f.argtypes = [ctypes.c_int, P, i64, i32, i64, i64, P, i64, i32, P, i32, i64, i64, P, i32, P]
        f.restype = i32
    L.qmv_moe_weighted_sum.argtypes = [P, i32, P, i64, i32, i64, P, i32, P]
    L.qmv_moe_weighted_sum.restype = i32
    L.qmv_lora.argtypes = [ctypes.c_int, P, i64, i64, P, i32, i64, i64, P, P, i32, i32, i32, P, P, P, i64, P, sz, P]
    L.qmv_lora.restype = i32
    L.qmv_spec_verify.argtypes = [P, i32, i64, i64, P, i64, i64, P, P, P, P, i64, i32, i64, P, P, P, sz, P]
    L.qmv_spec_verify.restype = i32
    L.qmv_dequant.argtypes = [ctypes.c_int, P, i64, i64, P, P]
    L.qmv_dequant.restype = i32
    L.qmv_stream_read.argtypes = [P, ctypes.c_size_t, P, ctypes.c_size_t, P]
    L.qmv_stream_read.restype = i32
    L.qmv_chain.argtypes = [ctypes.c_int, P, i32, P, ctypes.c_size_t, P]
    L.qmv_chain.restype = i32
    L.qmv_chain_noalloc.argtypes = [ctypes.c_int, P, i32, P]
    L.qmv_chain_noalloc.restype = i32
    L.qmv_last_error.argtypes = []
    L.qmv_last_error.restype = ctypes.c_char_p
    L.qmv_abi_version.argtypes = []
    L.qmv_abi_version.restype = i32
    return L


_lib = _open()


def lib():
    """The raw ctypes handle (C signatures as in include/qmv.h)."""
    return _lib


def last_error():
    return _lib.qmv_last_error().decode()


def abi_version():
    return int(_lib.qmv_abi_version())


def _check(rc):
    if rc != 0:
        raise QmvError(rc, last_error())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtype):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _new(shape, dtype, like, stream, returned=True):
    """A new tensor on like's device for a call on `stream` (None: the current
    stream), from the pool of that stream.  A block of the current stream's
    pool may still be in use by work queued there, which another stream does
    not wait for, and would go back there while that stream still writes it.
    A tensor that is returned is read on the current stream too, once that
    has waited, and does not go back before."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    here = torch.cuda.current_stream(like.device)
    if stream.cuda_stream == here.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    if returned:
        t.record_stream(here)
    return t


def _rows2d(t, name, K):
    """[K] or [B, K] with unit inner stride -> (tensor2d, B, ld)."""
    t2 = t.unsqueeze(0) if t.dim() == 1 else t
    if t2.dim() != 2 or t2.shape[1] != K or t2.stride(1) != 1:
        raise ValueError(f"{name} must be [K] or [B, K] with K={K} and unit inner stride")
    return t2, t2.shape[0], t2.stride(0) if t2.shape[0] > 1 else K


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _matvec(cfn, fmt, W, n_rows, n_cols, x, y, stream):
    torch = _torch()
    _dev(W, "W", torch.uint8)
    _dev(x, "x", torch.float32)
    need = n_rows * row_bytes(fmt, n_cols)
    if W.numel() * W.element_size() < need or not W.is_contiguous():
        raise ValueError(f"W must be contiguous and hold {need} bytes")
    x2, B, ldx = _rows2d(x, "x", n_cols)
    if y is None:
        y = _new((B, n_rows), torch.float32, x, stream)
    _dev(y, "y", torch.float32)
    y2, By, ldy = _rows2d(y, "y", n_rows)
    if By != B:
        raise ValueError("y must have as many rows as x")
    _check(cfn(W.data_ptr(), n_rows, n_cols, x2.data_ptr(), ldx, B, y2.data_ptr(), ldy, _stream(stream)))
    return y


def qmv_q8_0(W, n_rows, n_cols, x, y=None, stream=None):
    """y[b] = DEQ_Q8_0(W) @ x[b]; x float32 [K] or [B, K] (B <= 8)."""
    return _matvec(_lib.qmv_q8_0, Q8_0, W, n_rows, n_cols, x, y, stream)


def qmv_q4_0(W, n_rows, n_cols, x, y=None, stream=None):
    """y[b] = DEQ_Q4_0(W) @ x[b]; x float32 [K] or [B, K] (B <= 8)."""
    return _matvec(_lib.qmv_q4_0, Q4_0, W, n_rows, n_cols, x, y, stream)


def qmv_q4_1(W, n_rows, n_cols, x, y=None, stream=None):
    """y[b] = DEQ_Q4_1(W) @ x[b]; x float32 [K] or [B, K] (B <= 8)."""
    return _matvec(_lib.qmv_q4_1, Q4_1, W, n_rows, n_cols, x, y, stream)


def qmv_q4_k(W, n_rows, n_cols, x, y=None, stream=None):
    """y[b] = DEQ_Q4_K(W) @ x[b]; x float32 [K] or [B, K] (B <= 8), K a
    multiple of 256."""
    return _matvec(_lib.qmv_q4_k, Q4_K, W, n_rows, n_cols, x, y, stream)


def qmv_q6_k(W, n_rows, n_cols, x, y=None, stream=None):
    """y[b] = DEQ_Q6_K(W) @ x[b]; x float32 [K] or [B, K] (B <= 8), K a
    multiple of 256."""
    return _matvec(_lib.qmv_q6_k, Q6_K, W, n_rows, n_cols, x, y, stream)


def qmv_matvec_path(fmt, W, n_rows, n_cols, x, path, y=None, stream=None):
    """As qmv_q8_0/q4_0/q4_1/q4_k/q6_k for format fmt (Q8_0, Q4_0, Q4_1,
    Q4_K, Q6_K or its name) with the kernel family `path` (PATH_AUTO,
    PATH_FMA or PATH_MFMA)."""
    f = FORMATS.get(fmt, fmt)
    if f not in FORMATS.values():
        raise ValueError(f"unknown format {fmt!r}")

    def cfn(*a):
        return _lib.qmv_matvec_path(f, *a[:-1], path, a[-1])
    return _matvec(cfn, f, W, n_rows, n_cols, x, y, stream)


def qmv_matvec_xt(fmt, W, n_rows, n_cols, x, path=PATH_AUTO, y=None, stream=None):
    """As qmv_matvec_path with x float32, float16 or bfloat16 [K] or [B, K]
    (widened to fp32 exactly); y is float32."""
    torch = _torch()
    f = FORMATS.get(fmt, fmt)
    if f not in FORMATS.values():
        raise ValueError(f"unknown format {fmt!r}")
    xt = {torch.float32: X_F32, torch.float16: X_F16, torch.bfloat16: X_BF16}.get(x.dtype)
    if xt is None:
        raise ValueError(f"x must be float32, float16 or bfloat16 (got {x.dtype})")
    _dev(W, "W", torch.uint8)
    _dev(x, "x", x.dtype)
    need = n_rows * row_bytes(f, n_cols)
    if W.numel() * W.element_size() < need or not W.is_contiguous():
        raise ValueError(f"W must be contiguous and hold {need} bytes")
    x2, B, ldx = _rows2d(x, "x", n_cols)
    if y is None:
        y = _new((B, n_rows), torch.float32, x, stream)
    _dev(y, "y", torch.float32)
    y2, By, ldy = _rows2d(y, "y", n_rows)
    if By != B:
        raise ValueError("y must have as many rows as x")
    _check(_lib.qmv_matvec_xt(f, W.data_ptr(), n_rows, n_cols, x2.data_ptr(), xt, ldx, B, y2.data_ptr(), ldy, path,
                              _stream(stream)))
    return y


def qmv_i8_requant(W, x, mult, shift, y=None, stream=None):
    """int8 [N, K] weights x int8 [K] or [B, K] activations, per-row requant
    (mult, shift int32 [N]) -> int8 [B, N]."""
    return _i8(W, x, mult, shift, None, y, stream)


def qmv_i8_requant_lut(W, x, mult, shift, lut, y=None, stream=None):
    """qmv_i8_requant with the outputs mapped through a frozen table:
    y = lut[y_requant + 128]; lut int8 [256] on the GPU."""
    return _i8(W, x, mult, shift, lut, y, stream)


def _i8(W, x, mult, shift, lut, y, stream):
    torch = _torch()
    _dev(W, "W", torch.int8)
    _dev(x, "x", torch.int8)
    _dev(mult, "mult", torch.int32)
    _dev(shift, "shift", torch.int32)
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous [N, K] tensor")
    N, K = W.shape
    if mult.numel() != N or shift.numel() != N or not mult.is_contiguous() or not shift.is_contiguous():
        raise ValueError("mult and shift must be contiguous [N]")
    x2, B, ldx = _rows2d(x, "x", K)
    if y is None:
        y = _new((B, N), torch.int8, x, stream)
    _dev(y, "y", torch.int8)
    y2, By, ldy = _rows2d(y, "y", N)
    if By != B:
        raise ValueError("y must have as many rows as x")
    if lut is None:
        _check(_lib.qmv_i8_requant(W.data_ptr(), N, K, x2.data_ptr(), ldx, B, mult.data_ptr(), shift.data_ptr(),
                                   y2.data_ptr(), ldy, _stream(stream)))
    else:
        _dev(lut, "lut", torch.int8)
        if lut.numel() != 256 or not lut.is_contiguous():
            raise ValueError("lut must be a contiguous int8 [256] tensor")
        _check(_lib.qmv_i8_requant_lut(W.data_ptr(), N, K, x2.data_ptr(), ldx, B, mult.data_ptr(), shift.data_ptr(),
                                       lut.data_ptr(), y2.data_ptr(), ldy, _stream(stream)))
    return y


def _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, rows, n_cols, expert_ids, x, x_types=None):
    torch = _torch()
    fmt = _fmt(fmt)
    _dev(W_experts, "W_experts", torch.uint8)
    _dev(expert_ids, "expert_ids", torch.int32)
    if x_types is None:
        _dev(x, "x", torch.float32)
    else:
        _dev(x, "x", x.dtype)
        if x.dtype not in x_types:
            raise ValueError("x must be float32, float16 or bfloat16")
    if not W_experts.is_contiguous() or not expert_ids.is_contiguous() or not x.is_contiguous():
        raise ValueError("W_experts, expert_ids and x must be contiguous")
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [B, top_k]")
    B, T = expert_ids.shape
    if x.dim() == 2 and x.shape == (B, n_cols):
        st_tok, st_slot = n_cols, 0
    elif x.dim() == 3 and x.shape == (B, T, n_cols):
        st_tok, st_slot = T * n_cols, n_cols
    else:
        raise ValueError("x must be [B, K] or [B, top_k, K]")
    if W_experts.numel() < (n_experts - 1) * expert_stride_bytes + rows * row_bytes(fmt, n_cols):
        raise ValueError("W_experts is smaller than n_experts expert matrices")
    return torch, fmt, B, T, st_tok, st_slot


def _x_types(torch):
    return {torch.float32: X_F32, torch.float16: X_F16, torch.bfloat16: X_BF16}


def qmv_moe_xt(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols, expert_ids, x, y=None, stream=None):
    """qmv_moe with x float32, float16 or bfloat16 ([B, K] or [B, top_k, K])."""
    torch = _torch()
    xt = _x_types(torch)
    torch, fmt, B, T, st_tok, st_slot = _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols,
                                                  expert_ids, x, xt)
    if y is None:
        y = _new((B, T, n_rows), torch.float32, x, stream)
    _dev(y, "y", torch.float32)
    if y.shape != (B, T, n_rows) or not y.is_contiguous():
        raise ValueError("y must be a contiguous [B, top_k, n_rows] tensor")
    _check(_lib.qmv_moe_xt(fmt, W_experts.data_ptr(), expert_stride_bytes, n_experts, n_rows, n_cols,
                           expert_ids.data_ptr(), B, T, x.data_ptr(), xt[x.dtype], st_tok, st_slot, y.data_ptr(),
                           _stream(stream)))
    return y


def qmv_moe_swiglu_xt(fmt, W_experts, expert_stride_bytes, n_experts, n_ff, n_cols, expert_ids, x, h=None,
                      stream=None):
    """qmv_moe_swiglu with x float32, float16 or bfloat16."""
    torch = _torch()
    xt = _x_types(torch)
    torch, fmt, B, T, st_tok, st_slot = _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, 2 * n_ff, n_cols,
                                                  expert_ids, x, xt)
    if h is None:
        h = _new((B, T, n_ff), torch.float32, x, stream)
    _dev(h, "h", torch.float32)
    if h.shape != (B, T, n_ff) or not h.is_contiguous():
        raise ValueError("h must be a contiguous [B, top_k, n_ff] tensor")
    _check(_lib.qmv_moe_swiglu_xt(fmt, W_experts.data_ptr(), expert_stride_bytes, n_experts, n_ff, n_cols,
                                  expert_ids.data_ptr(), B, T, x.data_ptr(), xt[x.dtype], st_tok, st_slot,
                                  h.data_ptr(), _stream(stream)))
    return h


def qmv_moe_swiglu(fmt, W_experts, expert_stride_bytes, n_experts, n_ff, n_cols, expert_ids, x, h=None,
                   stream=None):
    """MoE gate||up with SwiGLU: every expert holds 2*n_ff rows (gate rows,
    then up rows); returns h float32 [B, top_k, n_ff] = SiLU(gate x) * (up x).
    x as qmv_moe."""
    torch, fmt, B, T, st_tok, st_slot = _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, 2 * n_ff, n_cols,
                                                  expert_ids, x)
    if h is None:
        h = _new((B, T, n_ff), torch.float32, x, stream)
    _dev(h, "h", torch.float32)
    if h.shape != (B, T, n_ff) or not h.is_contiguous():
        raise ValueError("h must be a contiguous [B, top_k, n_ff] tensor")
    _check(_lib.qmv_moe_swiglu(fmt, W_experts.data_ptr(), expert_stride_bytes, n_experts, n_ff, n_cols,
                               expert_ids.data_ptr(), B, T, x.data_ptr(), st_tok, st_slot, h.data_ptr(),
                               _stream(stream)))
    return h


def qmv_moe_combine(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols, expert_ids, weights, x,
                    out=None, stream=None):
    """MoE down with the router-weighted combine: out float32 [B, n_rows] =
    sum_s weights[b, s] * DEQ(W_{ids[b,s]}) x_{b,s}.  weights float32
    [B, top_k] on the GPU; x as qmv_moe."""
    torch, fmt, B, T, st_tok, st_slot = _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols,
                                                  expert_ids, x)
    _dev(weights, "weights", torch.float32)
    if weights.shape != (B, T) or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous [B, top_k] tensor")
    if out is None:
        out = _new((B, n_rows), torch.float32, x, stream)
    _dev(out, "out", torch.float32)
    if out.shape != (B, n_rows) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, n_rows] tensor")
    _check(_lib.qmv_moe_combine(fmt, W_experts.data_ptr(), expert_stride_bytes, n_experts, n_rows, n_cols,
                                expert_ids.data_ptr(), weights.data_ptr(), B, T, x.data_ptr(), st_tok, st_slot,
                                out.data_ptr(), _stream(stream)))
    return out


def qmv_moe(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols, expert_ids, x, y=None,
            stream=None):
    """Grouped MoE expert matvec.

    expert_ids: int32 [B, top_k] on the GPU.  x: float32 [B, K] (one input per
    token, gate/up) or [B, top_k, K] (one input per token and slot, down).
    Returns y float32 [B, top_k, n_rows]."""
    torch, fmt, B, T, st_tok, st_slot = _moe_args(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols,
                                                  expert_ids, x)
    if y is None:
        y = _new((B, T, n_rows), torch.float32, x, stream)
    _dev(y, "y", torch.float32)
    if y.shape != (B, T, n_rows) or not y.is_contiguous():
        raise ValueError("y must be a contiguous [B, top_k, n_rows] tensor")
    _check(_lib.qmv_moe(fmt, W_experts.data_ptr(), expert_stride_bytes, n_experts, n_rows, n_cols,
                        expert_ids.data_ptr(), B, T, x.data_ptr(), st_tok, st_slot, y.data_ptr(),
                        _stream(stream)))
    return y


class GroupPlan:
    """Items sorted by group (qmv_group_plan): the device buffer and its sizes,
    and the HIP stream whose pool the buffer is from (None: not known)."""
    __slots__ = ("buffer", "n_items", "n_groups", "stream")

    def __init__(self, buffer, n_items, n_groups, stream=None):
        self.buffer, self.n_items, self.n_groups, self.stream = buffer, n_items, n_groups, stream


# The calls below run once a layer or a step for a few microseconds of GPU
# time, so their checks are kept short: one comparison of all that a tensor
# has to be, and the words for what is wrong only where it is.
_types = None        # torch dtype -> x_type; set whole at the first call, which any thread may make


def _type_of(t, name):
    """x_type of a float GPU tensor."""
    global _types
    if _types is None:
        _types = _x_types(_torch())
    xt = _types.get(getattr(t, "dtype", None))
    if xt is None or not t.is_cuda:
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        raise ValueError(f"{name} must be float32, float16 or bfloat16 (got {t.dtype})")
    return xt


def _full(t, name, dtype, shape):
    """Address of a contiguous GPU tensor of this type and shape."""
    if getattr(t, "dtype", None) is not dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        _dev(t, name, dtype)
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor")
    return t.data_ptr()


def _bytes_of(t, name, need):
    """Address of a contiguous uint8 GPU tensor of at least `need` bytes."""
    if getattr(t, "dtype", None) is not _torch().uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() < need:
        _dev(t, name, _torch().uint8)
        raise ValueError(f"{name} must be contiguous and hold {need} bytes")
    return t.data_ptr()


def _scratch(buf, name, need, like, stream, returned=False):
    """A caller's uint8 buffer of at least `need` bytes, or a new one."""
    if buf is None:
        return _new((need or 16,), _torch().uint8, like, stream, returned)
    _bytes_of(buf, name, need)
    return buf


def _on(stream, t):
    """The HIP stream of a call: stream's, or the current one of t's device."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


def qmv_group_plan(group_ids, n_groups, plan=None, stream=None):
    """Sorts the items of group_ids (int32, any shape, contiguous, on the GPU)
    by group and returns the GroupPlan that the grouped products take.  plan:
    a uint8 GPU tensor to build it in (its size: the library's
    qmv_group_plan_bytes), or None for a new one."""
    torch = _torch()
    ids = _full(group_ids, "group_ids", torch.int32, getattr(group_ids, "shape", None))
    n = group_ids.numel()
    buf = _scratch(plan, "plan", _lib.qmv_group_plan_bytes(n, n_groups), group_ids, stream, True)
    on = _on(stream, group_ids)
    _check(_lib.qmv_group_plan(ids, n, n_groups, buf.data_ptr(), buf.numel(), on))
    return GroupPlan(buf, n, n_groups, on if plan is None else None)


def _grouped(cfn, fmt, W, stride, E, rows, matrix_rows, cols, plan, top_k, x, out, name, dtype, stream):
    f = _fmt(fmt)
    w = _bytes_of(W, "W_experts", (E - 1) * stride + matrix_rows * row_bytes(f, cols))
    xt = _type_of(x, "x")
    if x.dim() == 2 and x.shape[1] == cols and x.stride(1) == 1:
        st_tok, st_slot = x.stride(0), 0
    elif x.dim() == 3 and x.shape[1] == top_k and x.shape[2] == cols and x.stride(2) == 1:
        st_tok, st_slot, _ = x.stride()
    else:
        raise ValueError("x must be [tokens, K] or [tokens, top_k, K] with K = n_cols and unit inner stride")
    T = x.shape[0]
    if not isinstance(plan, GroupPlan) or plan.n_items != T * top_k or plan.n_groups != E:
        raise ValueError(f"plan must be qmv_group_plan's of {T * top_k} items and {E} groups")
    if out is None:
        out = _new((T, top_k, rows), dtype or _torch().float32, x, stream)
        ot = _type_of(out, name)
    else:
        ot = _type_of(out, name)
        _full(out, name, out.dtype, (T, top_k, rows))
    on = _on(stream, x)
    if plan.stream != on:      # its memory goes back to another stream's pool: not while this one reads it
        plan.buffer.record_stream(_torch().cuda.current_stream(x.device) if stream is None else stream)
    _check(cfn(f, w, stride, E, rows, cols, plan.buffer.data_ptr(), T, top_k, x.data_ptr(), xt, st_tok, st_slot,
               out.data_ptr(), ot, on))
    return out


def qmv_moe_grouped(fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_cols, plan, top_k, x, y=None,
                    y_dtype=None, stream=None):
    """Expert products for any number of tokens, grouped by expert.

    plan: qmv_group_plan(expert_ids, n_experts) of the int32 [tokens, top_k]
    expert ids.  x: float32, float16 or bfloat16, [tokens, K] or [tokens,
    top_k, K].  Returns y [tokens, top_k, n_rows] of y_dtype (float32 by
    default)."""
    return _grouped(_lib.qmv_moe_grouped, fmt, W_experts, expert_stride_bytes, n_experts, n_rows, n_rows, n_cols, plan,
                    top_k, x, y, "y", y_dtype, stream)


def qmv_moe_grouped_swiglu(fmt, W_experts, expert_stride_bytes, n_experts, n_ff, n_cols, plan, top_k, x, h=None,
                           h_dtype=None, stream=None):
    """qmv_moe_grouped over experts of 2*n_ff rows (gate, then up): returns
    h [tokens, top_k, n_ff] = SiLU(gate x) * (up x) of h_dtype."""
    return _grouped(_lib.qmv_moe_grouped_swiglu, fmt, W_experts, expert_stride_bytes, n_experts, n_ff, 2 * n_ff,
                    n_cols, plan, top_k, x, h, "h", h_dtype, stream)


def qmv_moe_weighted_sum(y, weights, out=None, out_dtype=None, stream=None):
    """out [tokens, n_rows] = sum over the slots of weights[t, s] * y[t, s];
    y float32, float16 or bfloat16 [tokens, top_k, n_rows], weights float32
    [tokens, top_k]."""
    yt = _type_of(y, "y")
    torch = _torch()
    if y.dim() != 3 or not y.is_contiguous():
        raise ValueError("y must be a contiguous [tokens, top_k, n_rows] tensor")
    T, S, N = y.shape
    w = _full(weights, "weights", torch.float32, (T, S))
    if out is None:
        out = _new((T, N), out_dtype or torch.float32, y, stream)
        ot = _type_of(out, "out")
    else:
        ot = _type_of(out, "out")
        _full(out, "out", out.dtype, (T, N))
    _check(_lib.qmv_moe_weighted_sum(y.data_ptr(), yt, w, T, S, N, out.data_ptr(), ot, _on(stream, y)))
    return out


def qmv_lora(fmt, W, n_rows, n_cols, x, A, B, scales, adapter_ids, y=None, workspace=None, stream=None):
    """y[t] = DEQ(W) @ x[t] + scales[a] * B[a] @ (A[a] @ x[t]) with a =
    adapter_ids[t] (-1: the base alone).

    x: float32, float16 or bfloat16 [tokens, K]; A [adapters, rank, K] and B
    [adapters, n_rows, rank] of one of these types; scales float32
    [adapters]; adapter_ids int32 [tokens].  y is float32 [tokens, n_rows].
    workspace: a uint8 GPU tensor of the library's qmv_lora_workspace_bytes,
    or None for a new one."""
    xt, at = _type_of(x, "x"), _type_of(A, "A")
    torch = _torch()
    f = _fmt(fmt)
    w = _bytes_of(W, "W", n_rows * row_bytes(f, n_cols))
    if x.dim() != 2 or x.shape[1] != n_cols or x.stride(1) != 1:
        raise ValueError(f"x must be [tokens, K] with K={n_cols} and unit inner stride")
    T, ldx = x.shape[0], x.stride(0)
    if A.dim() != 3 or A.shape[2] != n_cols or not A.is_contiguous():
        raise ValueError("A must be a contiguous [adapters, rank, K] tensor")
    G, R, _ = A.shape
    b = _full(B, "B", A.dtype, (G, n_rows, R))
    s = _full(scales, "scales", torch.float32, (G,))
    ids = _full(adapter_ids, "adapter_ids", torch.int32, (T,))
    if y is None:
        y = _new((T, n_rows), torch.float32, x, stream)
        ldy = n_rows
    else:
        _dev(y, "y", torch.float32)
        y2, Ty, ldy = _rows2d(y, "y", n_rows)
        if Ty != T:
            raise ValueError("y must have as many rows as x")
    ws = _scratch(workspace, "workspace", _lib.qmv_lora_workspace_bytes(T, R, G), x, stream)
    _check(_lib.qmv_lora(f, w, n_rows, n_cols, x.data_ptr(), xt, ldx if T > 1 else n_cols, T, A.data_ptr(), b, at, G, R, s,
                         ids, y.data_ptr(), ldy, ws.data_ptr(), ws.numel(), _on(stream, x)))
    return y


def qmv_spec_verify(logits, draft_probs, draft_tokens, n_draft, u_accept, u_last, tokens=None, n_kept=None,
                    workspace=None, stream=None):
    """Keeps drafted tokens while u q(x) < p(x), p the softmax of the target's
    logits, and draws one more token (see qmv.h).

    logits: float32, float16 or bfloat16 [requests, drafts + 1, vocab];
    draft_probs: float32 [requests, drafts, vocab], or None (each draft's
    probability all on its token); draft_tokens int32 [requests, drafts];
    n_draft int32 [requests]; u_accept float32 [requests, drafts]; u_last
    float32 [requests].  Returns (tokens int32 [requests, drafts + 1],
    n_kept int32 [requests])."""
    lt = _type_of(logits, "logits")
    torch = _torch()
    if logits.dim() != 3 or logits.stride(2) != 1:
        raise ValueError("logits must be [requests, drafts + 1, vocab] with unit inner stride")
    Q, D1, V = logits.shape
    D = D1 - 1
    lr, ll, _ = logits.stride()
    i32, f32 = torch.int32, torch.float32
    qp, qr, ql = None, 0, 0
    if draft_probs is not None:
        _dev(draft_probs, "draft_probs", f32)
        if draft_probs.shape != (Q, D, V) or draft_probs.stride(2) != 1:
            raise ValueError("draft_probs must be [requests, drafts, vocab] with unit inner stride")
        qp, (qr, ql, _) = draft_probs.data_ptr(), draft_probs.stride()
    x, n = _full(draft_tokens, "draft_tokens", i32, (Q, D)), _full(n_draft, "n_draft", i32, (Q,))
    u, ul = _full(u_accept, "u_accept", f32, (Q, D)), _full(u_last, "u_last", f32, (Q,))
    if tokens is None:
        tokens = _new((Q, D1), i32, logits, stream)
    else:
        _full(tokens, "tokens", i32, (Q, D1))
    if n_kept is None:
        n_kept = _new((Q,), i32, logits, stream)
    else:
        _full(n_kept, "n_kept", i32, (Q,))
    ws = _scratch(workspace, "workspace", _lib.qmv_spec_verify_workspace_bytes(Q, D, V), logits, stream)
    _check(_lib.qmv_spec_verify(logits.data_ptr(), lt, lr, ll, qp, qr, ql, x, n, u, ul, Q, D, V, tokens.data_ptr(),
                                n_kept.data_ptr(), ws.data_ptr(), ws.numel(), _on(stream, logits)))
    return tokens, n_kept


def qmv_dequant(fmt, W, n_rows, n_cols, out=None, stream=None):
    """fp32 [n_rows, n_cols] values of the stored blocks."""
    torch = _torch()
    fmt = _fmt(fmt)
    _dev(W, "W", torch.uint8)
    if out is None:
        out = _new((n_rows, n_cols), torch.float32, W, stream)
    _dev(out, "out", torch.float32)
    if out.shape != (n_rows, n_cols) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [n_rows, n_cols] tensor")
    _check(_lib.qmv_dequant(fmt, W.data_ptr(), n_rows, n_cols, out.data_ptr(), _stream(stream)))
    return out


def qmv_stream_read(buf, out, stream=None):
    """Reads the uint8 GPU tensor buf once (16-byte non-temporal loads); each
    launched thread writes the XOR of the words it read into out (uint32,
    >= 256 words).  A measurement aid: the device's stream-read ceiling."""
    torch = _torch()
    _dev(buf, "buf", torch.uint8)
    _dev(out, "out", torch.int32)
    if not buf.is_contiguous() or not out.is_contiguous():
        raise ValueError("buf and out must be contiguous")
    _check(_lib.qmv_stream_read(buf.data_ptr(), buf.numel(), out.data_ptr(), out.numel(), _stream(stream)))
    return out


def chain_stages(stages, fmt=None):
    """[(W, n_rows, n_cols, x, y, wait), ...] of GPU tensors -> ctypes array.
    With fmt, each W is checked to hold its n_rows x n_cols blocks."""
    torch = _torch()
    arr = (ChainStage * len(stages))()
    for i, (W, n_rows, n_cols, x, y, wait) in enumerate(stages):
        _dev(W, "W", torch.uint8)
        rb = row_bytes(_fmt(fmt), n_cols) if fmt is not None else 0   # unknown fmt: the library rejects it
        if rb:
            need = n_rows * rb
            if W.numel() < need or not W.is_contiguous():
                raise ValueError(f"stage {i}: W must be contiguous and hold {need} bytes")
        _dev(x, "x", torch.float32)
        _dev(y, "y", torch.float32)
        if x.numel() < n_cols or y.numel() < n_rows or not x.is_contiguous() or not y.is_contiguous():
            raise ValueError(f"stage {i}: x must hold n_cols and y n_rows contiguous floats")
        arr[i] = ChainStage(W.data_ptr(), x.data_ptr(), y.data_ptr(), n_rows, n_cols, 1 if wait else 0, 0)
    return arr


def qmv_chain(fmt, stages, workspace, stream=None):
    """Runs batch-1 matvec stages in one call (see qmv.h): one persistent
    launch for the 32-weight formats, stage groups as launches of their own
    for Q4_K and Q6_K.

    stages: list of (W, n_rows, n_cols, x, y, wait) with GPU tensors, or a
    ctypes array from chain_stages().  workspace: uint8 GPU tensor of at
    least CHAIN_WORKSPACE_BYTES, zero-filled before its first use."""
    torch = _torch()
    _dev(workspace, "workspace", torch.uint8)
    arr = stages if isinstance(stages, ctypes.Array) else chain_stages(stages, fmt)
    _check(_lib.qmv_chain(_fmt(fmt), ctypes.cast(arr, ctypes.c_void_p), len(arr), workspace.data_ptr(),
                          workspace.numel(), _stream(stream)))


def qmv_chain_noalloc(fmt, stages, stream=None):
    """qmv_chain with the barrier words held by the library (no workspace
    argument, nothing allocated; see qmv.h).  stages as for qmv_chain."""
    arr = stages if isinstance(stages, ctypes.Array) else chain_stages(stages, fmt)
    _check(_lib.qmv_chain_noalloc(_fmt(fmt), ctypes.cast(arr, ctypes.c_void_p), len(arr), _stream(stream)))


from . import serving  # noqa: E402
from .serving import (KVCache, Logprobs, cache_page_bytes, qmv_cache_attention, qmv_cache_read, qmv_cache_write,  # noqa: E402
                      qmv_logprobs)

serving.bind(_lib)
