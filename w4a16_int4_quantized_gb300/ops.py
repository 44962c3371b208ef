"""Thin Python binding over the C ABI of libw4gb300 (include/w4.h).

Argument marshalling only: every function passes torch tensors' device
pointers, sizes and the current CUDA stream to the ``w4_*`` entry point of
the same name, and raises ``W4Error`` on a non-OK status.  All arithmetic
runs in the library's CUDA kernels; if the library is missing this module
raises on import of the first call -- there is no CPU fallback.

A call runs on the current stream, or on the one given as ``stream``.  The
outputs and the workspace that it allocates belong to that stream's memory, as
if the call stood in ``with torch.cuda.stream(stream)``: what other streams
still do with memory that was freed there cannot reach them, and a tensor that
is used on another stream too is for the caller to order (an event, or
``record_stream``).  Inputs, and outputs or workspaces that the caller brings,
have to be ready on that stream.

``raw`` is the ctypes handle itself, for callers (and tests) that want to
drive the C functions with plain pointers.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4gb300.so")

W4_OK, W4_EINVAL, W4_ESHAPE, W4_ECUDA = 0, 1, 2, 3
LAYOUT_ROWMAJOR, LAYOUT_N64, LAYOUT_B32 = 0, 1, 2
FLAG_PDL = 1
OP_LINEAR_Q4, OP_LINEAR_Q8, OP_LINEAR_W4A16, OP_LINEAR_Q4_GROUP, OP_LINEAR_W8A16 = 0, 1, 2, 3, 4
CHAIN_MAX_LINEARS, CHAIN_MAX_K = 64, 8192


class ChainLinear(C.Structure):
    """w4_chain_linear of include/w4.h."""
    _fields_ = [("w", C.c_void_p), ("sw", C.c_void_p), ("y", C.c_void_p),
                ("N", C.c_int32), ("K", C.c_int32), ("input", C.c_int32), ("reserved", C.c_int32)]


F32, BF16, F16 = 0, 1, 2
MAX_DRAFT = 128
_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


class PagedCache(C.Structure):
    """w4_paged_cache of include/w4.h."""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("pages", C.c_int64), ("page_size", C.c_int32),
                ("heads", C.c_int32), ("head_dim", C.c_int32), ("type", C.c_int32), ("page_stride", C.c_int64),
                ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


# (name, restype, argtypes) of every exported symbol, in header order.
_vp, _i64, _i32, _u32, _sz, _f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_uint32, C.c_size_t, C.c_float
SIGNATURES = [
    ("w4_quantize_row_q8", _i32, [_vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    ("w4_quantize_matrix_q4", _i32, [_vp, _i64, _i64, _vp, _vp, _vp]),
    ("w4_quantize_matrix_q8", _i32, [_vp, _i64, _i64, _vp, _vp, _vp]),
    ("w4_dot_i32_q4", _i32, [_vp, _vp, _i64, _vp, _vp]),
    ("w4_linear_q4", _i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _sz, _u32, _vp]),
    ("w4_linear_q4_f32", _i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _sz, _u32, _vp]),
    ("w4_linear_q8", _i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    ("w4_linear_w4a16_group", _i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _u32, _vp]),
    ("w4_linear_q4_noalloc", _i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]),
    ("w4_linear_w8a16", _i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    ("w4_linear_q4_group", _i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _u32, _vp]),
    ("w4_chain_q4", _i32, [_vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, _vp]),
    ("w4_chain_q4_test_timeout", _i32, [_vp, _i32, _vp, _i32, _i32, _i32, _vp, _sz, C.c_uint64, _i32, _vp]),
    ("w4_chain_workspace_bytes", _sz, [_vp, _i32, _i32]),
    ("w4_quantize_mxfp4", _i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp]),
    ("w4_dequantize_mxfp4", _i32, [_vp, _vp, _i64, _i64, _vp, _i32, _vp]),
    ("w4_linear_mxfp4", _i32, [_vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _u32, _vp]),
    ("w4_linear_mxfp4_a4", _i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _u32, _vp]),
    ("w4_draft_plan", _i32, [_vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    ("w4_qk_norm_rope", _i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _f32, _vp, _vp, _i64, _i32, _i32, _vp, _vp,
                               _vp, _vp]),
    ("w4_tree_attention", _i32, [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _f32, _i64, _i32, _vp,
                                 _vp, _sz, _vp]),
    ("w4_tree_attention_workspace_bytes", _sz, [_i64, _i32, _i32, _i32, _i64, _i32]),
    ("w4_pack_interleaved_n64", _i32, [_vp, _vp, _i64, _i64, _vp]),
    ("w4_pack_block32", _i32, [_vp, _vp, _vp, _i64, _i64, _vp]),
    ("w4_workspace_bytes", _sz, [_i32, _i64, _i64, _i64, _i64]),
    ("w4_device_status", _i32, [_vp, _i32]),
    ("w4_last_cuda_error", _i32, []),
    ("w4_status_string", C.c_char_p, [_i32]),
    ("w4_probe_mma_peak", _i32, [_i32, _vp, _i64, _vp, _vp]),
    ("w4_version", _i32, []),
]


class W4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = raw.w4_status_string(status).decode() if raw is not None else str(status)
        if status == W4_ECUDA and raw is not None:
            msg += f" (cudaError {raw.w4_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


def load(path: str = LIB_PATH) -> C.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"libw4gb300 not built ({path}); run __graft_entry__.build() or "
                           "python -m w4a16_int4_quantized_gb300.build")
    lib = C.CDLL(path)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


raw = load()


def _check(status: int, what: str) -> None:
    if status != W4_OK:
        raise W4Error(status, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr() or None


def _stream(stream=None) -> int | None:
    if stream is None:
        # the handle of torch.cuda.current_stream(), without the 3 us that making a Stream object takes
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    return stream.cuda_stream or None


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory that the call's stream may write at once (torch orders a block with its own stream only)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# ---------------------------------------------------------------- quantizers

def quantize_row_q8(x: torch.Tensor, stream=None):
    """x f32 [M, K] (cuda) -> (q int8 [M, K], sx f32 [M], rowsum int32 [M])."""
    assert x.dtype == torch.float32 and x.is_contiguous() and x.dim() == 2
    M, K = x.shape
    q = _empty((M, K), torch.int8, x.device, stream)
    sx = _empty(M, torch.float32, x.device, stream)
    rs = _empty(M, torch.int32, x.device, stream)
    _check(raw.w4_quantize_row_q8(_ptr(x), M, K, _ptr(q), _ptr(sx), _ptr(rs), _stream(stream)),
           "w4_quantize_row_q8")
    return q, sx, rs


def quantize_matrix_q4(W: torch.Tensor, stream=None):
    """W f32 [N, K] -> (packed uint8 [N, ceil(K/2)], sw f32 [N])."""
    assert W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    packed = _empty((N, (K + 1) // 2), torch.uint8, W.device, stream)
    sw = _empty(N, torch.float32, W.device, stream)
    _check(raw.w4_quantize_matrix_q4(_ptr(W), N, K, _ptr(packed), _ptr(sw), _stream(stream)),
           "w4_quantize_matrix_q4")
    return packed, sw


def quantize_matrix_q8(W: torch.Tensor, stream=None):
    """W f32 [N, K] -> (q int8 [N, K], sw f32 [N])."""
    assert W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    q = _empty((N, K), torch.int8, W.device, stream)
    sw = _empty(N, torch.float32, W.device, stream)
    _check(raw.w4_quantize_matrix_q8(_ptr(W), N, K, _ptr(q), _ptr(sw), _stream(stream)), "w4_quantize_matrix_q8")
    return q, sw


# ---------------------------------------------------------------- dot / linears

def dot_i32_q4(xq: torch.Tensor, wrow: torch.Tensor, K: int | None = None, stream=None) -> torch.Tensor:
    """Exact biased-Q4 dot of one row -> int32 device scalar."""
    K = xq.numel() if K is None else K
    out = _empty(1, torch.int32, xq.device, stream)
    _check(raw.w4_dot_i32_q4(_ptr(xq), _ptr(wrow), K, _ptr(out), _stream(stream)), "w4_dot_i32_q4")
    return out


def _workspace(op, M, N, K, G, workspace, device, stream):
    need = raw.w4_workspace_bytes(op, M, N, K, G)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = _empty(need, torch.uint8, device, stream)
    return workspace, workspace.numel()


def linear_q4(xq, sx, w, sw, K: int | None = None, N: int | None = None, layout: int = LAYOUT_ROWMAJOR,
              flags: int = 0, out=None, workspace=None, stream=None) -> torch.Tensor:
    """W4A8: y[M, N] = (f32(sum xq * (u - 8)) * sx[m]) * sw[n]."""
    M = xq.shape[0]
    K = xq.shape[1] if K is None else K
    N = sw.numel() if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, xq.device, stream)
    ws, wsb = _workspace(OP_LINEAR_Q4, M, N, K, 0, workspace, xq.device, stream)
    _check(raw.w4_linear_q4(_ptr(xq), _ptr(sx), _ptr(w), _ptr(sw), _ptr(y), M, N, K, layout,
                            _ptr(ws), wsb, flags, _stream(stream)), "w4_linear_q4")
    return y


def linear_q4_f32(x, w, sw, K: int | None = None, N: int | None = None, layout: int = LAYOUT_ROWMAJOR,
                  flags: int = 0, out=None, xq=None, sx=None, workspace=None, stream=None):
    """quantize_row_q8(x) then linear_q4 in one call -> (y [M, N], xq [M, K], sx [M])."""
    assert x.dtype == torch.float32 and x.dim() == 2
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    N = sw.numel() if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, x.device, stream)
    xq = xq if xq is not None else _empty((M, K), torch.int8, x.device, stream)
    sx = sx if sx is not None else _empty(M, torch.float32, x.device, stream)
    ws, wsb = _workspace(OP_LINEAR_Q4, M, N, K, 0, workspace, x.device, stream)
    _check(raw.w4_linear_q4_f32(_ptr(x), _ptr(w), _ptr(sw), _ptr(y), _ptr(xq), _ptr(sx), M, N, K, layout,
                                _ptr(ws), wsb, flags, _stream(stream)), "w4_linear_q4_f32")
    return y, xq, sx


NOALLOC_SCRATCH_BYTES = 8 << 20


def linear_q4_noalloc(xq, sx, w, sw, K: int | None = None, N: int | None = None, layout: int = LAYOUT_ROWMAJOR,
                      out=None, stream=None) -> torch.Tensor:
    """linear_q4 for callers that may not allocate device scratch: large
    batches use the library's fixed NOALLOC_SCRATCH_BYTES array instead (calls
    on one device share it, so keep them on one stream).  `out` must be given
    by callers that may not allocate at all."""
    M = xq.shape[0]
    K = xq.shape[1] if K is None else K
    N = sw.numel() if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, xq.device, stream)
    st = raw.w4_linear_q4_noalloc(_ptr(xq), _ptr(sx), _ptr(w), _ptr(sw), _ptr(y), M, N, K, layout, _stream(stream))
    if st == W4_ESHAPE and raw.w4_workspace_bytes(OP_LINEAR_Q4, M, N, K, 0) > NOALLOC_SCRATCH_BYTES:
        raise W4Error(st, f"w4_linear_q4_noalloc: batch needs {raw.w4_workspace_bytes(OP_LINEAR_Q4, M, N, K, 0)} "
                          f"bytes of scratch, above the fixed {NOALLOC_SCRATCH_BYTES}")
    _check(st, "w4_linear_q4_noalloc")
    return y


def linear_q8(xq, sx, w, sw, flags: int = 0, out=None, workspace=None, stream=None) -> torch.Tensor:
    """W8A8: y[M, N] = (f32(sum xq * w) * sx[m]) * sw[n]."""
    M, K = xq.shape
    N = w.shape[0]
    y = out if out is not None else _empty((M, N), torch.float32, xq.device, stream)
    ws, wsb = _workspace(OP_LINEAR_Q8, M, N, K, 0, workspace, xq.device, stream)
    _check(raw.w4_linear_q8(_ptr(xq), _ptr(sx), _ptr(w), _ptr(sw), _ptr(y), M, N, K,
                            _ptr(ws), wsb, flags, _stream(stream)), "w4_linear_q8")
    return y


def linear_w4a16_group(x, w, scales, G: int, K: int | None = None, N: int | None = None,
                       layout: int = LAYOUT_ROWMAJOR, flags: int = 0, out=None, workspace=None,
                       stream=None) -> torch.Tensor:
    """Group-wise W4A16: y = sum_g s[n, g] * sum_{k in g} x[m, k] * q[n, k].

    x: bf16 [M, K] (torch.bfloat16, or int16/uint16 bit patterns);
    w: packed signed nibbles; scales: f16 [N, Kp/G] (torch.float16 or 16-bit patterns).
    """
    assert x.element_size() == 2 and scales.element_size() == 2
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    N = scales.shape[0] if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, x.device, stream)
    ws, wsb = _workspace(OP_LINEAR_W4A16, M, N, K, G, workspace, x.device, stream)
    _check(raw.w4_linear_w4a16_group(_ptr(x), _ptr(w), _ptr(scales), _ptr(y), M, N, K, G, layout,
                                     _ptr(ws), wsb, flags, _stream(stream)), "w4_linear_w4a16_group")
    return y


def linear_w8a16(x, w, sw, flags: int = 0, out=None, workspace=None, stream=None) -> torch.Tensor:
    """W8A16: y[M, N] = sw[n] * sum_k x[m, k] * q[n, k], x f32, q int8."""
    M, K = x.shape
    N = sw.numel()
    y = out if out is not None else _empty((M, N), torch.float32, x.device, stream)
    ws, wsb = _workspace(OP_LINEAR_W8A16, M, N, K, 0, workspace, x.device, stream)
    _check(raw.w4_linear_w8a16(_ptr(x), _ptr(w), _ptr(sw), _ptr(y), M, N, K, _ptr(ws), wsb, flags, _stream(stream)),
           "w4_linear_w8a16")
    return y


def linear_q4_group(xq, sx, w, scales, zeros, G: int, K: int | None = None, N: int | None = None,
                    layout: int = LAYOUT_ROWMAJOR, flags: int = 0, out=None, workspace=None,
                    stream=None) -> torch.Tensor:
    """Grouped asymmetric W4A8: y = sx[m] * sum_g (sum_{k in g} xq * (u - z[n, g])) * s[n, g]."""
    M = xq.shape[0]
    K = xq.shape[1] if K is None else K
    N = scales.shape[0] if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, xq.device, stream)
    ws, wsb = _workspace(OP_LINEAR_Q4_GROUP, M, N, K, G, workspace, xq.device, stream)
    _check(raw.w4_linear_q4_group(_ptr(xq), _ptr(sx), _ptr(w), _ptr(scales), _ptr(zeros), _ptr(y), M, N, K, G,
                                  layout, _ptr(ws), wsb, flags, _stream(stream)), "w4_linear_q4_group")
    return y


def chain_descriptors(linears):
    """ctypes array of w4_chain_linear for (w, sw, y, input) tuples."""
    arr = (ChainLinear * len(linears))()
    for i, (w, sw, y, inp) in enumerate(linears):
        arr[i] = ChainLinear(_ptr(w), _ptr(sw), _ptr(y), sw.numel(), 2 * w.shape[-1], inp, 0)
    return arr


def chain_workspace_bytes(linears, K0: int) -> int:
    return raw.w4_chain_workspace_bytes(chain_descriptors(linears), len(linears), K0)


def chain_q4(x0, linears, passes: int, pass_output: int, workspace=None, stream=None):
    """Runs a chain of M = 1 W4A8 linears as one kernel.  linears: sequence of
    (w, sw, y, input) with w packed [N][K/2] uint8, sw [N] f32, y [N] f32
    (written), input = -1 for the pass input or the index of an earlier
    linear.  Returns the y tensors."""
    arr = chain_descriptors(linears)
    need = raw.w4_chain_workspace_bytes(arr, len(linears), x0.numel())
    if workspace is None:
        workspace = _empty(need, torch.uint8, x0.device, stream)
    _check(raw.w4_chain_q4(_ptr(x0), x0.numel(), arr, len(linears), passes, pass_output, _ptr(workspace),
                           workspace.numel(), _stream(stream)), "w4_chain_q4")
    return [y for _, _, y, _ in linears]


def chain_q4_test_timeout(x0, linears, passes: int, pass_output: int, wait_limit_ns: int, hold_stage: int,
                          workspace=None, stream=None) -> int:
    """w4_chain_q4_test_timeout: the chain with a short wait limit and,
    hold_stage >= 0, one stage whose outputs are never published.  Returns
    the call's status (the device status word reports the timeout)."""
    arr = chain_descriptors(linears)
    need = raw.w4_chain_workspace_bytes(arr, len(linears), x0.numel())
    if workspace is None:
        workspace = _empty(need, torch.uint8, x0.device, stream)
    return raw.w4_chain_q4_test_timeout(_ptr(x0), x0.numel(), arr, len(linears), passes, pass_output,
                                        _ptr(workspace), workspace.numel(), int(wait_limit_ns), int(hold_stage),
                                        _stream(stream))


# ---------------------------------------------------------------- microscaled 4-bit floating point

def quantize_mxfp4(x: torch.Tensor, stream=None):
    """x f32, bf16 or f16 [R, K] -> (codes uint8 [R, nb * 16], scales uint8 [R, nb]), nb = ceil(K / 32)."""
    R, K = x.shape
    assert x.is_contiguous()
    nb = (K + 31) // 32
    dev = x.device
    codes = _empty((R, nb * 16), torch.uint8, dev, stream)
    scales = _empty((R, nb), torch.uint8, dev, stream)
    st = raw.w4_quantize_mxfp4(x.data_ptr(), _TYPES[x.dtype], R, K, codes.data_ptr(), scales.data_ptr(), _stream(stream))
    if st:
        raise W4Error(st, "w4_quantize_mxfp4")
    return codes, scales


def _mxfp4_rows(codes, scales, K, what):
    """Rows of an MXFP4 matrix of K columns; its planes have to be whole."""
    R, nb = scales.shape
    if (K + 31) >> 5 != nb or codes.numel() != R * nb * 16 or not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{what}: codes [R, nb * 16] and scales [R, nb], dense, with nb = ceil(K / 32)")
    return R


def _given(out, shape, what):
    """An output that the caller brought: of the call's shape, dense."""
    if out.shape != shape or not out.is_contiguous():
        raise ValueError(f"{what}: out has to be {tuple(shape)}, dense")
    return out


def dequantize_mxfp4(codes, scales, K: int, dtype=torch.float32, out=None, stream=None) -> torch.Tensor:
    """The values that codes and scales stand for, [R, K]."""
    R = _mxfp4_rows(codes, scales, K, "dequantize_mxfp4")
    y = _empty((R, K), dtype, codes.device, stream) if out is None else _given(out, (R, K), "dequantize_mxfp4")
    st = raw.w4_dequantize_mxfp4(codes.data_ptr(), scales.data_ptr(), R, K, y.data_ptr(), _TYPES[y.dtype],
                                 _stream(stream))
    if st:
        raise W4Error(st, "w4_dequantize_mxfp4")
    return y


def linear_mxfp4(x, w, sw, out_dtype=torch.float32, flags: int = 0, out=None, stream=None) -> torch.Tensor:
    """y[M, N] = x W^T: x bf16 [M, K], W the MXFP4 matrix (codes w, scales sw)."""
    M, K = x.shape
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    N = _mxfp4_rows(w, sw, K, "linear_mxfp4")
    y = _empty((M, N), out_dtype, x.device, stream) if out is None else _given(out, (M, N), "linear_mxfp4")
    st = raw.w4_linear_mxfp4(x.data_ptr(), w.data_ptr(), sw.data_ptr(), y.data_ptr(), _TYPES[y.dtype], M, N, K, flags,
                             _stream(stream))
    if st:
        raise W4Error(st, "w4_linear_mxfp4")
    return y


def linear_mxfp4_a4(xq, sx, w, sw, K: int, out_dtype=torch.float32, flags: int = 0, out=None,
                    stream=None) -> torch.Tensor:
    """y[M, N] = X W^T, both MXFP4 matrices (codes and scales of quantize_mxfp4) of K columns."""
    M = _mxfp4_rows(xq, sx, K, "linear_mxfp4_a4")
    N = _mxfp4_rows(w, sw, K, "linear_mxfp4_a4")
    y = _empty((M, N), out_dtype, xq.device, stream) if out is None else _given(out, (M, N), "linear_mxfp4_a4")
    st = raw.w4_linear_mxfp4_a4(xq.data_ptr(), sx.data_ptr(), w.data_ptr(), sw.data_ptr(), y.data_ptr(), _TYPES[y.dtype],
                                M, N, K, flags, _stream(stream))
    if st:
        raise W4Error(st, "w4_linear_mxfp4_a4")
    return y


# ---------------------------------------------------------------- drafted tokens over a paged cache

def draft_plan(ctx_len, new_len, parents, free_pages, block_table, page_size: int, max_tokens: int | None = None,
               stream=None):
    """Plan of a step of drafted tokens (w4_draft_plan): all tensors int32 on the GPU.

    ctx_len, new_len [B]; parents [max_tokens] or None (every token follows the
    one before it; max_tokens must then be given); free_pages [n]; block_table
    [B, width], extended in place.  Returns (cu_new int32 [B + 1], slots int64
    [max_tokens], positions int32 [max_tokens], mask int32 [max_tokens, 4] (bit
    patterns), taken int32 [1])."""
    i32 = torch.int32
    B, width = block_table.shape
    n = parents.numel() if max_tokens is None else max_tokens
    assert ctx_len.dtype is new_len.dtype is free_pages.dtype is block_table.dtype is i32
    assert ctx_len.numel() == new_len.numel() == B and ctx_len.is_contiguous() and new_len.is_contiguous()
    assert free_pages.is_contiguous() and block_table.is_contiguous()
    assert parents is None or (parents.dtype is i32 and parents.is_contiguous() and parents.numel() >= n)
    dev = ctx_len.device
    cu = _empty(B + 1, i32, dev, stream)
    slots = _empty(n, torch.int64, dev, stream)
    positions = _empty(n, i32, dev, stream)
    mask = _empty((n, 4), i32, dev, stream)
    taken = _empty(1, i32, dev, stream)
    st = raw.w4_draft_plan(ctx_len.data_ptr(), new_len.data_ptr(), None if parents is None else parents.data_ptr(),
                           free_pages.data_ptr(), free_pages.numel(), block_table.data_ptr(), B, width, page_size, n,
                           cu.data_ptr(), slots.data_ptr(), positions.data_ptr(), mask.data_ptr(), taken.data_ptr(),
                           _stream(stream))
    if st:
        raise W4Error(st, "w4_draft_plan")
    return cu, slots, positions, mask, taken


_CACHE_STRUCT = struct.Struct("PPqiiiiqqq")  # w4_paged_cache


def _cache_fields(k, v):
    """The fields of w4_paged_cache for two caches seen as [page, token, head, value]."""
    P, page, H, D = shape = k.shape
    sp, st, sh, sd = strides = k.stride()
    if shape != v.shape or strides != v.stride() or k.dtype != v.dtype or sd != 1:
        raise ValueError("k and v caches: [page, token, head, value] of one shape, type and strides, values dense")
    # the stride of an axis of one place is free; make it one that every layout rule allows
    if H == 1:
        sh = D
    if page == 1:
        st = H * D
    if P == 1:
        sp = page * H * D
    return k.data_ptr(), v.data_ptr(), P, page, H, D, _TYPES[k.dtype], sp, st, sh


def paged_cache(k: torch.Tensor, v: torch.Tensor) -> PagedCache:
    """The w4_paged_cache of two caches seen as [page, token, head, value] (any strides, values dense)."""
    if k.dim() != 4:
        raise ValueError("k and v caches: [page, token, head, value]")
    return PagedCache(*_cache_fields(k, v))


def qk_norm_rope(qkv, q_heads: int, wq, wk, positions, cos_sin, slots, k_cache, v_cache, eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None) -> torch.Tensor:
    """Head norms, rotation and cache store (w4_qk_norm_rope) -> q [T, q_heads, D] of the cache's type.

    qkv [T, >= (q_heads + 2 kv_heads) * D], rows of any stride; wq, wk f32 [D]
    or None; positions int32 [T]; cos_sin f32 [max_pos, rot] or None; slots
    int64 [T]; k_cache, v_cache [page, token, head, D]."""
    c = _cache_fields(k_cache, v_cache)
    D = c[5]
    T, cols = qkv.shape
    ld, one = qkv.stride()
    assert one == 1 and cols >= (q_heads + 2 * c[4]) * D
    assert positions.dtype == torch.int32 and positions.is_contiguous() and positions.numel() >= T
    assert slots.dtype == torch.int64 and slots.is_contiguous() and slots.numel() >= T
    f32 = torch.float32
    assert wq is None or (wq.dtype == f32 and wq.shape == (D,) and wq.is_contiguous())
    assert wk is None or (wk.dtype == f32 and wk.shape == (D,) and wk.is_contiguous())
    max_pos, rot = (1 << 31, 0) if cos_sin is None else cos_sin.shape
    assert cos_sin is None or (cos_sin.dtype == f32 and cos_sin.is_contiguous())
    dt = k_cache.dtype
    q = _empty((T, q_heads, D), dt, qkv.device, stream) if out is None else _given(out, (T, q_heads, D), "qk_norm_rope")
    assert q.dtype is dt
    st = raw.w4_qk_norm_rope(qkv.data_ptr(), _TYPES[qkv.dtype], ld if T > 1 else cols, T, q_heads,
                             None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(), eps,
                             positions.data_ptr(), None if cos_sin is None else cos_sin.data_ptr(), max_pos, rot,
                             interleaved, slots.data_ptr(), _CACHE_STRUCT.pack(*c), q.data_ptr(), _stream(stream))
    if st:
        raise W4Error(st, "w4_qk_norm_rope")
    return q


def tree_attention_workspace_bytes(B: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int,
                                   max_new: int) -> int:
    return int(raw.w4_tree_attention_workspace_bytes(B, q_heads, kv_heads, head_dim, max_len, max_new))


def tree_attention(q, k_cache, v_cache, block_table, ctx_len, cu_new, mask, scale: float, max_len: int, max_new: int,
                   out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of drafted tokens over a paged cache (w4_tree_attention) -> [T, q_heads, D].

    q [T, q_heads, D] of the cache's type, tokens of any stride; k_cache,
    v_cache [page, token, head, D]; block_table int32 [B, width]; ctx_len,
    cu_new, mask from the step's plan; max_len, max_new: bounds of ctx_len +
    new_len and of new_len."""
    c = _cache_fields(k_cache, v_cache)
    T, Hq, D = q.shape
    ld, sh, one = q.stride()
    B, width = block_table.shape
    i32, dt, dev = torch.int32, q.dtype, q.device
    assert dt == k_cache.dtype and D == c[5] and one == 1 and (Hq == 1 or sh == D)
    assert block_table.dtype == ctx_len.dtype == cu_new.dtype == i32 and mask.element_size() == 4
    assert block_table.is_contiguous() and ctx_len.is_contiguous() and cu_new.is_contiguous() and mask.is_contiguous()
    assert ctx_len.numel() >= B and cu_new.numel() > B and mask.numel() >= 4 * T
    o = _empty((T, Hq, D), dt, dev, stream) if out is None else _given(out, (T, Hq, D), "tree_attention")
    assert o.dtype is dt
    ws, have = 0, 0
    if workspace is not None:
        ws, have = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        need = raw.w4_tree_attention_workspace_bytes(B, Hq, c[4], D, max_len, max_new)
        if 0 < need < 1 << 62:  # more: sizes that the call refuses
            workspace = _empty(need, torch.uint8, dev, stream)
            ws, have = workspace.data_ptr(), need
    st = raw.w4_tree_attention(q.data_ptr(), ld if T > 1 else Hq * D, _CACHE_STRUCT.pack(*c), block_table.data_ptr(),
                               width, ctx_len.data_ptr(), cu_new.data_ptr(), mask.data_ptr(), B, T, Hq, scale, max_len,
                               max_new, o.data_ptr(), ws, have, _stream(stream))
    if st:
        raise W4Error(st, "w4_tree_attention")
    return o


def pack_interleaved_n64(w: torch.Tensor, K: int, stream=None) -> torch.Tensor:
    """Row-major packed int4 [N, ceil(K/2)] -> interleaved [N/64, K, 32]."""
    N = w.shape[0]
    il = _empty((N // 64, K, 32), torch.uint8, w.device, stream)
    _check(raw.w4_pack_interleaved_n64(_ptr(w), _ptr(il), N, K, _stream(stream)), "w4_pack_interleaved_n64")
    return il


def linear_w4a16_b32(x, blocks, K: int | None = None, N: int | None = None, flags: int = 0, out=None,
                     stream=None) -> torch.Tensor:
    """Group-wise W4A16 (G = 32) reading inline-scale blocks [N][Kp/32 * 18]."""
    assert x.element_size() == 2
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    N = blocks.shape[0] if N is None else N
    y = out if out is not None else _empty((M, N), torch.float32, x.device, stream)
    _check(raw.w4_linear_w4a16_group(_ptr(x), _ptr(blocks), None, _ptr(y), M, N, K, 32, LAYOUT_B32, None, 0, flags,
                                     _stream(stream)), "w4_linear_w4a16_group")
    return y


def pack_block32(w: torch.Tensor, scales: torch.Tensor, K: int, stream=None) -> torch.Tensor:
    """W4A16 planes (packed [N][Kp/2], f16 scales [N][Kp/32]) -> inline-scale blocks [N][Kp/32 * 18]."""
    N = w.shape[0]
    nb = (K + (K & 1)) // 32
    out = _empty((N, nb * 18), torch.uint8, w.device, stream)
    _check(raw.w4_pack_block32(_ptr(w), _ptr(scales), _ptr(out), N, K, _stream(stream)), "w4_pack_block32")
    return out


def workspace_bytes(op: int, M: int, N: int, K: int, G: int = 0) -> int:
    return int(raw.w4_workspace_bytes(op, M, N, K, G))


def device_status(clear: bool = False) -> int:
    v = C.c_uint32(0)
    _check(raw.w4_device_status(C.byref(v), 1 if clear else 0), "w4_device_status")
    return int(v.value)


def probe_mma_peak(kind: int) -> float:
    """Measured legacy mma.sync throughput in tera-ops/s (0: s8 m16n8k32, 1: bf16 m16n8k16)."""
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    scratch = torch.empty(4 * sms * 256, dtype=torch.int32, device="cuda")
    v = C.c_double(0.0)
    _check(raw.w4_probe_mma_peak(kind, _ptr(scratch), scratch.numel(), C.byref(v), _stream()), "w4_probe_mma_peak")
    return float(v.value)


def version() -> int:
    return int(raw.w4_version())
