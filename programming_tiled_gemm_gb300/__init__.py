"""Python binding of the GB300 GEMM library (``include/gemm.h``).

Argument marshalling only: every function forwards to the C entry point of the same
name in ``lib/libgemm_gb300.so``; all arithmetic runs in the library's CUDA kernels.
PyTorch is used for device memory and streams (``matmul`` and ``conv4d`` take tensors).
There is no fallback: if the library is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
# GEMM_GB300_DEBUG=1 loads the debug build (computed global indices checked in the
# kernels; a failed check is reported by gemm_get_device_status as GEMM_ERR_DEVICE_BOUNDS).
DEBUG = os.environ.get("GEMM_GB300_DEBUG") == "1"
LIB_PATH = os.path.join(_PKG, "lib", "libgemm_gb300_debug.so" if DEBUG else "libgemm_gb300.so")

GEMM_F32, GEMM_BF16, GEMM_F16 = 0, 1, 2
GEMM_OK = 0
GEMM_ERR_INVALID_ARG = -1
GEMM_ERR_ALIGNMENT = -2
GEMM_ERR_UNSUPPORTED = -3
GEMM_ERR_CUDA = -4
GEMM_ERR_DEVICE_TIMEOUT = -5
GEMM_ERR_DEVICE_BOUNDS = -6
GEMM_OPT_F32_KERNEL, GEMM_OPT_SPLIT_K, GEMM_OPT_WAIT_LIMIT_US, GEMM_OPT_TC_CHUNK, GEMM_OPT_TC_PAIR = 1, 2, 3, 4, 5
GEMM_OPT_TEST_STALL = 6
GEMM_OPT_CONV_STACK = 7
GEMM_OPT_CONV_SPLIT = 8
GEMM_OPT_TEST_STALL_PAIR = 9

# Every symbol include/gemm.h declares (the ABI test checks the library exports them).
EXPORTS = ["gemm_create", "gemm_destroy", "gemm_run", "gemm_run_ex", "gemm_run_host", "gemm_run_host_batch",
           "conv4d_im2col",
           "conv4d_forward", "conv4d_forward_cl", "conv4d_forward_tc",
           "gemm_get_device_status", "gemm_set_option", "gemm_launch_count", "gemm_status_string",
           "gemm_run_f32_skinny_noalloc",
           "gemm_linear", "gemm_linear_backward", "moe_route", "moe_route_backward", "moe_dispatch", "moe_combine",
           "moe_combine_backward"]

GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_TANH, GEMM_ACT_SILU, GEMM_ACT_SWIGLU = 0, 1, 2, 3, 4, 5
ACTIVATIONS = {"none": GEMM_ACT_NONE, "relu": GEMM_ACT_RELU, "gelu": GEMM_ACT_GELU, "gelu_tanh": GEMM_ACT_GELU_TANH,
               "silu": GEMM_ACT_SILU, "swiglu": GEMM_ACT_SWIGLU}


class HostProblem(ctypes.Structure):
    """gemm_host_problem: one product of gemm_run_host_batch."""
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("A", ctypes.c_void_p),
                ("lda", ctypes.c_int64), ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("C", ctypes.c_void_p),
                ("ldc", ctypes.c_int64), ("dtype", ctypes.c_int)]


class LinearArgs(ctypes.Structure):
    """gemm_linear_args."""
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("X", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("w_stride", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("R", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("Z", ctypes.c_void_p),
                ("ldz", ctypes.c_int64), ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("dtype", ctypes.c_int), ("y_dtype", ctypes.c_int),
                ("act", ctypes.c_int)]


class LinearGradArgs(ctypes.Structure):
    """gemm_linear_grad_args."""
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("dY", ctypes.c_void_p),
                ("lddy", ctypes.c_int64), ("X", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("Z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("dX", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dW", ctypes.c_void_p), ("lddw", ctypes.c_int64),
                ("dw_stride", ctypes.c_int64), ("db", ctypes.c_void_p), ("groups", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("dtype", ctypes.c_int), ("dw_dtype", ctypes.c_int),
                ("act", ctypes.c_int)]


class Routing(NamedTuple):
    """What moe_route leaves: torch tensors, see include/gemm.h."""
    weights: object  # fp32 [T, k]
    experts: object  # int32 [T, k], -1: none
    slots: object    # int32 [T, k], the pick's row in the order by expert, -1: none
    rows: object     # int32 [T * k], the pick t * k + j at each row, -1 past the last
    offsets: object  # int32 [E + 1], the groups of grouped_linear


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s%s (status %d)" % (what + ": " if what else "", status_string(status), status))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("%s is not built; run __graft_entry__.build() first" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.gemm_create.argtypes = [ctypes.POINTER(p), i32]
    lib.gemm_destroy.argtypes = [p]
    lib.gemm_run.argtypes = [p, i64, i64, i64, p, i64, p, i64, p, i64, i32, p]
    lib.gemm_run_host.argtypes = [p, i64, i64, i64, p, i64, p, i64, p, i64, i32, p]
    lib.gemm_run_host_batch.argtypes = [p, i32, ctypes.POINTER(HostProblem), p]
    f32 = ctypes.c_float
    lib.gemm_run_ex.argtypes = [p, i64, i64, i64, f32, p, i64, p, i64, f32, p, i64, i32, i32, p]
    lib.conv4d_im2col.argtypes = [p, p, i64, ctypes.POINTER(i64), ctypes.POINTER(i64), p, p]
    lib.conv4d_forward.argtypes = [p, p, i64, ctypes.POINTER(i64), p, i64, ctypes.POINTER(i64), p, i64, p]
    lib.conv4d_forward_cl.argtypes = [p, p, i64, ctypes.POINTER(i64), p, i64, ctypes.POINTER(i64), p, i32, p]
    lib.conv4d_forward_tc.argtypes = [p, p, i64, ctypes.POINTER(i64), p, i64, ctypes.POINTER(i64), p, i64, i32, p]
    lib.gemm_get_device_status.argtypes = [p, p]
    lib.gemm_set_option.argtypes = [p, i32, i64]
    lib.gemm_launch_count.argtypes = [p]
    lib.gemm_run_f32_skinny_noalloc.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, i32, p]
    lib.gemm_linear.argtypes = [p, ctypes.POINTER(LinearArgs), p]
    lib.gemm_linear_backward.argtypes = [p, ctypes.POINTER(LinearGradArgs), p]
    lib.moe_route.argtypes = [p, i64, i64, i64, p, i64, i32, i32, p, p, p, p, p, p]
    lib.moe_route_backward.argtypes = [p, i64, i64, i64, p, p, i64, i32, p, i32, p, i64, p]
    lib.moe_dispatch.argtypes = [p, i64, i64, i64, p, i64, i32, p, p, i64, p]
    lib.moe_combine.argtypes = [p, i64, i64, i64, p, i64, i64, i32, p, p, p, i64, p, i64, p]
    lib.moe_combine_backward.argtypes = [p, i64, i64, i64, p, i64, p, i64, i32, p, p, p, p, i64, p, p]
    lib.gemm_status_string.argtypes = [i32]
    lib.gemm_status_string.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name != "gemm_status_string":
            getattr(lib, name).restype = i32
    lib.gemm_launch_count.restype = i64
    return lib


_lib = _load()


def library():
    """The loaded ctypes library (for callers that want the raw C ABI)."""
    return _lib


# ----------------------------------------------------------------- C ABI, same names

def gemm_create(device: int = 0) -> int:
    h = ctypes.c_void_p()
    rc = _lib.gemm_create(ctypes.byref(h), int(device))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_create")
    return h.value


def gemm_destroy(h: int) -> int:
    return _lib.gemm_destroy(h)


def gemm_run(h, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream=0) -> int:
    return _lib.gemm_run(h, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream)


def gemm_run_ex(h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, ab_dtype, c_dtype, stream=0) -> int:
    return _lib.gemm_run_ex(h, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, ab_dtype, c_dtype, stream)


def gemm_run_host(h, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream=0) -> int:
    return _lib.gemm_run_host(h, M, N, K, A, lda, B, ldb, C, ldc, dtype, stream)


def gemm_run_host_batch(h, problems, stream=0) -> int:
    """problems: a sequence of HostProblem (or tuples of its fields)."""
    arr = (HostProblem * len(problems))(*[q if isinstance(q, HostProblem) else HostProblem(*q) for q in problems])
    return _lib.gemm_run_host_batch(h, len(problems), arr, stream)


def conv4d_im2col(h, x, C_in, in_dims, k_dims, col, stream=0) -> int:
    ins = (ctypes.c_int64 * 4)(*[int(v) for v in in_dims])
    ks = (ctypes.c_int64 * 4)(*[int(v) for v in k_dims])
    return _lib.conv4d_im2col(h, x, C_in, ins, ks, col, stream)


def conv4d_forward(h, x, C_in, in_dims, w, C_out, k_dims, y, ldy, stream=0) -> int:
    ins = (ctypes.c_int64 * 4)(*[int(v) for v in in_dims])
    ks = (ctypes.c_int64 * 4)(*[int(v) for v in k_dims])
    return _lib.conv4d_forward(h, x, C_in, ins, w, C_out, ks, y, ldy, stream)


def conv4d_forward_cl(h, x, C_in, in_dims, w, C_out, k_dims, y, dtype, stream=0) -> int:
    ins = (ctypes.c_int64 * 4)(*[int(v) for v in in_dims])
    ks = (ctypes.c_int64 * 4)(*[int(v) for v in k_dims])
    return _lib.conv4d_forward_cl(h, x, C_in, ins, w, C_out, ks, y, dtype, stream)


def conv4d_forward_tc(h, x, C_in, in_dims, w, C_out, k_dims, y, ldy, dtype, stream=0) -> int:
    ins = (ctypes.c_int64 * 4)(*[int(v) for v in in_dims])
    ks = (ctypes.c_int64 * 4)(*[int(v) for v in k_dims])
    return _lib.conv4d_forward_tc(h, x, C_in, ins, w, C_out, ks, y, ldy, dtype, stream)


def gemm_linear(h, args: LinearArgs, stream=0) -> int:
    return _lib.gemm_linear(h, args, stream)


def gemm_linear_backward(h, args: LinearGradArgs, stream=0) -> int:
    return _lib.gemm_linear_backward(h, args, stream)


def moe_route(h, T, E, k, logits, ldl, dtype, renormalize, weights, experts, slots, rows, offsets, stream=0) -> int:
    return _lib.moe_route(h, T, E, k, logits, ldl, dtype, renormalize, weights, experts, slots, rows, offsets, stream)


def moe_route_backward(h, T, E, k, dweights, logits, ldl, dtype, experts, renormalize, dlogits, lddl, stream=0) -> int:
    return _lib.moe_route_backward(h, T, E, k, dweights, logits, ldl, dtype, experts, renormalize, dlogits, lddl,
                                   stream)


def moe_dispatch(h, T, N, k, x, ldx, dtype, rows, xr, ldxr, stream=0) -> int:
    return _lib.moe_dispatch(h, T, N, k, x, ldx, dtype, rows, xr, ldxr, stream)


def moe_combine(h, T, N, k, y, ldy, rows_y, dtype, slots, weights, R, ldr, out, ldo, stream=0) -> int:
    return _lib.moe_combine(h, T, N, k, y, ldy, rows_y, dtype, slots, weights, R, ldr, out, ldo, stream)


def moe_combine_backward(h, T, N, k, dout, lddo, y, ldy, dtype, slots, rows, weights, dy, lddy, dweights,
                         stream=0) -> int:
    return _lib.moe_combine_backward(h, T, N, k, dout, lddo, y, ldy, dtype, slots, rows, weights, dy, lddy, dweights,
                                     stream)


def gemm_get_device_status(h, stream=0) -> int:
    return _lib.gemm_get_device_status(h, stream)


def gemm_set_option(h, option: int, value: int) -> int:
    return _lib.gemm_set_option(h, int(option), int(value))


def gemm_launch_count(h) -> int:
    return _lib.gemm_launch_count(h)


def status_string(status: int) -> str:
    return _lib.gemm_status_string(int(status)).decode()


gemm_status_string = status_string


# ------------------------------------------------------- tensor conveniences (torch)

_DTYPES = {}


def _dtype_code(t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        import torch
        _DTYPES.update({torch.float32: GEMM_F32, torch.bfloat16: GEMM_BF16, torch.float16: GEMM_F16})
        code = _DTYPES.get(t.dtype)
        if code is None:
            raise TypeError("unsupported input dtype %s" % t.dtype)
    return code


def _row_major_2d(t, name):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("%s must be a 2-D row-major tensor (unit column stride), got strides %s"
                         % (name, tuple(t.stride())))
    return max(t.stride(0), t.shape[1], 1)


def _ptr(t):
    return t.data_ptr() if t is not None else 0


# The argument structures packed into a buffer of the handle's (a ctypes structure of twenty
# fields takes several microseconds to build), and entry points that take their addresses.
_LINEAR = struct.Struct("@qqqPqPqqPPqPqPqqPiii")
_LINEAR_GRAD = struct.Struct("@qqqPqPqPqqPqPqPqqPqPiii")
_raw = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p)
_linear_raw, _linear_backward_raw = _raw(("gemm_linear", _lib)), _raw(("gemm_linear_backward", _lib))


class Gemm:
    """A library handle bound to one CUDA device."""

    def __init__(self, device: int = 0):
        self.device = int(device)
        self.handle = gemm_create(self.device)
        self._args = ctypes.create_string_buffer(max(_LINEAR.size, _LINEAR_GRAD.size) + 8)
        self._args_at = ctypes.addressof(self._args)
        self._dev = None

    def close(self):
        if self.handle:
            gemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_option(self, option: int, value: int):
        rc = gemm_set_option(self.handle, option, value)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_set_option")

    def matmul(self, A, B, out=None, stream=None, alpha=1.0, beta=0.0, out_dtype=None):
        """out[M, N] = alpha * A[M, K] @ B[K, N] + beta * out; A, B fp32 / bf16 / fp16 CUDA
        tensors; out fp32 (default) or bf16 / fp16; out is read only when beta != 0."""
        import torch
        if A.dtype != B.dtype:
            raise TypeError("A and B must have the same dtype")
        M, K = A.shape
        K2, N = B.shape
        if K2 != K:
            raise ValueError("inner dimensions differ")
        if out is None:
            if beta != 0.0:
                raise ValueError("beta != 0 needs an existing out")
            out = torch.empty((M, N), dtype=out_dtype or torch.float32, device=A.device)
        lda, ldb, ldc = _row_major_2d(A, "A"), _row_major_2d(B, "B"), _row_major_2d(out, "out")
        s = torch.cuda.current_stream(A.device).cuda_stream if stream is None else int(stream)
        if alpha == 1.0 and beta == 0.0 and out.dtype == torch.float32:
            rc = gemm_run(self.handle, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc,
                          _dtype_code(A), s)
        else:
            rc = gemm_run_ex(self.handle, M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(), ldb, float(beta),
                             out.data_ptr(), ldc, _dtype_code(A), _dtype_code(out), s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run")
        return out

    def matmul_host(self, A, B, out=None, stream=None):
        """The same product with CPU tensors in and out (copies inside the library)."""
        import torch
        M, K = A.shape
        N = B.shape[1]
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32)
        lda, ldb, ldc = _row_major_2d(A, "A"), _row_major_2d(B, "B"), _row_major_2d(out, "out")
        s = 0 if stream is None else int(stream)
        rc = gemm_run_host(self.handle, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc,
                           _dtype_code(A), s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run_host")
        return out

    def matmul_host_batch(self, pairs, outs=None, stream=None):
        """Several products of CPU tensors as one pipeline: pairs = [(A, B), ...]."""
        import torch
        if outs is None:
            outs = [torch.empty((A.shape[0], B.shape[1]), dtype=torch.float32) for A, B in pairs]
        probs = []
        for (A, B), out in zip(pairs, outs):
            if A.shape[1] != B.shape[0] or tuple(out.shape) != (A.shape[0], B.shape[1]) or A.dtype != B.dtype:
                raise ValueError("shapes or dtypes do not match")
            probs.append(HostProblem(A.shape[0], B.shape[1], A.shape[1], A.data_ptr(), _row_major_2d(A, "A"),
                                     B.data_ptr(), _row_major_2d(B, "B"), out.data_ptr(), _row_major_2d(out, "out"),
                                     _dtype_code(A)))
        s = 0 if stream is None else int(stream)
        rc = gemm_run_host_batch(self.handle, probs, s)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run_host_batch")
        return outs

    def im2col4d(self, x, ks, col=None, stream=None):
        """Column matrix [C_in*prod(ks), prod(in-ks+1)] of a valid 4-D cross-correlation."""
        import torch
        if x.dim() != 5 or x.dtype != torch.float32 or not x.is_contiguous():
            raise ValueError("x must be a contiguous fp32 [C_in, I0, I1, I2, I3] tensor")
        cin = x.shape[0]
        ins = list(x.shape[1:])
        outs = [i - k + 1 for i, k in zip(ins, ks)]
        rows = cin * ks[0] * ks[1] * ks[2] * ks[3]
        cols = outs[0] * outs[1] * outs[2] * outs[3]
        if col is None:
            col = torch.empty((rows, cols), dtype=torch.float32, device=x.device)
        s = torch.cuda.current_stream(x.device).cuda_stream if stream is None else int(stream)
        rc = conv4d_im2col(self.handle, x.data_ptr(), cin, ins, ks, col.data_ptr(), s)
        if rc != GEMM_OK:
            raise GemmError(rc, "conv4d_im2col")
        return col

    def conv4d_implicit(self, x, w, out=None, stream=None):
        """Valid 4-D cross-correlation as an implicit GEMM: y[C_out, P0, P1, P2, P3]."""
        import torch
        if x.dim() != 5 or w.dim() != 6 or x.dtype != torch.float32 or w.dtype != torch.float32:
            raise ValueError("x must be fp32 [C_in, I0..I3] and w fp32 [C_out, C_in, R0..R3]")
        if not (x.is_contiguous() and w.is_contiguous()):
            raise ValueError("x and w must be contiguous")
        cin, cout = x.shape[0], w.shape[0]
        ks = list(w.shape[2:])
        outs = [i - k + 1 for i, k in zip(x.shape[1:], ks)]
        npos = outs[0] * outs[1] * outs[2] * outs[3]
        if out is None:
            out = torch.empty((cout, npos), dtype=torch.float32, device=x.device)
        ldy = _row_major_2d(out, "out")
        s = torch.cuda.current_stream(x.device).cuda_stream if stream is None else int(stream)
        rc = conv4d_forward(self.handle, x.data_ptr(), cin, list(x.shape[1:]), w.data_ptr(), cout, ks,
                            out.data_ptr(), ldy, s)
        if rc != GEMM_OK:
            raise GemmError(rc, "conv4d_forward")
        return out.view(cout, *outs) if out.is_contiguous() else out

    def conv4d_cl(self, x, w, out=None, stream=None):
        """Valid 4-D cross-correlation on the tensor cores, channel-last 16-bit operands.

        x: [I0, I1, I2, I3, C_in] and w: [C_out, R0, R1, R2, R3, C_in], both bf16 or both
        fp16, contiguous; returns y: fp32 [P0, P1, P2, P3, C_out]."""
        import torch
        dt = {torch.bfloat16: GEMM_BF16, torch.float16: GEMM_F16}.get(x.dtype)
        if x.dim() != 5 or w.dim() != 6 or dt is None or w.dtype != x.dtype:
            raise ValueError("x must be [I0..I3, C_in] and w [C_out, R0..R3, C_in], both bf16 or both fp16")
        if not (x.is_contiguous() and w.is_contiguous()) or w.shape[5] != x.shape[4]:
            raise ValueError("x and w must be contiguous with the same C_in")
        cin, cout = x.shape[4], w.shape[0]
        ins, ks = list(x.shape[:4]), list(w.shape[1:5])
        outs = [i - k + 1 for i, k in zip(ins, ks)]
        if out is None:
            out = torch.empty(outs + [cout], dtype=torch.float32, device=x.device)
        elif list(out.shape) != outs + [cout] or out.dtype != torch.float32 or not out.is_contiguous():
            raise ValueError("out must be contiguous fp32 %s" % (outs + [cout],))
        s = torch.cuda.current_stream(x.device).cuda_stream if stream is None else int(stream)
        rc = conv4d_forward_cl(self.handle, x.data_ptr(), cin, ins, w.data_ptr(), cout, ks, out.data_ptr(), dt, s)
        if rc != GEMM_OK:
            raise GemmError(rc, "conv4d_forward_cl")
        return out

    def conv4d_tc(self, x, w, out=None, stream=None):
        """Valid 4-D cross-correlation on the tensor cores, channel-first 16-bit operands.

        x: [C_in, I0, I1, I2, I3] and w: [C_out, C_in, R0, R1, R2, R3], both bf16 or both
        fp16, contiguous; returns y: fp32 [C_out, P0, P1, P2, P3] (or writes `out`, whose
        rows over the output positions may be strided: out[o] at out.data_ptr() + o
        out.stride(0))."""
        import torch
        dt = {torch.bfloat16: GEMM_BF16, torch.float16: GEMM_F16}.get(x.dtype)
        if x.dim() != 5 or w.dim() != 6 or dt is None or w.dtype != x.dtype:
            raise ValueError("x must be [C_in, I0..I3] and w [C_out, C_in, R0..R3], both bf16 or both fp16")
        if not (x.is_contiguous() and w.is_contiguous()) or w.shape[1] != x.shape[0]:
            raise ValueError("x and w must be contiguous with the same C_in")
        cin, cout = x.shape[0], w.shape[0]
        ins, ks = list(x.shape[1:]), list(w.shape[2:])
        outs = [i - k + 1 for i, k in zip(ins, ks)]
        npos = 1
        for v in outs:
            npos *= v
        if out is None:
            out = torch.empty([cout] + outs, dtype=torch.float32, device=x.device)
        if out.dtype != torch.float32 or out.shape[0] != cout or out[0].numel() != npos or \
                not out[0].is_contiguous():
            raise ValueError("out must be fp32 [%d, %s] with contiguous rows" % (cout, outs))
        s = torch.cuda.current_stream(x.device).cuda_stream if stream is None else int(stream)
        rc = conv4d_forward_tc(self.handle, x.data_ptr(), cin, ins, w.data_ptr(), cout, ks, out.data_ptr(),
                               out.stride(0), dt, s)
        if rc != GEMM_OK:
            raise GemmError(rc, "conv4d_forward_tc")
        return out

    def conv4d(self, x, w, col=None, out=None, stream=None):
        """Valid 4-D cross-correlation as im2col + GEMM: y[C_out, P0, P1, P2, P3]."""
        ks = list(w.shape[2:])
        col = self.im2col4d(x, ks, col=col, stream=stream)
        cout = w.shape[0]
        y = self.matmul(w.reshape(cout, -1), col, out=out, stream=stream)
        outs = [i - k + 1 for i, k in zip(x.shape[1:], ks)]
        return y.view(cout, *outs)

    # ---- linear layers and routing

    def _new(self, shape, dtype, stream):
        """An output of the call on `stream` (None: the current one)."""
        import torch
        if self._dev is None:
            self._dev = torch.device("cuda", self.device)
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._dev)
        with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=self._dev)):
            return torch.empty(shape, dtype=dtype, device=self._dev)

    def _stream(self, stream):
        if stream is not None:
            return int(stream)
        import torch
        return torch._C._cuda_getCurrentRawStream(self.device)

    def _mat(self, t, name, rows, cols, dtype):
        """Leading dimension of a row-major matrix of that shape and type on this device."""
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != (rows, cols):
            raise ValueError("%s must have shape %s, got %s" % (name, (rows, cols), tuple(t.shape)))
        if t.get_device() != self.device:
            raise ValueError("%s must be on cuda:%d, got %s" % (name, self.device, t.device))
        ld, step = t.stride()
        if (step != 1 and cols > 1) or (ld < cols and rows > 1):
            raise ValueError("%s must be row-major (unit column stride), got strides %s" % (name, (ld, step)))
        return ld if ld > cols else (cols or 1)

    def _flat(self, t, name, shape, dtype):
        """Address of a contiguous tensor of that shape and type on this device."""
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d" % (name, dtype, shape, self.device))
        return t.data_ptr()

    def _weights(self, w, K, dtype, offsets):
        """(groups, ldw, w_stride, columns) of w: [K, Nw], or [G, K, Nw] with offsets [G + 1]."""
        shape = w.shape
        if offsets is None:
            if len(shape) != 2 or shape[0] != K:
                raise ValueError("w must be [K, N] with K = %d, got %s" % (K, tuple(shape)))
            return 0, self._mat(w, "w", K, shape[1], dtype), 0, shape[1]
        if len(shape) != 3 or shape[1] != K or shape[0] == 0:
            raise ValueError("w must be [G, K, N] with K = %d, got %s" % (K, tuple(shape)))
        G, _, Nw = shape
        ld = self._mat(w[0], "w", K, Nw, dtype)
        stride = w.stride(0)
        import torch
        self._flat(offsets, "offsets", (G + 1,), torch.int32)
        return G, ld, stride, Nw

    def _linear(self, x, w, offsets, bias, act, residual, out, out_dtype, save_preact, stream):
        code = ACTIVATIONS[act]
        if x.dim() != 2:
            raise ValueError("x must be [M, K]")
        M, K = x.shape
        dt = x.dtype
        dcode = _dtype_code(x)
        ldx = self._mat(x, "x", M, K, dt)
        G, ldw, w_stride, Nw = self._weights(w, K, dt, offsets)
        if code == GEMM_ACT_SWIGLU:
            if Nw % 2:
                raise ValueError("swiglu needs an even number of columns of w (gate, then up)")
            N = Nw // 2
        else:
            N = Nw
        at_bias = self._flat(bias, "bias", (G, Nw) if G else (Nw,), dt) if bias is not None else 0
        if out is None:
            out = self._new((M, N), out_dtype or (residual.dtype if residual is not None else dt), stream)
            ldy = N
        else:
            ldy = self._mat(out, "out", M, N, out.dtype)
        ycode = dcode if out.dtype is dt else _dtype_code(out)
        ldr = at_r = 0
        if residual is not None:
            ldr, at_r = self._mat(residual, "residual", M, N, out.dtype), residual.data_ptr()
        z = self._new((M, Nw), dt, stream) if save_preact else None
        _LINEAR.pack_into(self._args, 0, M, K, N, x.data_ptr(), ldx, w.data_ptr(), ldw, w_stride, at_bias, at_r, ldr,
                          _ptr(z), Nw, out.data_ptr(), ldy, G, _ptr(offsets), dcode, ycode, code)
        rc = _linear_raw(self.handle, self._args_at, self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_linear")
        return (out, z) if save_preact else out

    def linear(self, x, w, bias=None, act="none", residual=None, out=None, out_dtype=None, save_preact=False,
               stream=None):
        """act(x @ w + bias) + residual: x [M, K], w [K, N] ([K, 2 N] for "swiglu": gate columns,
        then up columns), bf16 or fp16; act one of ACTIVATIONS.  The result (of x's type, or
        float32: out_dtype, residual's or out's type) has shape [M, N].  save_preact=True
        returns (result, x @ w + bias) for linear_backward."""
        return self._linear(x, w, None, bias, act, residual, out, out_dtype, save_preact, stream)

    def grouped_linear(self, x, w, offsets, bias=None, act="none", residual=None, out=None, out_dtype=None,
                       save_preact=False, stream=None):
        """linear with one weight matrix a group of rows: w [G, K, N], bias [G, N]; rows
        offsets[g] .. offsets[g + 1] - 1 of x use w[g].  offsets: int32 [G + 1] on the device.
        Rows from offsets[G] on are not written."""
        if offsets is None:
            raise ValueError("grouped_linear needs offsets")
        return self._linear(x, w, offsets, bias, act, residual, out, out_dtype, save_preact, stream)

    def _linear_backward(self, dy, x, w, offsets, z, act, bias, need_dx, need_dw, dw_dtype, stream):
        import torch
        code = ACTIVATIONS[act]
        if x.dim() != 2:
            raise ValueError("x must be [M, K]")
        M, K = x.shape
        dt = x.dtype
        dcode = _dtype_code(x)
        ldx = self._mat(x, "x", M, K, dt)
        G, ldw, w_stride, Nw = self._weights(w, K, dt, offsets)
        if code == GEMM_ACT_SWIGLU:
            if Nw % 2:
                raise ValueError("swiglu needs an even number of columns of w (gate, then up)")
            N = Nw // 2
        else:
            N = Nw
        lddy = self._mat(dy, "dy", M, N, dt)
        ldz = at_z = 0
        if code != GEMM_ACT_NONE:
            if z is None:
                raise ValueError("act %r needs z, the activation's input" % act)
            ldz, at_z = self._mat(z, "z", M, Nw, dt), z.data_ptr()
        dx = self._new((M, K), dt, stream) if need_dx else None
        dw = self._new(w.shape, dw_dtype or dt, stream) if need_dw else None
        db = self._new((G, Nw) if G else (Nw,), torch.float32, stream) if bias else None
        _LINEAR_GRAD.pack_into(self._args, 0, M, K, N, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw, w_stride,
                               at_z, ldz, _ptr(dx), K, _ptr(dw), Nw, K * Nw, _ptr(db), G, _ptr(offsets), dcode,
                               _dtype_code(dw) if need_dw else dcode, code)
        rc = _linear_backward_raw(self.handle, self._args_at, self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_linear_backward")
        return dx, dw, db

    def linear_backward(self, dy, x, w, z=None, act="none", bias=False, need_dx=True, need_dw=True, dw_dtype=None,
                        stream=None):
        """(dx, dw, db) of linear for the gradient dy of its result; z is what save_preact returned
        (not needed for "none").  db (float32) is None unless bias; dx, dw None where not needed.
        The residual's gradient is dy."""
        return self._linear_backward(dy, x, w, None, z, act, bias, need_dx, need_dw, dw_dtype, stream)

    def grouped_linear_backward(self, dy, x, w, offsets, z=None, act="none", bias=False, need_dx=True, need_dw=True,
                                dw_dtype=None, stream=None):
        """(dx, dw, db) of grouped_linear; dw [G, K, N], db [G, N], zeros for a group without rows."""
        if offsets is None:
            raise ValueError("grouped_linear_backward needs offsets")
        return self._linear_backward(dy, x, w, offsets, z, act, bias, need_dx, need_dw, dw_dtype, stream)

    def moe_route(self, logits, k, renormalize=True, stream=None):
        """Top-k of softmax(logits) over the experts and the order of the picks by expert: a Routing.
        logits [T, E]; -inf marks an expert as not there."""
        import torch
        if logits.dim() != 2:
            raise ValueError("logits must be [T, E]")
        T, E = logits.shape
        k = int(k)
        dcode = _dtype_code(logits)
        ld = self._mat(logits, "logits", T, E, logits.dtype)
        if not 1 <= k <= E:
            raise ValueError("k must be between 1 and the number of experts")
        weights = self._new((T, k), torch.float32, stream)
        i32 = torch.int32
        r = Routing(weights, self._new((T, k), i32, stream), self._new((T, k), i32, stream),
                    self._new((T * k,), i32, stream), self._new((E + 1,), i32, stream))
        rc = _lib.moe_route(self.handle, T, E, k, logits.data_ptr(), ld, dcode, 1 if renormalize else 0,
                            weights.data_ptr(), r.experts.data_ptr(), r.slots.data_ptr(), r.rows.data_ptr(),
                            r.offsets.data_ptr(), self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "moe_route")
        return r

    def moe_route_backward(self, dweights, logits, experts, renormalize=True, out=None, stream=None):
        """The gradient of the logits for the gradient dweights [T, k] of Routing.weights."""
        import torch
        if logits.dim() != 2 or experts.dim() != 2:
            raise ValueError("logits must be [T, E] and experts [T, k]")
        T, E = logits.shape
        k = experts.shape[1]
        dt = logits.dtype
        dcode = _dtype_code(logits)
        ld = self._mat(logits, "logits", T, E, dt)
        if out is None:
            out, ldo = self._new((T, E), dt, stream), E
        else:
            ldo = self._mat(out, "out", T, E, dt)
        rc = _lib.moe_route_backward(self.handle, T, E, k, self._flat(dweights, "dweights", (T, k), torch.float32),
                                     logits.data_ptr(), ld, dcode, self._flat(experts, "experts", (T, k), torch.int32),
                                     1 if renormalize else 0, out.data_ptr(), ldo, self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "moe_route_backward")
        return out

    def moe_dispatch(self, x, rows, k, out=None, stream=None):
        """x [T, N] in the experts' order: [T * k, N], zeros where rows is -1.  Its gradient is
        moe_combine of the rows' gradients without weights."""
        import torch
        if x.dim() != 2:
            raise ValueError("x must be [T, N]")
        T, N = x.shape
        k = int(k)
        dt = x.dtype
        dcode = _dtype_code(x)
        ldx = self._mat(x, "x", T, N, dt)
        at_rows = self._flat(rows, "rows", (T * k,), torch.int32)
        if out is None:
            out, ldo = self._new((T * k, N), dt, stream), N
        else:
            ldo = self._mat(out, "out", T * k, N, dt)
        rc = _lib.moe_dispatch(self.handle, T, N, k, x.data_ptr(), ldx, dcode, at_rows, out.data_ptr(), ldo,
                               self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "moe_dispatch")
        return out

    def moe_combine(self, y, slots, weights=None, residual=None, out=None, stream=None):
        """sum over j of weights[t, j] * y[slots[t, j]] + residual[t]: [T, N].  weights None: ones."""
        import torch
        if y.dim() != 2 or slots.dim() != 2:
            raise ValueError("y must be [rows, N] and slots [T, k]")
        T, k = slots.shape
        R, N = y.shape
        dt = y.dtype
        dcode = _dtype_code(y)
        ldy = self._mat(y, "y", R, N, dt)
        if out is None:
            out, ldo = self._new((T, N), dt, stream), N
        else:
            ldo = self._mat(out, "out", T, N, dt)
        at_w = self._flat(weights, "weights", (T, k), torch.float32) if weights is not None else 0
        ldr = at_r = 0
        if residual is not None:
            ldr, at_r = self._mat(residual, "residual", T, N, dt), residual.data_ptr()
        rc = _lib.moe_combine(self.handle, T, N, k, y.data_ptr(), ldy, R, dcode,
                              self._flat(slots, "slots", (T, k), torch.int32), at_w, at_r, ldr, out.data_ptr(), ldo,
                              self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "moe_combine")
        return out

    def moe_combine_backward(self, dout, y, slots, rows, weights, stream=None):
        """(dy, dweights) of moe_combine: dy [T * k, N] like y, dweights float32 [T, k]."""
        import torch
        if dout.dim() != 2 or slots.dim() != 2:
            raise ValueError("dout must be [T, N] and slots [T, k]")
        T, N = dout.shape
        k = slots.shape[1]
        dt = dout.dtype
        dcode = _dtype_code(dout)
        lddo = self._mat(dout, "dout", T, N, dt)
        ldy = self._mat(y, "y", T * k, N, dt)
        at_slots = self._flat(slots, "slots", (T, k), torch.int32)
        at_rows = self._flat(rows, "rows", (T * k,), torch.int32)
        at_w = self._flat(weights, "weights", (T, k), torch.float32)
        dy = self._new((T * k, N), dt, stream)
        dweights = self._new((T, k), torch.float32, stream)
        rc = _lib.moe_combine_backward(self.handle, T, N, k, dout.data_ptr(), lddo, y.data_ptr(), ldy, dcode, at_slots,
                                       at_rows, at_w, dy.data_ptr(), N, dweights.data_ptr(), self._stream(stream))
        if rc != GEMM_OK:
            raise GemmError(rc, "moe_combine_backward")
        return dy, dweights

    def launch_count(self) -> int:
        return gemm_launch_count(self.handle)

    def device_status(self, stream=None) -> int:
        import torch
        s = torch.cuda.current_stream(self.device).cuda_stream if stream is None else int(stream)
        return gemm_get_device_status(self.handle, s)


__all__ = ["Gemm", "GemmError", "HostProblem", "gemm_create", "gemm_destroy", "gemm_run", "gemm_run_ex",
           "gemm_run_host", "gemm_run_host_batch",
           "conv4d_im2col", "conv4d_forward", "conv4d_forward_cl", "conv4d_forward_tc", "gemm_get_device_status", "gemm_set_option", "gemm_launch_count",
           "gemm_status_string",
           "gemm_linear", "gemm_linear_backward", "moe_route", "moe_route_backward", "moe_dispatch", "moe_combine",
           "moe_combine_backward", "LinearArgs", "LinearGradArgs", "Routing", "ACTIVATIONS",
           "status_string", "library", "LIB_PATH", "EXPORTS"]
