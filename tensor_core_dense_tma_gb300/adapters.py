"""Low-rank adapters of many requests beside a shared product (the C ABI of
``include/adapters.h``): ``Plan.linear_adapters`` and ``Plan.linear_adapters_grad``.

This module reads sizes, storage orders and strides from the tensors; the
computation is the library's kernels on the given (or current) stream.  A
stack of factors is G x R x K (``down``) or G x N x R (``up``), with unit stride
along either of its last two dimensions: ``up.transpose(1, 2)`` is a ``down``
for the backward direction without a copy.

What a call returns belongs to torch's current stream; with another ``stream``
order the two, as for any tensor used on a second stream.  A result that is not
looked at (``hidden`` where one serves) may be dropped at once.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from .logits import _stream

__all__ = ["AdaptersGrad", "MAX_RANK"]

MAX_RANK = 128


class AdaptersGrad(NamedTuple):
    dX: object             # [M, K] of the plan's type
    d_down: object         # [G, R, K]
    d_up: object           # [G, N, R]


class Adapters(ctypes.Structure):
    """gemm_adapters_t."""
    _fields_ = [("count", ctypes.c_int64), ("rank", ctypes.c_int64), ("down", ctypes.c_void_p),
                ("down_ld", ctypes.c_int64), ("down_stride", ctypes.c_int64), ("down_layout", ctypes.c_int),
                ("up", ctypes.c_void_p), ("up_ld", ctypes.c_int64), ("up_stride", ctypes.c_int64),
                ("up_layout", ctypes.c_int), ("scale", ctypes.c_void_p), ("index", ctypes.c_void_p),
                ("ldp", ctypes.c_int64), ("wide", ctypes.c_int32), ("wide_h", ctypes.c_int32)]


def declare(lib: ctypes.CDLL) -> None:
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    stacks = ctypes.POINTER(Adapters)
    lib.gemm_adapters_hidden_width.argtypes = [i64]
    lib.gemm_adapters_hidden_width.restype = i64
    lib.gemm_run_adapters.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, p, stacks, p, i64, p]
    lib.gemm_run_adapters.restype = i32
    lib.gemm_adapters_grad.argtypes = [p, p, p, i64, i64, i64, i64, i64, stacks, p, p, i64, i32, p, i64, i64, p, i64,
                                       i64, p]
    lib.gemm_adapters_grad.restype = i32


_calls: dict = {}     # the library's entry points and torch, filled on the first use


def _lib():
    import torch
    from . import load, DTYPE, GemmError
    lib = load()
    _calls.update(torch=torch, error=GemmError, run=lib.gemm_run_adapters, grad=lib.gemm_adapters_grad,
                  codes={torch.float16: DTYPE["f16"], torch.bfloat16: DTYPE["bf16"], torch.float32: DTYPE["f32"]},
                  types={"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}, empty=torch.empty,
                  stream=torch._C._cuda_getCurrentRawStream, f32=torch.float32, f16=torch.float16,
                  i32=torch.int32)
    return _calls


def hidden_width(rank: int) -> int:
    """Columns of the hidden rows of adapters of this rank (gemm_adapters_hidden_width)."""
    return 32 if rank <= 16 else 64 if rank <= 32 else 128 if rank <= 64 else 256


# A decoding step's kernels take ten to thirty microseconds, so what follows looks at each
# tensor once (an attribute of a tensor is 0.1 us, a call 0.2), and sorts out what
# is wrong only once something is.

def _refuse_matrix(t, what: str, di: int, dtype):
    if t.dim() != 2 or t.dtype != dtype or t.get_device() != di:
        raise ValueError(f"{what} must be a 2-D {dtype} tensor on X's device")
    raise ValueError(f"{what} must be row-major (strides {t.stride()})")


def _row_ld(t, what: str, di: int, dtype) -> int:
    """Row stride of a row-major matrix of the plan's type on device di."""
    if t.dim() != 2 or t.dtype is not dtype or t.get_device() != di:
        _refuse_matrix(t, what, di, dtype)
    (r, c), (s0, s1) = t.shape, t.stride()
    if (s1 != 1 and c > 1) or (s0 < c and r > 1):
        _refuse_matrix(t, what, di, dtype)
    return s0 if r > 1 else -(-c // 8) * 8


def _order(r, c, s0, s1):
    """(leading dimension, layout) of an r x c matrix, or None: by the dimension
    that has unit stride and more than one element.  A single row or column has
    no stride of its own: any will do."""
    if c > 1 and s1 == 1 and (s0 >= c or r <= 1):
        return (s0 if r > 1 else -(-c // 8) * 8), 0
    if r > 1 and s0 == 1 and (s1 >= r or c <= 1):
        return (s1 if c > 1 else -(-r // 8) * 8), 1
    if c <= 1:
        return (s0 if r > 1 else 8), 0
    return (s1, 1) if r <= 1 else None


def _stack(t, what: str, di: int, dtype, G, r, c):
    """(address, leading dimension, stride, layout) of a stack of matrices."""
    if t.dtype is not dtype or t.get_device() != di or t.shape != (G, r, c):
        raise ValueError(f"{what} must be a {G} x {r} x {c} {dtype} tensor on X's device")
    s, s0, s1 = t.stride()
    order = _order(r, c, s0, s1)
    if order is None:
        raise ValueError(f"{what} must have unit stride along one of its last two dimensions (strides {t.stride()})")
    return t.data_ptr(), order[0], (s if G > 1 else 0), order[1]


def _adapters(down, up, index, scale, M, N, K, di, dtype):
    """G, R, the fields of gemm_adapters_t that describe down and up, and the
    addresses of scale and index."""
    if down.dim() != 3 or up.dim() != 3:
        raise ValueError("down must be G x R x K, up G x N x R")
    G, R, _ = down.shape
    if not 1 <= R <= MAX_RANK:
        raise ValueError(f"the rank must be 1..{MAX_RANK}")
    if index.dtype is not _calls["i32"] or index.shape != (M,) or index.get_device() != di or not index.is_contiguous():
        raise ValueError("index must be a contiguous int32 vector with one entry per row on X's device")
    if scale is not None and (scale.dtype is not _calls["f32"] or scale.shape != (G,) or scale.get_device() != di
                              or not scale.is_contiguous()):
        raise ValueError("scale must be a contiguous fp32 vector with one entry per adapter on X's device")
    return (G, R, _stack(down, "down", di, dtype, G, R, K), _stack(up, "up", di, dtype, G, N, R),
            None if scale is None else scale.data_ptr(), index.data_ptr())


def _hidden(hidden, M, R, dev, di, dtype):
    """(hidden, its row stride, whether it is wide); allocated if not given."""
    width = hidden_width(R)
    if hidden is None:
        return _calls["empty"]((M, width), dtype=dtype, device=dev), width, 0
    wide = 1 if dtype is _calls["f16"] and hidden.shape == (M, width // 2 * 3) else 0
    if not wide and hidden.shape != (M, width):
        raise ValueError(f"hidden must be {M} x {width}" + (f" or {M} x {width // 2 * 3}" if dtype is _calls["f16"] else ""))
    return hidden, _row_ld(hidden, "hidden", di, dtype), wide


def _weights(B, di: int, dtype, K, N):
    """(leading dimension, layout) of the K x N matrix B."""
    if B.dtype is not dtype or B.get_device() != di:
        raise ValueError(f"B must be a 2-D {dtype} tensor on X's device")
    order = _order(K, N, *B.stride())
    if order is None:
        raise ValueError(f"B must be row- or column-major (strides {B.stride()})")
    return order


def _result(D, what: str, M, N, di: int, dev, wanted, own):
    """(D, its type, its row stride); allocated if not given, of the type that is wanted or the plan's own."""
    if D is None:
        out = wanted or own
        return _calls["empty"]((M, N), dtype=out, device=dev), out, N
    out = D.dtype
    if wanted is not None and out is not wanted:
        raise ValueError(f"{what} must have the output type")
    d0, d1 = D.stride() if D.dim() == 2 else (0, 0)
    if out not in _calls["codes"] or D.shape != (M, N) or D.get_device() != di or (d1 != 1 and N > 1) or \
            (d0 < N and M > 1):
        raise ValueError(f"{what} must be a row-major matrix of the result's size on X's device")
    return D, out, (d0 if M > 1 else N)


def linear(plan, X, B, down, up, index, scale, D, bias, hidden, out_dtype, stream):
    """Plan.linear_adapters."""
    calls = _calls or _lib()
    types = calls["types"]
    dtype, dev, di = types.get(plan.in_dtype), X.device, X.get_device()
    if dtype is None or dtype is calls["f32"] or di != plan.device or X.dim() != 2 or B.dim() != 2:
        raise ValueError("adapters take 2-D tensors on the plan's device and an f16 or bf16 plan")
    (M, K), (KB, N) = X.shape, B.shape
    ldx = _row_ld(X, "X", di, dtype)
    if KB != K:
        raise ValueError("inner dimensions differ")
    order = _weights(B, di, dtype, K, N)
    G, R, lower, upper, scales, at = _adapters(down, up, index, scale, M, N, K, di, dtype)
    given = D, hidden
    D, out, ldd = _result(D, "D", M, N, di, dev, None if out_dtype is None else types[out_dtype], dtype)
    if bias is not None and (bias.dtype is not calls["f32"] or bias.shape != (N,) or bias.get_device() != di
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous fp32 vector of length N on X's device")
    hidden, ldh, wide = _hidden(hidden, M, R, dev, di, dtype)
    a = Adapters(G, R, *lower, *upper, scales, at, 0, wide)
    if stream is None:
        stream = calls["stream"](di)
    else:
        _stream(stream, dev, *[t for t, g in zip((D, hidden), given) if g is None])
    st = calls["run"](plan.handle, X.data_ptr(), B.data_ptr(), D.data_ptr(), M, N, K, ldx, order[0], ldd, order[1],
                      calls["codes"][out], None if bias is None else bias.data_ptr(), ctypes.byref(a),
                      hidden.data_ptr(), ldh, stream)
    if st != 0:
        raise calls["error"](st, "gemm_run_adapters")
    return D, hidden


def _gradient(t, dtype, dev, di, shape, what):
    """(tensor, leading dimension, stride) of an output stack, allocated if not given."""
    G, rows, cols = shape
    if t is None:
        return _calls["empty"](shape, dtype=dtype, device=dev), cols, rows * cols
    if t.shape != shape or t.get_device() != di:
        raise ValueError(f"{what} must be a {G} x {rows} x {cols} tensor on X's device")
    s, s0, s1 = t.stride()
    if (cols > 1 and s1 != 1) or (rows > 1 and s0 < cols) or (G > 1 and s < (rows - 1) * s0 + cols):
        raise ValueError(f"{what} must have unit stride along its last dimension (strides {t.stride()})")
    return t, (s0 if rows > 1 else cols), (s if G > 1 else 0)


def linear_grad(plan, dY, B, X, hidden, down, up, index, scale, dX, d_down, d_up, stream):
    """Plan.linear_adapters_grad."""
    calls = _calls or _lib()
    dtype, dev, di = calls["types"].get(plan.in_dtype), X.device, X.get_device()
    if dtype is None or dtype is calls["f32"] or di != plan.device or X.dim() != 2 or dY.dim() != 2 or B.dim() != 2:
        raise ValueError("adapters take 2-D tensors on the plan's device and an f16 or bf16 plan")
    (M, K), (MY, N) = X.shape, dY.shape
    if MY != M or B.shape != (K, N):
        raise ValueError("dY must be M x N, B K x N")
    ldx = _row_ld(X, "X", di, dtype)
    lddy = _row_ld(dY, "dY", di, dtype)
    ldb, layout = _weights(B, di, dtype, K, N)
    G, R, lower, upper, scales, at = _adapters(down, up, index, scale, M, N, K, di, dtype)
    if hidden is None and M and G:
        raise ValueError("hidden must be what linear_adapters returned")
    given = dX, d_down, d_up
    dX, x_type, lddx = _result(dX, "dX", M, K, di, dev, None, dtype)
    hidden, ldh, wide = _hidden(hidden, M, R, dev, di, dtype)
    like = d_down if d_down is not None else d_up
    out = dtype if like is None else like.dtype
    if out not in (calls["f32"], dtype) or (d_up is not None and d_up.dtype is not out):
        raise ValueError("d_down and d_up must both be fp32 or both of the plan's type")
    d_down, down_ld, down_stride = _gradient(d_down, out, dev, di, (G, R, K), "d_down")
    d_up, up_ld, up_stride = _gradient(d_up, out, dev, di, (G, N, R), "d_up")
    # (p is far smaller than h while up is near 0)
    f16 = 1 if dtype is calls["f16"] else 0
    ldp = hidden_width(R) // 2 * (2 + f16)
    p = calls["empty"]((M, ldp), dtype=dtype, device=dev)
    if stream is None:
        stream = calls["stream"](di)
    else:
        _stream(stream, dev, p, *[t for t, g in zip((dX, d_down, d_up), given) if g is None])
    # dX is the same product the other way round (a matrix's transpose is the same memory in
    # the other order), and leaves p as its hidden rows
    a = Adapters(G, R, *upper[:3], 1 - upper[3], *lower[:3], 1 - lower[3], scales, at, ldp, f16, wide)
    this, other, kept, mine = X.data_ptr(), dY.data_ptr(), hidden.data_ptr(), p.data_ptr()
    st = calls["run"](plan.handle, other, B.data_ptr(), dX.data_ptr(), M, K, N, lddy, ldb, lddx, 1 - layout,
                      calls["codes"][x_type], None, ctypes.byref(a), mine, ldp, stream)
    if st == 0:
        st = calls["grad"](plan.handle, this, other, M, N, K, ldx, lddy, ctypes.byref(a), kept, mine, ldh,
                           calls["codes"][out], d_down.data_ptr(), down_ld, down_stride, d_up.data_ptr(), up_ld,
                           up_stride, stream)
    if st != 0:
        raise calls["error"](st, "gemm_run_adapters or gemm_adapters_grad")
    return AdaptersGrad(dX, d_down, d_up)
