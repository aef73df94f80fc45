"""Operators on the rows of a logits matrix (the C ABI of ``include/logits.h``):
token log-probabilities with entropy and top alternatives, distillation from
a teacher's top logits, and the gradients of both for the logits.

Like the rest of the binding, the functions check and marshal arguments; the
computation is one CUDA kernel per call on the given (or current) stream.

``logits`` is a T x V device tensor of fp32, fp16 or bf16 with unit column
stride; rows may be padded (the product that feeds on a gradient wants row
strides of whole 16 bytes, and an allocated gradient has them).  Logits should
have such rows too, or the gradient be given with the logits' stride: a gradient
row that starts elsewhere within 16 bytes than its logits is stored element by
element (2048 x 65537 bf16 282 us, with equal rows 96).

What a call allocates belongs to torch's current stream; with another
``stream`` order the two, as for any tensor used on a second stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

__all__ = ["TokenLogprobs", "TokenLogprobsGrad", "token_logprobs", "token_logprobs_grad", "distill_topk",
           "distill_topk_grad", "MAX_TOP", "MAX_TEACHER"]

MAX_TOP = 128
MAX_TEACHER = 1024


class TokenLogprobs(NamedTuple):
    logprob: object        # [T] fp32, or None without tokens
    entropy: object        # [T] fp32
    lse: object            # [T] fp32
    top_logprob: object    # [T, top] fp32
    top_token: object      # [T, top] int64


class TokenLogprobsGrad(NamedTuple):
    logprob: object
    entropy: object
    lse: object
    dlogits: object        # [T, V] of the logits' type


def declare(lib: ctypes.CDLL) -> None:
    p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    rows = [i32, i32, p, i64, i64, i64]
    lib.logits_logprobs.argtypes = rows + [p, f32, i32, p, p, p, p, p, p]
    lib.logits_logprobs_grad.argtypes = rows + [p, f32, p, p, p, p, p, p, i64, p]
    teacher = [i64, p, i32, p, i64, f32]
    lib.logits_distill.argtypes = rows + teacher + [p, p, p]
    lib.logits_distill_grad.argtypes = rows + teacher + [p, p, p, p, i64, p]
    for f in (lib.logits_logprobs, lib.logits_logprobs_grad, lib.logits_distill, lib.logits_distill_grad):
        f.restype = i32


_types: dict = {}      # filled on the first use, with the library's entry points


def _dtype(t) -> int:
    if not _types:
        import torch
        _types.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _types.get(t.dtype)
    if code is None:
        raise ValueError(f"fp32, fp16 or bf16 wanted, got {t.dtype}")
    return code


def _matrix(t, what: str):
    """(rows, columns, row stride) of a 2-D device tensor with unit column stride."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D device tensor")
    T, V = t.shape
    s0, s1 = t.stride()
    if (V > 1 and s1 != 1) or (T > 1 and s0 < V):
        raise ValueError(f"{what} must be row-major with unit column stride (strides {t.stride()})")
    return T, V, (s0 if T > 1 else V)


def _vector(v, n: int, dtype, device, what: str):
    """Address of a contiguous device vector, or None."""
    if v is None:
        return None
    if v.dtype != dtype or v.dim() != 1 or v.shape[0] != n or v.device != device or (n > 1 and v.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous {dtype} vector of length {n} on the logits' device")
    return v.data_ptr()


def _gradient(dlogits, logits):
    import torch
    T, V = logits.shape
    if dlogits is None:
        unit = 16 // logits.element_size()
        dlogits = torch.empty((T, -(-V // unit) * unit), dtype=logits.dtype, device=logits.device)[:, :V]
    elif dlogits.dtype != logits.dtype or dlogits.shape != logits.shape or dlogits.device != logits.device:
        raise ValueError("dlogits must have the logits' shape, type and device")
    return dlogits, _matrix(dlogits, "dlogits")[2]


def _outputs(T: int, dev, first: bool):
    """Three fp32 vectors of length T (the first one only if asked for).
    Allocated one by one: views of a common buffer take twice as long to make."""
    import torch
    f32 = torch.float32
    return (torch.empty((T,), dtype=f32, device=dev) if first else None,
            torch.empty((T,), dtype=f32, device=dev), torch.empty((T,), dtype=f32, device=dev))


_entry = {}


def _call(name: str, *args):
    f = _entry.get(name)
    if f is None:
        from . import load
        f = _entry[name] = getattr(load(), name)
    st = f(*args)
    if st != 0:
        from . import GemmError
        raise GemmError(st, name)


def _stream(stream, device):
    if stream is not None:
        return stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)    # current_stream() takes 2 us to make an object


def token_logprobs(logits, tokens=None, top: int = 0, *, temperature: float = 1.0, stream=None) -> TokenLogprobs:
    """Log-probability of tokens[i] (int64; one outside 0..V-1 gives 0) under
    softmax(logits[i] / temperature), the row's entropy and log-sum-exp, and
    its `top` most likely tokens with their log-probabilities, equal ones by
    the lowest token (logits_logprobs)."""
    import torch
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    code = _dtype(logits)
    tok = _vector(tokens, T, torch.int64, dev, "tokens")
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be 0..{MAX_TOP}")
    lp, entropy, lse = _outputs(T, dev, tokens is not None)
    top_lp = torch.empty((T, top), dtype=torch.float32, device=dev)
    top_tok = torch.empty((T, top), dtype=torch.int64, device=dev)
    _call("logits_logprobs", dev.index, code, logits.data_ptr(), T, V, ld, tok, temperature, top,
          lp.data_ptr() if lp is not None else None, entropy.data_ptr(), lse.data_ptr(), top_lp.data_ptr(),
          top_tok.data_ptr(), _stream(stream, dev))
    return TokenLogprobs(lp, entropy, lse, top_lp, top_tok)


def token_logprobs_grad(logits, tokens=None, grad_logprob=None, grad_entropy=None, *, temperature: float = 1.0,
                        dlogits=None, stream=None) -> TokenLogprobsGrad:
    """token_logprobs without alternatives, and the gradient for the logits of
    sum(grad_logprob * logprob + grad_entropy * entropy), in one kernel
    (logits_logprobs_grad).  dlogits may be the logits themselves."""
    import torch
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    code = _dtype(logits)
    tok = _vector(tokens, T, torch.int64, dev, "tokens")
    g = _vector(grad_logprob, T, torch.float32, dev, "grad_logprob")
    h = _vector(grad_entropy, T, torch.float32, dev, "grad_entropy")
    if grad_logprob is not None and tokens is None:
        raise ValueError("grad_logprob needs tokens")
    dlogits, ldd = _gradient(dlogits, logits)
    lp, entropy, lse = _outputs(T, dev, tokens is not None)
    _call("logits_logprobs_grad", dev.index, code, logits.data_ptr(), T, V, ld, tok, temperature, g, h,
          lp.data_ptr() if lp is not None else None, entropy.data_ptr(), lse.data_ptr(), dlogits.data_ptr(), ldd,
          _stream(stream, dev))
    return TokenLogprobsGrad(lp, entropy, lse, dlogits)


def _teacher(teacher_tokens, teacher_logits, T, dev):
    import torch
    if teacher_tokens.dtype != torch.int64:
        raise ValueError("teacher_tokens must be int64")
    if teacher_tokens.shape != teacher_logits.shape or teacher_tokens.dim() != 2 or teacher_tokens.shape[0] != T:
        raise ValueError("teacher_tokens and teacher_logits must be T x K")
    if teacher_tokens.device != dev or teacher_logits.device != dev:
        raise ValueError("the teacher's tensors must be on the logits' device")
    _, K, ldt = _matrix(teacher_tokens, "teacher_tokens")
    ldl = _matrix(teacher_logits, "teacher_logits")[2]
    if ldt != ldl:
        raise ValueError("teacher_tokens and teacher_logits must have the same row stride")
    if K > MAX_TEACHER:
        raise ValueError(f"at most {MAX_TEACHER} teacher tokens per row")
    return K, teacher_tokens.data_ptr(), _dtype(teacher_logits), teacher_logits.data_ptr(), ldt


def distill_topk(logits, teacher_tokens, teacher_logits, *, temperature: float = 1.0, stream=None):
    """Per-row distillation loss temperature^2 * KL(P || Q): P the softmax of
    the teacher's top logits (T x K with their int64 tokens; a token outside
    0..V-1 is padding) at `temperature`, Q the student's over the vocabulary.
    Returns (loss, lse), lse that of logits / temperature (logits_distill)."""
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    code = _dtype(logits)
    teacher = _teacher(teacher_tokens, teacher_logits, T, dev)
    _, loss, lse = _outputs(T, dev, False)
    _call("logits_distill", dev.index, code, logits.data_ptr(), T, V, ld, *teacher, temperature, loss.data_ptr(),
          lse.data_ptr(), _stream(stream, dev))
    return loss, lse


def distill_topk_grad(logits, teacher_tokens, teacher_logits, weight, *, temperature: float = 1.0, dlogits=None,
                      stream=None):
    """distill_topk's loss and the gradient for the logits of
    sum(weight * loss), in one kernel (logits_distill_grad).  Returns
    (loss, dlogits); dlogits may be the logits themselves."""
    import torch
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    code = _dtype(logits)
    teacher = _teacher(teacher_tokens, teacher_logits, T, dev)
    if weight is None:
        raise ValueError("weight must be given")
    w = _vector(weight, T, torch.float32, dev, "weight")
    dlogits, ldd = _gradient(dlogits, logits)
    loss = torch.empty((T,), dtype=torch.float32, device=dev)
    _call("logits_distill_grad", dev.index, code, logits.data_ptr(), T, V, ld, *teacher, temperature, w,
          loss.data_ptr(), None, dlogits.data_ptr(), ldd, _stream(stream, dev))
    return loss, dlogits
