"""Operators on the rows of a logits matrix (the C ABI of ``include/logits.h``):
token log-probabilities with entropy and top alternatives, distillation from
a teacher's top logits, a clipped policy loss, a preference loss of paired
sequences, and the gradients of all four for the logits.

Like the rest of the binding, the functions check and marshal arguments; the
computation is one CUDA kernel per call (two or three for the preference loss)
on the given (or current) stream.

``logits`` is a T x V device tensor of fp32, fp16 or bf16 with unit column
stride; rows may be padded (the product that feeds on a gradient wants row
strides of whole 16 bytes, and an allocated gradient has them).  Logits should
have such rows too, or the gradient be given with the logits' stride: a gradient
row that starts elsewhere within 16 bytes than its logits is stored element by
element (2048 x 65537 bf16 282 us, with equal rows 96).

What a call returns belongs to torch's current stream; with another
``stream`` order the two, as for any tensor used on a second stream.  A result that
is not looked at may be dropped at once.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

__all__ = ["TokenLogprobs", "TokenLogprobsGrad", "token_logprobs", "token_logprobs_grad", "distill_topk",
           "distill_topk_grad", "PolicyLoss", "PolicyLossGrad", "policy_loss", "policy_loss_grad",
           "PreferenceLoss", "PreferenceLossGrad", "preference_loss", "preference_loss_grad", "MAX_TOP", "MAX_TEACHER"]

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


class PolicyLoss(NamedTuple):
    loss: object           # [T] fp32
    logprob: object        # [T] fp32
    kl: object             # [T] fp32
    entropy: object        # [T] fp32


class PolicyLossGrad(NamedTuple):
    loss: object
    logprob: object
    kl: object
    entropy: object
    dlogits: object        # [T, V] of the logits' type


class PreferenceLoss(NamedTuple):
    loss: object           # [pairs] fp32
    reward: object         # [2 pairs] fp32
    logprob: object        # [T] fp32


class PreferenceLossGrad(NamedTuple):
    loss: object
    reward: object
    logprob: object
    dlogits: object        # [T, V] of the logits' type


class _Policy(ctypes.Structure):
    """logits_policy_t."""
    _fields_ = [("old_logprob", ctypes.c_void_p), ("advantage", ctypes.c_void_p), ("ref_logprob", ctypes.c_void_p),
                ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("entropy_bonus", ctypes.c_float)]


class _Preference(ctypes.Structure):
    """logits_preference_t."""
    _fields_ = [("offsets", ctypes.c_void_p), ("pairs", ctypes.c_int64), ("ref_logprob", ctypes.c_void_p),
                ("beta", ctypes.c_float), ("smoothing", ctypes.c_float)]


def declare(lib: ctypes.CDLL) -> None:
    p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    rows = [i32, i32, p, i64, i64, i64]
    lib.logits_logprobs.argtypes = rows + [p, f32, i32, p, p, p, p, p, p]
    lib.logits_logprobs_grad.argtypes = rows + [p, f32, p, p, p, p, p, p, i64, p]
    teacher = [i64, p, i32, p, i64, f32]
    lib.logits_distill.argtypes = rows + teacher + [p, p, p]
    lib.logits_distill_grad.argtypes = rows + teacher + [p, p, p, p, i64, p]
    policy = [p, f32, ctypes.POINTER(_Policy)]
    lib.logits_policy.argtypes = rows + policy + [p, p, p, p, p]
    lib.logits_policy_grad.argtypes = rows + policy + [p, p, p, p, p, p, i64, p]
    preference = [p, f32, ctypes.POINTER(_Preference)]
    lib.logits_preference.argtypes = rows + preference + [p, p, p, p]
    lib.logits_preference_grad.argtypes = rows + preference + [p, p, p, p, p, i64, p, p]
    for f in (lib.logits_logprobs, lib.logits_logprobs_grad, lib.logits_distill, lib.logits_distill_grad,
              lib.logits_policy, lib.logits_policy_grad, lib.logits_preference, lib.logits_preference_grad):
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
    """(gradient, its row stride, the same if it was allocated here)."""
    import torch
    T, V = logits.shape
    own = None
    if dlogits is None:
        unit = 16 // logits.element_size()
        own = dlogits = torch.empty((T, -(-V // unit) * unit), dtype=logits.dtype, device=logits.device)[:, :V]
    elif dlogits.dtype != logits.dtype or dlogits.shape != logits.shape or dlogits.device != logits.device:
        raise ValueError("dlogits must have the logits' shape, type and device")
    return dlogits, _matrix(dlogits, "dlogits")[2], own


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


def _stream(stream, device, *own):
    """The stream of a call: the given or the current one.  The memory of its `own` tensors (those it
    allocated, of the current stream's; None: none) goes back there once nobody holds them, say an output that
    the caller does not look at; with a given stream, not before what is on that one now has ended."""
    import torch
    current = torch._C._cuda_getCurrentRawStream(device.index)    # current_stream() takes 2 us to make an object
    if stream is None or stream == current:
        return current
    # (torch has no stream of the handle cudaStreamLegacy, 1, which is 0's)
    other = torch.cuda.ExternalStream(0 if stream == 1 else stream, device=device)
    for t in own:
        if t is not None:
            t.record_stream(other)
    return stream


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
          top_tok.data_ptr(), _stream(stream, dev, lp, entropy, lse, top_lp, top_tok))
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
    dlogits, ldd, own = _gradient(dlogits, logits)
    lp, entropy, lse = _outputs(T, dev, tokens is not None)
    _call("logits_logprobs_grad", dev.index, code, logits.data_ptr(), T, V, ld, tok, temperature, g, h,
          lp.data_ptr() if lp is not None else None, entropy.data_ptr(), lse.data_ptr(), dlogits.data_ptr(), ldd,
          _stream(stream, dev, lp, entropy, lse, own))
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
          lse.data_ptr(), _stream(stream, dev, loss, lse))
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
    dlogits, ldd, own = _gradient(dlogits, logits)
    loss = torch.empty((T,), dtype=torch.float32, device=dev)
    _call("logits_distill_grad", dev.index, code, logits.data_ptr(), T, V, ld, *teacher, temperature, w,
          loss.data_ptr(), None, dlogits.data_ptr(), ldd, _stream(stream, dev, loss, own))
    return loss, dlogits


def _vectors(dtype, n: int, device, **vs):
    """Addresses of contiguous device vectors (None: None), looked at once each;
    what is wrong is said once something is."""
    size, di, out = (n,), device.index, []
    for what, v in vs.items():
        if v is None:
            out.append(None)
        elif v.dtype is dtype and v.shape == size and v.get_device() == di and v.is_contiguous():
            out.append(v.data_ptr())
        else:
            raise ValueError(f"{what} must be a contiguous {dtype} vector of length {n} on the logits' device")
    return out


def _policy_args(logits, tokens, old_logprob, advantage, weight, ref_logprob, clip, kl, entropy_bonus):
    """The arguments from the device to the tokens, the policy, the weights' address and the outputs."""
    import torch
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    if tokens is None or old_logprob is None or advantage is None:
        raise ValueError("tokens, old_logprob and advantage must be given")
    if kl != 0 and ref_logprob is None:
        raise ValueError("a KL term needs ref_logprob")
    low, high = clip
    tok, = _vectors(torch.int64, T, dev, tokens=tokens)
    old, adv, ref, w = _vectors(torch.float32, T, dev, old_logprob=old_logprob, advantage=advantage,
                                ref_logprob=ref_logprob, weight=weight)
    new = torch.empty_like
    out = new(old_logprob), new(old_logprob), new(old_logprob), new(old_logprob)
    return (dev.index, _dtype(logits), logits.data_ptr(), T, V, ld, tok), \
        _Policy(old, adv, ref, low, high, kl, entropy_bonus), w, out


def policy_loss(logits, tokens, old_logprob, advantage, ref_logprob=None, *, clip=(0.2, 0.2), kl: float = 0.0,
                entropy_bonus: float = 0.0, temperature: float = 1.0, stream=None) -> PolicyLoss:
    """Clipped policy loss of each row's token (int64): -min(r A, clip(r, 1 - clip[0],
    1 + clip[1]) A) + kl * KL term - entropy_bonus * entropy, with
    r = exp(logprob - old_logprob) and A the advantage (fp32 vectors).
    ref_logprob gives the KL term against a reference policy.  A row with a
    token outside 0..V-1 has zeros and is not read (logits_policy)."""
    rows, policy, _, out = _policy_args(logits, tokens, old_logprob, advantage, None, ref_logprob, clip, kl,
                                        entropy_bonus)
    loss, lp, k, ent = out
    _call("logits_policy", *rows, temperature, ctypes.byref(policy), loss.data_ptr(), lp.data_ptr(), k.data_ptr(),
          ent.data_ptr(), _stream(stream, logits.device, *out))
    return PolicyLoss(loss, lp, k, ent)


def policy_loss_grad(logits, tokens, old_logprob, advantage, weight, ref_logprob=None, *, clip=(0.2, 0.2),
                     kl: float = 0.0, entropy_bonus: float = 0.0, temperature: float = 1.0, dlogits=None,
                     stream=None) -> PolicyLossGrad:
    """policy_loss and the gradient for the logits of sum(weight * loss), in
    one kernel (logits_policy_grad).  Rows without a token or of weight 0 have
    gradients of zeros.  dlogits may be the logits themselves."""
    if weight is None:
        raise ValueError("weight must be given")
    rows, policy, w, out = _policy_args(logits, tokens, old_logprob, advantage, weight, ref_logprob, clip, kl,
                                        entropy_bonus)
    dlogits, ldd, own = _gradient(dlogits, logits)
    loss, lp, k, ent = out
    _call("logits_policy_grad", *rows, temperature, ctypes.byref(policy), w, loss.data_ptr(), lp.data_ptr(),
          k.data_ptr(), ent.data_ptr(), dlogits.data_ptr(), ldd, _stream(stream, logits.device, *out, own))
    return PolicyLossGrad(loss, lp, k, ent, dlogits)


def _preference_args(logits, tokens, offsets, weight, ref_logprob, beta, smoothing):
    """The arguments from the device to the tokens, the preference, the weights' address and the outputs."""
    import torch
    T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    if tokens is None or offsets is None:
        raise ValueError("tokens and offsets must be given")
    if offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets must have an entry for each sequence of a pair and one more")
    ends = offsets.shape[0]
    pairs = ends // 2
    f32 = torch.float32
    tok, = _vectors(torch.int64, T, dev, tokens=tokens)
    at, = _vectors(torch.int64, ends, dev, offsets=offsets)
    ref, = _vectors(f32, T, dev, ref_logprob=ref_logprob)
    w, = _vectors(f32, pairs, dev, weight=weight)
    new = torch.empty
    out = new((pairs,), dtype=f32, device=dev), new((2 * pairs,), dtype=f32, device=dev), new((T,), dtype=f32, device=dev)
    return (dev.index, _dtype(logits), logits.data_ptr(), T, V, ld, tok), _Preference(at, pairs, ref, beta, smoothing), \
        w, out


def preference_loss(logits, tokens, offsets, ref_logprob=None, *, beta: float = 0.1, smoothing: float = 0.0,
                    temperature: float = 1.0, stream=None) -> PreferenceLoss:
    """Preference loss of pairs of packed sequences: sequence s has the rows
    offsets[s] .. offsets[s + 1] - 1 (int64, on the device), 2q is the
    preferred one of pair q and 2q + 1 the other.  A sequence's reward is beta
    times the sum of logprob - ref_logprob over its rows whose token (int64) is
    in 0..V-1, the loss -(1 - smoothing) log sigma(m) - smoothing log sigma(-m)
    of the rewards' difference m (logits_preference)."""
    rows, preference, _, out = _preference_args(logits, tokens, offsets, None, ref_logprob, beta, smoothing)
    loss, reward, lp = out
    _call("logits_preference", *rows, temperature, ctypes.byref(preference), loss.data_ptr(), reward.data_ptr(),
          lp.data_ptr(), _stream(stream, logits.device, *out))
    return PreferenceLoss(loss, reward, lp)


def preference_loss_grad(logits, tokens, offsets, weight, ref_logprob=None, *, beta: float = 0.1,
                         smoothing: float = 0.0, temperature: float = 1.0, dlogits=None,
                         stream=None) -> PreferenceLossGrad:
    """preference_loss and the gradient for the logits of sum(weight * loss),
    weight one fp32 number a pair (logits_preference_grad).  Rows without a
    token or in no sequence have gradients of zeros.  dlogits may be the logits
    themselves."""
    import torch
    if weight is None:
        raise ValueError("weight must be given")
    rows, preference, w, out = _preference_args(logits, tokens, offsets, weight, ref_logprob, beta, smoothing)
    dlogits, ldd, own = _gradient(dlogits, logits)
    loss, reward, lp = out
    work = torch.empty((4 * rows[3],), dtype=torch.float32, device=logits.device)
    _call("logits_preference_grad", *rows, temperature, ctypes.byref(preference), w, loss.data_ptr(),
          reward.data_ptr(), lp.data_ptr(), dlogits.data_ptr(), ldd, work.data_ptr(),
          _stream(stream, logits.device, *out, work, own))
    return PreferenceLossGrad(loss, reward, lp, dlogits)
