"""Argument checks of the logits operators and the 8-bit product on the host
(no GPU needed): the documented status before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest

import tensor_core_dense_tma_gb300 as tc
from tensor_core_dense_tma_gb300 import build as tcbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = 0x10000        # an aligned stand-in address (never dereferenced: T = 0 or a refused call)


@pytest.fixture(scope="module")
def lib():
    tcbuild.build()
    return tc.load()


def test_every_declared_symbol_is_exported(lib):
    text = "".join(open(os.path.join(ROOT, "include", n)).read() for n in ("gemm.h", "logits.h"))
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b((?:gemm|logits)_[a-z0-9_]+)\s*\(", text)))
    assert "gemm_run_i8" in names and "logits_distill_grad" in names
    out = subprocess.run(["nm", "-D", "--defined-only", tcbuild.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert not [n for n in names if n not in exported]


ROWS = dict(device=0, dtype=2, z=P, T=4, V=100, ld=100)


def rows(kw, *names):
    a = dict(ROWS)
    a.update(kw)
    return [a[k] for k in ("device", "dtype", "z", "T", "V", "ld")] + [a[n] for n in names]


BAD_ROWS = [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(z=None), INVALID), (dict(T=-1), INVALID),
    (dict(V=-1), INVALID), (dict(ld=99), INVALID), (dict(V=1 << 31, ld=1 << 31), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(ld=1 << 41), UNSUPPORTED), (dict(z=P + 2), MISALIGNED),
    (dict(temperature=0.0), INVALID), (dict(temperature=-2.0), INVALID), (dict(temperature=float("nan")), INVALID),
    (dict(temperature=float("inf")), INVALID), (dict(temperature=1e-40), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(top=-1), INVALID), (dict(top=129), INVALID), (dict(top=3, tv=None), INVALID), (dict(top=3, tt=None), INVALID),
    (dict(tokens=P + 4), MISALIGNED), (dict(lp=P + 2), MISALIGNED), (dict(ent=P + 1), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED), (dict(tt=P + 4), MISALIGNED), (dict(T=0), OK), (dict(T=0, z=None), OK),
])
def test_logprobs(lib, kw, code):
    a = dict(tokens=P, temperature=1.0, top=2, lp=P, ent=P, lse=P, tv=P, tt=P)
    a.update(kw)
    assert lib.logits_logprobs(*rows(a, "tokens", "temperature", "top", "lp", "ent", "lse", "tv", "tt"), None) == code


@pytest.mark.parametrize("kw,code", BAD_ROWS + [
    (dict(tokens=None), INVALID), (dict(dz=None), INVALID), (dict(ldd=99), INVALID), (dict(ldd=1 << 41), UNSUPPORTED),
    (dict(dz=P + 2), MISALIGNED), (dict(g=P + 2), MISALIGNED), (dict(h=P + 2), MISALIGNED), (dict(T=0), OK),
])
def test_logprobs_grad(lib, kw, code):
    a = dict(tokens=P, temperature=1.0, g=P, h=P, lp=P, ent=P, lse=P, dz=P, ldd=100)
    a.update(kw)
    if a.get("V", 0) > 100:
        a["ldd"] = a["V"]
    assert lib.logits_logprobs_grad(*rows(a, "tokens", "temperature", "g", "h", "lp", "ent", "lse", "dz", "ldd"),
                                    None) == code


BAD_TEACHER = BAD_ROWS + [
    (dict(K=-1), INVALID), (dict(K=1025, ldt=1025), INVALID), (dict(ldt=7), INVALID), (dict(td=4), INVALID),
    (dict(tt=None), INVALID), (dict(tv=None), INVALID), (dict(loss=None), INVALID), (dict(tt=P + 4), MISALIGNED),
    (dict(tv=P + 2), MISALIGNED), (dict(loss=P + 1), MISALIGNED), (dict(ldt=1 << 41), UNSUPPORTED), (dict(T=0), OK),
]


@pytest.mark.parametrize("kw,code", BAD_TEACHER)
def test_distill(lib, kw, code):
    a = dict(K=8, tt=P, td=2, tv=P, ldt=8, temperature=1.0, loss=P, lse=None)
    a.update(kw)
    assert lib.logits_distill(*rows(a, "K", "tt", "td", "tv", "ldt", "temperature", "loss", "lse"), None) == code


@pytest.mark.parametrize("kw,code", BAD_TEACHER + [
    (dict(w=None), INVALID), (dict(dz=None), INVALID), (dict(ldd=99), INVALID), (dict(dz=P + 2), MISALIGNED),
    (dict(w=P + 2), MISALIGNED),
])
def test_distill_grad(lib, kw, code):
    a = dict(K=8, tt=P, td=2, tv=P, ldt=8, temperature=1.0, w=P, loss=P, lse=None, dz=P, ldd=100)
    a.update(kw)
    if a.get("V", 0) > 100:
        a["ldd"] = a["V"]
    assert lib.logits_distill_grad(*rows(a, "K", "tt", "td", "tv", "ldt", "temperature", "w", "loss", "lse", "dz", "ldd"),
                                   None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(xt=3), INVALID), (dict(R=-1), INVALID), (dict(K=-1), INVALID), (dict(ldx=63), INVALID),
    (dict(ldq=63), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(scale=None), INVALID),
    (dict(X=P + 2), MISALIGNED), (dict(scale=P + 2), MISALIGNED), (dict(device=-1), INVALID),
    (dict(R=1 << 31), UNSUPPORTED),
])
def test_quantize_rows(lib, kw, code):
    a = dict(device=0, X=P, xt=2, R=4, K=64, ldx=64, Q=P, ldq=64, scale=P)
    a.update(kw)
    assert lib.gemm_quantize_rows_i8(*[a[k] for k in ("device", "X", "xt", "R", "K", "ldx", "Q", "ldq", "scale")],
                                     None) == code


def test_product_without_a_plan(lib):
    assert lib.gemm_run_i8(None, P, P, P, 4, 4, 64, 64, 64, 4, 2, None, None) == INVALID
    assert lib.gemm_run_i8_dynamic(None, P, 2, P, P, 4, 4, 64, 64, 64, 4, 2, None, None) == INVALID
    ep = tc.Epilogue(None, P, None, 0)
    assert lib.gemm_run_i8_dynamic(None, P, 2, P, P, 4, 4, 64, 64, 64, 4, 2, ctypes.byref(ep), None) == INVALID
