"""The adapters' host-side calls (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest

import tensor_core_dense_tma_gb300 as tc
from tensor_core_dense_tma_gb300 import build as tcbuild
from tensor_core_dense_tma_gb300.adapters import Adapters, hidden_width

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000        # an aligned stand-in address (never dereferenced: a refused call)


@pytest.fixture(scope="module")
def lib():
    tcbuild.build()
    return tc.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "adapters.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text))
    assert names == {"gemm_adapters_hidden_width", "gemm_run_adapters", "gemm_adapters_grad"}
    out = subprocess.run(["nm", "-D", "--defined-only", tcbuild.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if line.strip()}


def test_hidden_width(lib):
    assert [lib.gemm_adapters_hidden_width(r) for r in (-1, 0, 1, 16, 17, 32, 33, 64, 65, 128, 129)] == \
        [0, 0, 32, 32, 64, 64, 128, 128, 256, 256, 0]
    assert all(lib.gemm_adapters_hidden_width(r) == hidden_width(r) for r in range(1, 129))


def test_without_a_plan(lib):
    a = Adapters(2, 8, P, 64, 512, 0, P, 8, 256, 0, None, P)
    run = lambda q: lib.gemm_run_adapters(None, P, P, P, 4, 32, 64, 64, 64, 32, 1, 0, None, q, P, 32, None)   # noqa: E731
    assert run(ctypes.byref(a)) == 1 and run(None) == 1
    assert lib.gemm_adapters_grad(None, P, P, 4, 32, 64, 64, 32, ctypes.byref(a), P, P, 32, 2, P, 64, 512, P, 8, 256,
                                  None) == 1
