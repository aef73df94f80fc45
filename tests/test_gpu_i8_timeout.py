"""Failure detection in the 8-bit product without a GPU fault: a bounded wait
runs out.

As for the fp16 kernel, a test build of the library lets a producer arm a
stage's barrier and then skip the loads of its tokens, so the bytes never
arrive.  The kernel records GEMM_ERR_TIMEOUT, winds down and returns; the same
plan then computes a correct product.
"""
import ctypes
import os
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 5


@pytest.fixture(scope="module")
def fi_lib():
    from tensor_core_dense_tma_gb300 import build as tb
    import tensor_core_dense_tma_gb300 as tc
    path = os.path.join(tb.OUT_DIR, "libtcdt_gemm_fi.so")
    tb.build(extra_flags=["-DTCDT_FAULT_INJECTION"], out=path)
    lib = tc.load(path)
    lib.gemm_test_inject_skip_load.argtypes = [ctypes.c_void_p, ctypes.c_int64]
    lib.gemm_test_inject_skip_load.restype = ctypes.c_int
    return lib


# one range of K a tile; ranges shared by a cluster; wide tiles; CTA pairs; a stage within the first ones and a later one
@pytest.mark.parametrize("M,N,K,stage", [(16, 20000, 2048, 1), (16, 512, 4096, 0), (60, 512, 4096, 3),
                                         (1000, 2048, 1024, 7), (1024, 4096, 4096, 9)], ids=lambda v: str(v))
def test_stalled_tokens_report_timeout_and_recover(fi_lib, M, N, K, stage):
    lib = fi_lib
    h = ctypes.c_void_p()
    assert lib.gemm_plan_create(ctypes.byref(h), 0, 0) == OK
    plan = h.value
    try:
        assert lib.gemm_plan_set_timeout_ns(plan, 20_000_000) == OK
        g = np.random.default_rng(M)
        a = g.integers(-127, 128, (M, K)).astype(np.int8)
        w = g.integers(-127, 128, (N, K)).astype(np.int8)
        A, W = torch.from_numpy(a).cuda(), torch.from_numpy(w).cuda()
        D = torch.zeros((M, N), device="cuda")

        def run():
            return lib.gemm_run_i8(plan, A.data_ptr(), W.data_ptr(), D.data_ptr(), M, N, K, K, K, N, 2, None,
                                   torch.cuda.current_stream().cuda_stream)

        assert lib.gemm_test_inject_skip_load(plan, stage) == OK
        t0 = time.monotonic()
        assert run() == OK
        torch.cuda.synchronize()
        assert time.monotonic() - t0 < 20.0
        assert lib.gemm_plan_device_status(plan, 1) == TIMEOUT
        assert lib.gemm_test_inject_skip_load(plan, -1) == OK
        assert run() == OK
        torch.cuda.synchronize()
        assert lib.gemm_plan_device_status(plan, 0) == OK
        rows = g.integers(0, N, 300)
        assert np.array_equal(D.cpu().numpy()[:, rows].astype(np.int64), a.astype(np.int64) @ w[rows].T.astype(np.int64))
    finally:
        torch.cuda.synchronize()
        assert lib.gemm_plan_destroy(plan) == OK
