"""Waits of the adapters' kernels that run out, without a fault: the
fault-injection build (see test_gpu_timeout.py) arms a barrier of each kernel's
pipeline for copies that it then does not start.  Each kernel records
GEMM_ERR_TIMEOUT, winds down and returns; the plan then computes as before."""
import ctypes
import time

import pytest
import torch

from tensor_core_dense_tma_gb300.adapters import Adapters, declare, hidden_width
from test_gpu_timeout import OK, TIMEOUT, fi_lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,up_col,skip", [(16, 0, 3), (300, 0, 1), (300, 1, 0), (40, 1, 2), (2000, 0, 0)])
def test_forward(fi_lib, M, up_col, skip):      # noqa: F811
    lib = fi_lib
    declare(lib)
    N, K, R, G = 520, 1040, 16, 3
    g = torch.Generator(device="cuda").manual_seed(M)
    z = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").half()      # noqa: E731
    X, W, down, up = z(M, K), z(N, K), z(G, R, K), z(G, N, R)
    if up_col:      # both factors the other way round: h from the tile kernel for any number of rows
        down, up = down.transpose(1, 2).contiguous(), up.transpose(1, 2).contiguous()
    index = (torch.arange(M, device="cuda") % (G + 1) - 1).int()
    hidden = torch.zeros((M, hidden_width(R)), dtype=torch.float16, device="cuda")
    D = torch.zeros((M, N), device="cuda")
    a = Adapters(G, R, down.data_ptr(), down.stride(1), down.stride(0), up_col, up.data_ptr(), up.stride(1), up.stride(0),
                 up_col, None, index.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    d_down, d_up = torch.zeros((G, R, K), device="cuda"), torch.zeros((G, N, R), device="cuda")

    def forward():
        return lib.gemm_run_adapters(plan, X.data_ptr(), W.data_ptr(), D.data_ptr(), M, N, K, K, K, N, 1, 2, None,
                                     ctypes.byref(a), hidden.data_ptr(), hidden.stride(0), stream)

    def backward():
        return lib.gemm_adapters_grad(plan, X.data_ptr(), X.data_ptr(), M, K, K, K, K, ctypes.byref(a),
                                      hidden.data_ptr(), hidden.data_ptr(), hidden.stride(0), 2, d_down.data_ptr(), K,
                                      R * K, None, R, R, stream)

    h = ctypes.c_void_p()
    assert lib.gemm_plan_create(ctypes.byref(h), 0, 0) == OK
    plan = h.value
    try:
        assert lib.gemm_plan_set_timeout_ns(plan, 20_000_000) == OK
        for call in (forward, backward):
            assert call() == OK
            torch.cuda.synchronize()
            assert lib.gemm_plan_device_status(plan, 0) == OK
            want = [t.clone() for t in (D, hidden, d_down)]
            for at in (0, skip):
                assert lib.gemm_test_inject_skip_load(plan, at) == OK
                t0 = time.monotonic()
                assert call() == OK
                torch.cuda.synchronize()
                assert time.monotonic() - t0 < 10.0
                status = lib.gemm_plan_device_status(plan, 1)
                # (a CTA of the backward pass may have fewer steps than `at`)
                assert status == TIMEOUT or (call is backward and at > 0)
            assert lib.gemm_test_inject_skip_load(plan, -1) == OK
            assert call() == OK
            torch.cuda.synchronize()
            assert lib.gemm_plan_device_status(plan, 0) == OK
            assert all(torch.equal(x, y) for x, y in zip((D, hidden, d_down), want))
    finally:
        lib.gemm_plan_destroy(plan)
