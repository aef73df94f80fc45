"""The operators on logits when a copy into the ring of shared memory or another
CTA's statistics do not arrive, without a GPU fault: bounded waits run out.

A test build of the library (-DTCDT_FAULT_INJECTION, a separate .so) lets the
warp that copies arm a chunk's barrier and start no copy, or lets some of the
computing warps give up on a chunk at once while the others see it arrive, in
every CTA or in one CTA of a row.  The kernel makes up for it by plain loads, so
the results are those without the fault, bit for bit.  A CTA that keeps back its
statistics makes the rows that it shares NaN.
"""
import ctypes
import os
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

LIMIT_NS = 4_000_000
TYPES = {"f32": (torch.float32, 2), "bf16": (torch.bfloat16, 1)}


@pytest.fixture(scope="module")
def fi():
    from tensor_core_dense_tma_gb300 import build as tb
    import tensor_core_dense_tma_gb300 as tc
    path = os.path.join(tb.OUT_DIR, "libtcdt_gemm_fi.so")
    tb.build(extra_flags=["-DTCDT_FAULT_INJECTION"], out=path)
    lib = tc.load(path)
    lib.logits_test_inject.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int,
                                       ctypes.c_int]
    lib.logits_test_inject.restype = ctypes.c_int
    yield lib
    inject(lib)


def inject(lib, skip_copy=-1, late_chunk=-1, late_warps=0, silent=0, rank=-1):
    assert lib.logits_test_inject(LIMIT_NS, skip_copy, late_chunk, late_warps, silent, rank) == 0


class Case:
    """Inputs of T rows, and each operator's results on them through `lib`."""

    def __init__(self, T, V, kind, pad=3):
        self.T, self.V, self.pad = T, V, pad
        self.dtype, self.code = TYPES[kind]
        g = torch.Generator(device="cuda").manual_seed(V)
        self.z = (torch.randn((T, V + pad), generator=g, device="cuda") * 3).to(self.dtype)
        self.tok = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.g, self.h, self.w = (torch.randn(T, generator=g, device="cuda") for _ in range(3))
        self.tt = torch.randint(0, V, (T, 9), generator=g, device="cuda")
        self.tv = torch.randn((T, 9), generator=g, device="cuda")

    def run(self, lib, op):
        T, V = self.T, self.V
        f = [torch.full((T,), 7.0, device="cuda") for _ in range(3)]
        tv, ti = torch.full((T, 20), 7.0, device="cuda"), torch.full((T, 20), 7, device="cuda")
        z = self.z.clone()
        d = z if op.endswith("inplace") else torch.full_like(z, 7.0)
        rows = (0, self.code, z.data_ptr(), T, V, V + self.pad)
        s = torch.cuda.current_stream().cuda_stream
        p = [x.data_ptr() for x in f]
        if op in ("logprobs", "top"):
            st = lib.logits_logprobs(*rows, self.tok.data_ptr(), 0.9, 20 if op == "top" else 0, *p, tv.data_ptr(),
                                     ti.data_ptr(), s)
        elif op.startswith("grad"):
            st = lib.logits_logprobs_grad(*rows, self.tok.data_ptr(), 0.9, self.g.data_ptr(), self.h.data_ptr(), *p,
                                          d.data_ptr(), V + self.pad, s)
        else:
            teacher = (9, self.tt.data_ptr(), 2, self.tv.data_ptr(), 9, 0.9)
            if op == "distill":
                st = lib.logits_distill(*rows, *teacher, p[0], p[1], s)
            else:
                st = lib.logits_distill_grad(*rows, *teacher, self.w.data_ptr(), p[0], p[1], d.data_ptr(), V + self.pad, s)
        assert st == 0
        torch.cuda.synchronize()
        return [x[:, :V] if x is d else x for x in (*f, tv, ti, d)]


OPS = ["logprobs", "top", "grad", "grad_inplace", "distill", "distill_grad", "distill_grad_inplace"]
# rows split over eight CTAs; one CTA a row, more chunks than its ring; two rows a CTA
CASES = [(3, 131072, "f32"), (400, 50001, "bf16"), (9001, 8200, "bf16")]
FAULTS = [dict(skip_copy=0), dict(skip_copy=1), dict(skip_copy=3), dict(skip_copy=5), dict(skip_copy=0, rank=1),
          dict(late_chunk=0, late_warps=0x0F), dict(late_chunk=1, late_warps=0x01), dict(late_chunk=2, late_warps=0xFE),
          dict(late_chunk=1, late_warps=0xF0, rank=0), dict(late_chunk=0, late_warps=0xFF), dict(late_chunk=3, late_warps=0x55),
          dict(skip_copy=4, late_chunk=2, late_warps=0x80)]


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("T,V,kind", CASES, ids=lambda v: str(v))
@pytest.mark.parametrize("op", OPS)
def test_late_copies_are_made_up_for(fi, T, V, kind, op):
    case = Case(T, V, kind)
    inject(fi)
    want = case.run(fi, op)
    assert not any(torch.isnan(x[:, :V] if x.dim() == 2 else x).any() for x in want if x.is_floating_point())
    for fault in FAULTS:
        inject(fi, **fault)
        t0 = time.monotonic()
        got = case.run(fi, op)
        waited = time.monotonic() - t0
        assert waited < 10.0, fault
        if fault == dict(skip_copy=0):
            assert waited > LIMIT_NS * 1e-9       # a wait did run out
        assert same(got, want), fault
    inject(fi)
    assert same(case.run(fi, op), want)


@pytest.mark.parametrize("rank", [0, 1, 7])
@pytest.mark.parametrize("op", OPS)
def test_statistics_that_do_not_arrive(fi, op, rank):
    """Rows split over eight CTAs, one of which tells the others nothing."""
    T, V = 3, 131072
    case = Case(T, V, "f32")
    inject(fi)
    want = case.run(fi, op)
    inject(fi, silent=1, rank=rank)
    t0 = time.monotonic()
    *f, tv, ti, d = case.run(fi, op)
    assert LIMIT_NS * 2e-9 < time.monotonic() - t0 < 10.0
    for x in f[:2] if op.startswith("distill") else f:
        assert torch.isnan(x).all()
    if op == "top":
        assert torch.isnan(tv).all() and bool((ti == -1).all())
    if "grad" in op:
        assert torch.isnan(d).all()
    inject(fi)
    assert same(case.run(fi, op), want)
