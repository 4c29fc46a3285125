"""Bounded waits of the centre network's tensor-core kernels that run out, without a GPU fault.

Through the library's test hook the first CTA withholds one handover of operands (or, in the kernel of
gathered operands, the arrival that its epilogue waits for), so that a wait of 50 ms runs out. Each kernel
records the time-out, stops, frees its tensor memory and returns; the status is read and cleared on the
host, and an ordinary call right after is correct."""

import ctypes
import time

import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300 import _lib
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = ctypes.c_void_p


def ptr(t):
    return P(0 if t is None else t.data_ptr())


# rows, in, out: of the first CTA's handovers there are two or more in each kernel (128 of k to each of
# two CTAs in the first two); pairs run more than one tile each in the last size.
@pytest.mark.parametrize("kernel,rows,k,n,withhold", [
    (0, 70, 256, 200, 0), (0, 70, 256, 200, 1), (0, 70, 256, 200, 2),
    (1, 70, 512, 200, 0), (1, 70, 512, 200, 3),
    (2, 300, 512, 520, 0), (2, 300, 512, 520, 7), (2, 5000, 512, 2048, 5)])
def test_a_wait_that_runs_out_is_recorded(kernel, rows, k, n, withhold):
    build()
    lib = _lib.load()
    g = torch.Generator().manual_seed(withhold + k)
    x, w, r = (torch.randn(s, generator=g).bfloat16().to(DEV) for s in ((rows, k), (n, k), (rows, n)))
    y, z = torch.empty_like(r), torch.empty_like(r)
    stream = P(torch.cuda.current_stream().cuda_stream)
    vn.device_status()
    want = x.double() @ w.double().t()
    bound = (2 * k + 18) * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t())

    def call(at):
        assert lib.vn_testhook_linear_withhold(kernel, ptr(x), ptr(w), ptr(r), rows, k, n, ptr(y), ptr(z), at, 50.0, stream) == 0

    def right(y, z):
        full = want + r.double()
        assert bool(((z.double() - want).abs() <= bound + 2.0 ** -8 * 1.01 * want.abs()).all())
        assert bool(((y.double() - full).abs() <= bound + 2.0 ** -24 * r.double().abs() * 2 + 2.0 ** -8 * 1.01 * full.abs()).all())

    if kernel > 0:
        call(1 << 20)                                   # nothing withheld: the kernels as they are
        assert lib.vn_device_status(stream) == 0
        right(y, z)
    call(withhold)
    assert lib.vn_device_status(stream) == 7            # VN_ERR_TIMEOUT
    assert lib.vn_device_status(stream) == 0            # and cleared
    right(*vn.linear(x, w, residual=r, preact=True, check_status=True))


def test_hook_refuses_bad_arguments():
    build()
    f = _lib.load().vn_testhook_linear_withhold
    a = 0x100000

    def call(kernel=0, x=a, w=a + 0x10000, r=0, rows=8, k=128, n=8, y=a + 0x20000, z=0, at=0, ms=50.0):
        return f(kernel, P(x), P(w), P(r), rows, k, n, P(y), P(z), at, ms, P(0))
    assert call(kernel=3) == 4 and call(at=-1) == 4 and call(ms=0.0) == 4
    assert call(k=64) == 2 and call(k=132) == 2 and call(n=7) == 2 and call(rows=0) == 2
    assert call(x=0) == 1 and call(y=a + 0x20008) == 5 and call(y=a) == 4


def test_the_status_of_all_kernels_is_one_read():
    """Every kernel sets the same word: a check of the status costs about one read of a few bytes (a word
    for each of the three tensor-core kernels cost twice that)."""
    build()
    x = torch.zeros(8, device=DEV)

    def median(call):
        times = []
        for _ in range(301):
            t = time.perf_counter()
            call()
            times.append(time.perf_counter() - t)
        return sorted(times)[150]

    median(vn.device_status)
    ratio = min(median(vn.device_status) / median(x[0].item) for _ in range(5))
    assert ratio < 1.7, ratio


def terms(t):
    """An fp32 matrix as three bf16 ones that add up to it: its top 8 significant bits, the next, the last."""
    out = []
    for _ in range(3):
        top = (t.view(torch.int32) & -65536).view(torch.float32)
        out.append(top.bfloat16())
        t = t - top
    return torch.stack(out)


# In fp32 sums are taken in pieces of k: the first CTA hands over to several of them (64 of k each; on tiles six
# times as often, once for each product of terms).
@pytest.mark.parametrize("kernel,rows,k,n,withhold", [
    (4, 70, 8192, 200, 0), (4, 70, 8192, 200, 40), (4, 70, 8192, 200, 64),
    (5, 70, 2048, 200, 0), (5, 70, 2048, 200, 95), (5, 70, 8192, 200, 200),
    (6, 300, 2048, 520, 0), (6, 300, 2048, 520, 165), (6, 300, 2048, 520, 191), (6, 5000, 512, 2048, 45)])
def test_a_wait_that_runs_out_is_recorded_in_fp32(kernel, rows, k, n, withhold):
    build()
    lib = _lib.load()
    g = torch.Generator().manual_seed(withhold + k)
    x, w, r = (torch.randn(s, generator=g).to(DEV) for s in ((rows, k), (n, k), (rows, n)))
    xs, ws = (x, w) if kernel == 4 else (terms(x), terms(w))
    y, z = torch.empty_like(r), torch.empty_like(r)
    stream = P(torch.cuda.current_stream().cuda_stream)
    vn.device_status()
    want = x.double() @ w.double().t()
    bound = (2 * k + 18) * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t())

    def call(at):
        assert lib.vn_testhook_linear_withhold(kernel, ptr(xs), ptr(ws), ptr(r), rows, k, n, ptr(y), ptr(z), at, 50.0,
                                               stream) == 0

    def right(y, z):
        full = want + r.double()
        assert bool(((z.double() - want).abs() <= bound).all())
        assert bool(((y.double() - full).abs() <= bound + 2.0 ** -23 * (r.double().abs() + full.abs())).all())

    if kernel > 4:
        call(1 << 20)
        assert lib.vn_device_status(stream) == 0
        right(y, z)
    call(withhold)
    assert lib.vn_device_status(stream) == 7
    assert lib.vn_device_status(stream) == 0
    right(*vn.linear(x, w, residual=r, preact=True, check_status=True))
