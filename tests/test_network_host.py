"""The centre network's entry points without a GPU: refusals before any launch, workspaces, and the
float64 oracle against independent forms."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import network as ora
from virtual_noise_perturbed_gb300 import _lib, build

P = ctypes.c_void_p
F = 0x100000          # never dereferenced: every call below returns from the host's checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_linear_refusals(lib):
    def call(x=F, w=F + 0x1000, dt=0, b=0, bdt=0, r=0, rows=4, k=8, n=8, act=0, y=F + 0x2000, z=0, ws=0, wb=0):
        return lib.vn_linear(P(x), P(w), dt, P(b), bdt, P(r), rows, k, n, act, P(y), P(z), P(ws), wb, P(0))
    assert call(dt=2) == 3
    assert call(b=F + 0x4000, bdt=9) == 3
    assert call(act=5) == 4
    assert call(act=-1) == 4
    assert call(rows=-1) == 2
    assert call(rows=1 << 40, n=1 << 40) == 6
    assert call(x=0) == 1 and call(w=0) == 1 and call(y=0) == 1
    assert call(x=F + 2) == 5 and call(y=F + 0x2001) == 5 and call(r=F + 0x3002) == 5 and call(z=F + 0x3001) == 5
    assert call(ws=F + 0x8001) == 5
    assert call(y=F + 64) == 4                        # y over x
    assert call(z=F + 0x2000) == 4                    # preact over y
    assert call(r=F + 0x2000) == 4                    # residual over y
    assert call(rows=0, x=0, y=0) == 0 and call(n=0, w=0, y=0) == 0


def test_linear_backward_refusals(lib):
    def call(g=F, x=F + 0x1000, w=F + 0x2000, z=0, dt=0, rows=4, k=8, n=8, act=0, gx=F + 0x3000, gw=F + 0x4000,
             gb=F + 0x5000, gdt=0, ws=F + 0x10000, wb=1 << 20):
        return lib.vn_linear_backward(P(g), P(x), P(w), P(z), dt, rows, k, n, act, P(gx), P(gw), P(gb), gdt, P(ws), wb, P(0))
    assert call(dt=7) == 3 and call(gdt=7) == 3
    assert call(act=9) == 4
    assert call(k=-1) == 2
    assert call(k=1 << 40, n=1 << 40) == 6
    assert call(g=0) == 1 and call(x=0) == 1 and call(w=0) == 1
    assert call(act=1) == 1                           # an activation's gradient needs preact
    assert call(gx=F + 0x3002) == 5
    assert call(wb=0) == 11 and call(ws=0) == 11      # VN_ERR_WORKSPACE
    assert call(gx=F) == 4 and call(gw=F + 0x1000) == 4 and call(gb=F + 0x4000) == 4
    assert call(ws=F + 0x1000 - 0x1000) == 4          # the workspace over grad
    assert call(gx=0, gw=0, gb=0) == 0
    assert lib.vn_linear_backward_workspace(-1, 4, 4, 0, 0, 1) == -1
    assert lib.vn_linear_backward_workspace(4, 4, 4, 3, 0, 1) == -1
    assert lib.vn_linear_backward_workspace(4, 4, 4, 0, 8, 1) == -1
    assert lib.vn_linear_workspace(4, 1 << 40, 1 << 40, 0, 1) == -1


def test_layer_norm_refusals(lib):
    def call(x=F, dt=0, w=F + 0x1000, b=F + 0x1100, wdt=0, rows=4, n=8, eps=1e-5, y=F + 0x2000, m=F + 0x3000, r=F + 0x3100):
        return lib.vn_layer_norm(P(x), dt, P(w), P(b), wdt, rows, n, eps, P(y), P(m), P(r), P(0))
    assert call(dt=5) == 3 and call(wdt=5) == 3
    assert call(eps=-1e-5) == 4 and call(eps=float("inf")) == 4 and call(eps=float("nan")) == 4
    assert call(rows=-1) == 2 and call(n=0) == 2
    assert call(rows=1 << 40, n=1 << 40) == 6
    assert call(x=0) == 1 and call(y=0) == 1
    assert call(x=F + 2) == 5 and call(m=F + 0x3001) == 5
    assert call(y=F) == 4 and call(r=F + 0x3004) == 4 and call(m=F + 0x1100) == 4
    assert call(rows=0, x=0, y=0) == 0

    def back(g=F, x=F + 0x1000, dt=0, m=F + 0x2000, r=F + 0x2100, w=F + 0x2200, wdt=0, rows=4, n=8, gx=F + 0x3000,
             gw=F + 0x4000, gb=F + 0x4100, ws=F + 0x10000, wb=1 << 16):
        return lib.vn_layer_norm_backward(P(g), P(x), dt, P(m), P(r), P(w), wdt, rows, n, P(gx), P(gw), P(gb), P(ws), wb, P(0))
    assert back(dt=5) == 3 and back(wdt=5) == 3
    assert back(n=0) == 2 and back(rows=-1) == 2
    assert back(g=0) == 1 and back(m=0) == 1 and back(gx=0) == 1
    assert back(gw=F + 0x4002) == 5
    assert back(ws=0) == 11 and back(wb=8) == 11
    assert back(gx=F + 0x1000) == 4 and back(gb=F + 0x4000) == 4
    assert back(rows=0, gw=0, gb=0, g=0, x=0, gx=0) == 0
    assert lib.vn_layer_norm_backward_workspace(4, 0) == -1


class Tensor(ctypes.Structure):
    _fields_ = [("p", P), ("g", P), ("m", P), ("v", P), ("ms", P), ("vs", P), ("n", ctypes.c_int64), ("wd", ctypes.c_double)]


def test_adamw_refusals(lib):
    assert ctypes.sizeof(Tensor) == 64

    def call(n=8, bits=32, pdt=0, gdt=0, lr=0.1, b1=0.9, b2=0.99, eps=1e-8, step=1, count=1, **k):
        t = dict(p=F, g=F + 0x1000, m=F + 0x2000, v=F + 0x3000, ms=F + 0x4000, vs=F + 0x5000, wd=0.0)
        t.update(k)
        arr = (Tensor * 1)(Tensor(t["p"], t["g"], t["m"], t["v"], t["ms"], t["vs"], n, t["wd"]))
        return lib.vn_adamw(ctypes.cast(arr, P), count, pdt, gdt, bits, lr, b1, b2, eps, step, 0, P(0))
    assert call(pdt=4) == 3 and call(gdt=4) == 3
    assert call(bits=16) == 4
    assert call(lr=float("nan")) == 4 and call(b1=1.0) == 4 and call(b2=-0.1) == 4 and call(eps=-1.0) == 4 and call(step=0) == 4
    assert call(wd=float("inf")) == 4
    assert call(n=-1) == 2 and call(count=-1) == 2
    assert call(n=1 << 60) == 6
    assert call(p=0) == 1 and call(g=0) == 1 and call(v=0) == 1 and call(bits=8, ms=0) == 1
    assert call(p=F + 2) == 5 and call(m=F + 0x2002) == 5 and call(bits=8, vs=F + 0x5002) == 5
    assert call(g=F) == 4 and call(m=F + 0x3000) == 4
    assert call(n=0, p=0, g=0) == 0 and call(count=0) == 0
    mo = lib.vn_adamw_moments
    assert mo(P(F), P(F + 64), P(F + 128), P(F + 256), -1, P(F + 512), P(F + 1024), P(0)) == 2
    assert mo(P(0), P(F + 64), P(F + 128), P(F + 256), 8, P(F + 512), P(F + 1024), P(0)) == 1
    assert mo(P(F), P(F + 64), P(F + 128), P(F + 256), 8, P(F + 514), P(F + 1024), P(0)) == 5
    assert mo(P(F), P(F + 64), P(F + 128), P(F + 256), 8, P(F), P(F + 1024), P(0)) == 4
    assert mo(P(0), P(0), P(0), P(0), 0, P(0), P(0), P(0)) == 0


def test_python_has_no_cpu_path():
    import virtual_noise_perturbed_gb300 as vn
    x, w = torch.ones(3, 8), torch.ones(4, 8)
    for call in (lambda: vn.linear(x, w), lambda: vn.linear_backward(x, x, w), lambda: vn.layer_norm(x),
                 lambda: vn.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: vn.AdamW([x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("act", ["none", "tanh", "relu", "gelu", "silu"])
def test_oracle_linear_against_autograd(act):
    """The oracle's forward and gradients against torch's float64 autograd of torch's own activations."""
    g = torch.Generator().manual_seed(1)
    x, w, b, c = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((9, 7), (5, 7), (5,), (9, 5)))
    for t in (x, w, b):
        t.requires_grad_()
    z = x @ w.t() + b
    f = {"none": lambda t: t, "tanh": torch.tanh, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "silu": torch.nn.functional.silu}[act]
    y = f(z)
    (y * c).sum().backward()
    xn, wn, bn = (t.detach().numpy() for t in (x, w, b))
    oy, oz = ora.linear(xn, wn, bn, act)
    gx, gw, gb, _ = ora.linear_backward(c.numpy(), xn, wn, oz, act)
    for got, want in ((oy, y), (gx, x.grad), (gw, w.grad), (gb, b.grad)):
        assert np.allclose(got, want.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_oracle_layer_norm_against_autograd():
    g = torch.Generator().manual_seed(2)
    x, w, b, c = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((9, 7), (7,), (7,), (9, 7)))
    for t in (x, w, b):
        t.requires_grad_()
    y = torch.nn.functional.layer_norm(x, (7,), w, b, 1e-5)
    (y * c).sum().backward()
    xn, wn, bn = (t.detach().numpy() for t in (x, w, b))
    oy, mean, rstd = ora.layer_norm(xn, wn, bn, 1e-5)
    gx, gw, gb = ora.layer_norm_backward(c.numpy(), xn, mean, rstd, wn)
    for got, want in ((oy, y), (gx, x.grad), (gw, w.grad), (gb, b.grad)):
        assert np.allclose(got, want.detach().numpy(), rtol=1e-11, atol=1e-12)


def test_oracle_adamw_against_torch():
    g = torch.Generator().manual_seed(3)
    p = torch.nn.Parameter(torch.randn(50, generator=g, dtype=torch.float64))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1, maximize=True)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in (1, 2, 3):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        opt.step()
        q, m, v = ora.adamw(q, p.grad.numpy(), m, v, lr=0.01, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.1, step=step,
                            maximize=True)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12)


def test_oracle_e4m3_against_torch():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.exp(np.linspace(-9, 6.1, 3000)), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    want = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ora.e4m3(x.astype(np.float32).astype(np.float64)), want)
    q, s = ora.pack(np.array([0.0, 1.0, 1e-9, -1.0]), root=True)
    assert q[0] == 0 and q[1] == 448 and q[2] == 2.0 ** -9 and math.isclose(s[0], 1 / 448)


def test_workspaces_cover_what_the_calls_lay_out(lib):
    """Sizes on both sides of each route: a converted matrix is whole rows of a multiple of 8 elements,
    bf16 as one plane, fp32 as three."""
    w = lib.vn_linear_workspace
    assert w(1021, 256, 256, 0, 1) == 0                                  # gathered
    assert w(8192, 4096, 4096, 1, 1) == 0                                # taken as it is
    assert w(8192, 4097, 4096, 1, 1) >= 2 * 4104 * (8192 + 4096)         # rows padded
    assert w(8192, 4096, 4096, 1, 0) >= 2 * 4096 * (8192 + 4096)         # not aligned
    assert w(8192, 1000, 4096, 0, 1) >= 6 * 1000 * (8192 + 4096)         # three planes
    b = lib.vn_linear_backward_workspace
    assert b(8192, 4096, 4096, 1, 0, 1) < 2 * 8192 * 4096                # only the bias's sums
    assert b(8192, 4096, 4096, 1, 3, 1) >= 2 * 8192 * 4096               # and d
    assert b(8192, 1000, 4096, 0, 3, 1) >= 6 * (8192 * 4096 + 1000 * (8192 + 4096))
    assert b(100, 0, 8, 0, 0, 1) > 0 and b(0, 8, 8, 0, 0, 1) > 0
