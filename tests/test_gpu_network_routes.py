"""Every tensor-core kernel of the linear layer and its gradients, with its whole epilogue, against the
formulas in float64 on the device. Sizes and what they reach are in network_routes.py (a CPU test holds them
to the library's plan); tolerances are those of test_gpu_network.py."""

import math

import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from tests.network_routes import SIZES, WIDTHS
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def normal(gen, shape, kind, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale + shift).to(KINDS[kind])


def generator(rows, k, n):
    return torch.Generator(device=DEV).manual_seed(rows * 7919 + k * 31 + n)


def within(got, want, bound, what):
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    error = (got.double() - want).abs()
    worst = float((error - bound).max())
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound, largest error {float(error.max()):.3e}"


def rounding(kind, y):
    return (2.0 ** -8 if kind == "bf16" else U) * y.abs() * 1.01 + 1e-37


def slack(kind, z):
    return (2.0 ** -14 if kind == "bf16" else 16 * U) * (1 + z.abs())


def gelu(z):
    return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))


def silu_slope(z):
    t = torch.sigmoid(z)
    return t * (1 + z * (1 - t))


def check_forward(rows, k, n, kind):
    g = generator(rows, k, n)
    x, w, b, r = normal(g, (rows, k), kind), normal(g, (n, k), kind, k ** -0.5), normal(g, (n,), kind), normal(g, (rows, n), kind)
    xd, wd, bd, rd = (t.double() for t in (x, w, b, r))
    wz = xd @ wd.t() + bd
    err = (2 * k + 18) * U * (xd.abs() @ wd.abs().t() + bd.abs())
    plain = vn.linear(x, w, b, check_status=True)
    within(plain, wz, err + rounding(kind, wz), "plain")
    y, z = vn.linear(x, w, b, activation="gelu", residual=r, preact=True, check_status=True)
    within(z, wz, err + rounding(kind, wz), "preact")
    wy = gelu(wz) + rd
    within(y, wy, 1.13 * err + slack(kind, wz) + 2 * U * rd.abs() + rounding(kind, wy), "y")
    again, z2 = vn.linear(x, w, b, activation="gelu", residual=r, preact=True)
    assert torch.equal(y, again) and torch.equal(z, z2)


def check_backward(rows, k, n, kind):
    g = generator(rows, k, n)
    x, w = normal(g, (rows, k), kind), normal(g, (n, k), kind, k ** -0.5)
    d, z = normal(g, (rows, n), kind), normal(g, (rows, n), kind)
    xd, wd, dd, zd = (t.double() for t in (x, w, d, z))
    ax, aw = xd.abs(), wd.abs()

    def against(grads, dz, e):
        """e: of d itself. The products take bf16 ones rounded once where there is an activation."""
        ad = dz.abs() + e
        er = e + (2.0 ** -8 * ad if kind == "bf16" and bool((e > 0).any()) else 0)
        for got, want, bound, what in (
                (grads[0], dz @ wd, (2 * n + 18) * U * (ad @ aw) + er @ aw, "grad_x"),
                (grads[1], dz.t() @ xd, (2 * rows + 18) * U * (ad.t() @ ax) + er.t() @ ax, "grad_w"),
                (grads[2], dz.sum(0), (2 * rows + 2) * U * ad.sum(0) + e.sum(0), "grad_b")):
            within(got, want, bound + rounding(kind, want), what)
    against(vn.linear_backward(d, x, w, check_status=True), dd, torch.zeros_like(dd))
    grads = vn.linear_backward(d, x, w, z, activation="silu", check_status=True)
    against(grads, dd * silu_slope(zd), dd.abs() * slack(kind, zd))
    for a, b in zip(grads, vn.linear_backward(d, x, w, z, activation="silu")):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind,backward,rows,k,n",
                         [(kind, backward, *s) for (kind, backward), sizes in SIZES.items() for s in sizes])
def test_every_kernel(kind, backward, rows, k, n):
    (check_backward if backward else check_forward)(rows, k, n, kind)


# Over several tiles a pair: in the gradient of the weight, whose operands both lie with their outputs'
# dimension contiguous, halves of a tile end anywhere within a 64-wide block.
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,k,n", WIDTHS)
def test_weight_gradients_of_every_tile_width(kind, rows, k, n):
    check_backward(rows, k, n, kind)
