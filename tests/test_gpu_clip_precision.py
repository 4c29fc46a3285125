"""The gradient norm of few elements and of equal ones.

The norm is the exact one rounded once to fp32: the float32 next to it, but where the exact norm lies within 2^-34 of itself
from a border between two (sums are kept to 2^-36 there)."""

import math

import numpy as np
import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def exact(t):
    return math.sqrt(math.fsum((f64(t).reshape(-1) ** 2).tolist()))  # squares of 24 bits are exact in 64


def rounded(got, want):
    """Whether got is want's float32, or its neighbour where want is next to the border of both."""
    near = np.float32(want)
    if np.float32(got) == near:
        return True
    border = (float(near) + float(np.float32(got))) / 2
    other = np.nextafter(near, np.float32(got))
    return other == np.float32(got) and abs(want - border) <= 2.0 ** -34 * want


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 16, 31, 64, 100, 256, 1000, 5000])
def test_the_norm_of_few_elements_is_rounded_once(n, kind):
    g = torch.Generator().manual_seed(n)
    bad = []
    for i in range(60):
        x = torch.randn(n, generator=g) * 10.0 ** (i % 7 - 3)
        if i % 3 == 1:
            x *= torch.exp(2 * torch.randn(n, generator=g))
        if i % 3 == 2:
            x = x.abs() * 0 + x[0]
        x = x.to(KINDS[kind])
        got, want = float(vn.gradient_norm(x.to(DEV))), exact(x)
        if not rounded(got, want):
            bad.append((i, got, want))
    assert not bad, (len(bad), bad[:3])


@pytest.mark.parametrize("n", [100, 4096, 100_003, 3_000_001, 40_000_000])
@pytest.mark.parametrize("value", [0.1, 1.1549045, 1.6333187, 1.9999999, 1.0000001, 3e-20])
def test_the_norm_of_equal_elements_is_rounded_once(n, value):
    """Their squares round the same way, so no average over them helps."""
    x = torch.full((n,), value, device=DEV)
    v = float(x[0])
    want = math.sqrt(n * (v * v))  # v v is exact; the product and the root are good to 2^-52
    assert rounded(float(vn.gradient_norm(x)), want), (float(vn.gradient_norm(x)), want)


@pytest.mark.parametrize("n", [8, 64, 300])
def test_the_factor_takes_the_norm_before_its_rounding(n):
    """An element is off by the factor's rounding and its product's: 2 u, and 2^-34 for the sums."""
    g = torch.Generator().manual_seed(n + 1)
    for _ in range(40):
        x = torch.randn(n, generator=g)
        want = exact(x)
        out = torch.empty(n, device=DEV)
        vn.clip_gradients(x.to(DEV), 0.3 * want, out=out)
        f = np.float64(np.float32(0.3 * want / want))
        scaled = f64(x) * (0.3 * want / want)
        assert np.all(np.abs(f64(out) - scaled) <= (2 * U + 2.0 ** -33) * np.abs(scaled)), f


@pytest.mark.parametrize("bound", [0.2, 1e9])
def test_clipped_elements_are_fp32_products(bound):
    """out = type(fp32(g factor)) with the factor in fp32, in both types."""
    for kind in ("fp32", "bf16"):
        g = torch.Generator().manual_seed(2)
        x = [torch.randn(s, generator=g).to(KINDS[kind]) for s in ((40, 1000), (7,), (8195,))]
        out = [torch.empty_like(t, device=DEV) for t in x]
        vn.clip_gradients([t.to(DEV) for t in x], bound, out=out)
        norm = math.sqrt(math.fsum(exact(t) ** 2 for t in x))
        f = torch.tensor(1.0 if norm <= bound else bound / norm, dtype=torch.float32)
        for o, t in zip(out, x):
            assert torch.equal(o.cpu(), (t.float() * f).to(KINDS[kind]))




@pytest.mark.parametrize("grow", [1.9, 1.4])
def test_squares_that_grow_beyond_what_fp32_sums_hold(grow):
    """Every eight elements of a thread (4096 a CTA's turn in fp32, two eights a thread; 912 turns side by side) have larger squares than
    those before them, from 2^96 to beyond 2^127."""
    rounds = int(math.ceil(32 / math.log2(grow)))
    square = 2.0 ** 96 * grow ** np.arange(rounds)
    value = np.sqrt(square).astype(np.float32)
    per = torch.from_numpy(value).to(DEV)
    x = per.view(-1, 2).repeat_interleave(912, 0) if rounds % 2 == 0 else per[:-1].view(-1, 2).repeat_interleave(912, 0)
    x = x[:, :, None].expand(-1, 2, 2048).reshape(-1)
    used = value[:rounds // 2 * 2].astype(np.float64)
    want = math.sqrt(math.fsum((used ** 2 * (912 * 2048)).tolist()))
    assert want < 3e38
    got = float(vn.gradient_norm(x))
    assert abs(got - want) <= U * (1 + 2.0 ** -10) * want, (got, want)
