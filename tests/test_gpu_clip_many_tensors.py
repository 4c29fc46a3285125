"""AdamW's clipped step over more tensors than a launch takes: the factor reaches every one of them."""

import numpy as np
import pytest
import torch

from oracle import network as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("flat", [False, True])
def test_moments_over_many_launches(flat, bits):
    """They are bit for bit those of a step on clipped gradients."""
    g = torch.Generator().manual_seed(12)
    shapes = [(1 + i % 5, 7) for i in range(2001)]
    a = [torch.randn(s, generator=g).to(DEV) for s in shapes]
    b = [t.clone() for t in a]
    grads = [torch.randn(s, generator=g).to(DEV) for s in shapes]
    one, two = vn.AdamW(a, lr=1e-2, state_bits=bits), vn.AdamW(b, lr=1e-2, state_bits=bits)
    norm = one.step(torch.cat([t.reshape(-1) for t in grads]) if flat else grads, max_norm=0.2)
    want = ora.gradient_norm([f64(t) for t in grads])
    assert abs(float(norm) - want) <= U * (1 + 2.0 ** -10) * want
    clipped = [torch.empty_like(t) for t in grads]
    assert float(vn.clip_gradients(grads, 0.2, out=clipped)) == float(norm)
    two.step(clipped)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert all(torch.equal(p, q) for p, q in zip(one.moments(), two.moments()))
    m = one.moments()[0].double().cpu()
    if bits == 32:  # and what they are, (1 - beta1) g factor: four roundings, of the factor, the product, 1 - beta1 and theirs
        for i in range(2001):
            at = one.offsets[i]
            e = m[at:at + grads[i].numel()].numpy()
            w = (1 - one.betas[0]) * f64(grads[i]).reshape(-1) * (0.2 / want)
            assert np.all(np.abs(e - w) <= 4.1 * U * np.abs(w)), i
