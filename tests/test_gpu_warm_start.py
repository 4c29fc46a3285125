"""The warm-start example: both phases learn, its gradients are the formulas', and runs repeat."""

import numpy as np
import pytest
import torch

from oracle import network as oracle

pytestmark = pytest.mark.gpu

WIDTHS = (24, 40, 33, 5)


def _policy(device="cuda"):
    from virtual_noise_perturbed_gb300.examples.warm_start import Policy

    g = torch.Generator().manual_seed(3)
    policy = Policy(WIDTHS, device, g)
    obs = torch.randn(37, WIDTHS[0], generator=g) * 3 + 1
    target = torch.randn(37, WIDTHS[-1], generator=g)
    return policy, obs, target


def test_gradients_against_differences():
    """Along a random direction: (L(p + h d) - L(p - h d)) / 2h in float64 by the oracle's formulas.

    The difference's own error is O(h^2) of the loss's third derivative, 1e-8 at h = 1e-4 for values
    of order one. The kernels' float32 rounding: every sum has at most 64 terms of order one and four
    layers follow one another, 4 * (64 + 8) * 2^-24 = 2e-5 of the gradient's norm; a direction of unit
    length keeps that as a bound."""
    policy, obs, target = _policy()
    loss, grads = policy.gradients(obs.cuda(), target.cuda())
    params = [p.detach().cpu().numpy().astype(np.float64) for p in policy.parameters()]
    x, t = obs.numpy().astype(np.float64), target.numpy().astype(np.float64)

    def value(ps):
        c = x - x.mean(axis=1, keepdims=True)
        h = c / np.sqrt((c * c).mean(axis=1, keepdims=True) + 1e-5) * ps[0] + ps[1]
        for l in range(2, len(ps), 2):
            h = h @ ps[l].T + ps[l + 1]
            if l + 2 < len(ps):
                h = np.tanh(h)
        return ((h - t) ** 2).mean()

    got = [g.cpu().numpy().astype(np.float64) for g in grads]
    assert abs(float(loss) - value(params)) <= 1e-5 * value(params)
    norm = np.sqrt(sum((g * g).sum() for g in got))
    rng = np.random.default_rng(5)
    for _ in range(4):
        d = [rng.standard_normal(p.shape) for p in params]
        length = np.sqrt(sum((v * v).sum() for v in d))
        d = [v / length for v in d]
        h = 1e-4
        want = (value([p + h * v for p, v in zip(params, d)]) - value([p - h * v for p, v in zip(params, d)])) / (2 * h)
        assert abs(sum((g * v).sum() for g, v in zip(got, d)) - want) <= 2e-5 * norm + 1e-7


def test_forward_is_the_unperturbed_chain():
    policy, obs, _ = _policy()
    p = [v.detach().cpu().numpy().astype(np.float64) for v in policy.parameters()]
    y = policy(obs.cuda()).cpu().numpy()
    h = oracle.layer_norm(obs.numpy().astype(np.float64), p[0], p[1])[0]
    for l in range(2, len(p), 2):
        h = h @ p[l].T + p[l + 1]
        if l + 2 < len(p):
            h = np.tanh(h)
    assert np.max(np.abs(y - h)) <= 2e-5 * np.max(np.abs(h))


@pytest.mark.parametrize("state_bits", [32, 8])
def test_both_phases_learn(state_bits):
    from virtual_noise_perturbed_gb300.examples.warm_start import run

    losses, returns = run((16, 64, 64, 4), batch=256, steps=150, pop=512, generations=25, sigma=0.05, lr=5e-3,
                          es_lr=2e-3, state_bits=state_bits)
    assert losses[-1] < 0.25 * losses[0]
    assert returns[-1] > 0.5 * returns[0]  # returns are negative: the squared distance halves


def test_runs_repeat():
    from virtual_noise_perturbed_gb300.examples.warm_start import run

    kw = dict(batch=64, steps=5, pop=64, generations=3)
    assert run((16, 32, 4), **kw) == run((16, 32, 4), **kw)
