"""A policy warm-started by its gradients, then improved by evolution strategies.

The policy is a layer norm of the observation and a chain of linear layers with tanh between
them. First its centre is fitted to a teacher's actions: ``layer_norm`` and ``linear`` forward,
``linear_backward`` and ``layer_norm_backward``, one ``AdamW`` over all parameters. Then the
population perturbs the chain (``virtual_perturbed_mlp``) on the normalised observations, the
returns become centered ranks, ``virtual_flat_gradient`` estimates the direction, and an
``AdamW`` that ascends takes it. The chain's weights and biases are views of one flat vector,
laid out as ``compute_offsets`` says, so both phases update the same memory.

    python -m virtual_noise_perturbed_gb300.examples.warm_start
"""

from __future__ import annotations

import argparse
from typing import List, Sequence

import torch

import virtual_noise_perturbed_gb300 as vn


class Policy:
    """layer_norm(obs), then linear layers of the given widths with tanh between them."""

    def __init__(self, widths: Sequence[int], device, generator: torch.Generator):
        shapes = []
        for n_in, n_out in zip(widths[:-1], widths[1:]):
            shapes += [(n_out, n_in), (n_out,)]
        self.offsets = vn.compute_offsets(shapes)
        blocks = [torch.randn(s, generator=generator) / s[1] ** 0.5 if len(s) == 2 else torch.zeros(s) for s in shapes]
        self.theta = torch.cat([b.reshape(-1) for b in blocks]).to(device)
        views = [self.theta[o:o + b.numel()].view(b.shape) for o, b in zip(self.offsets, blocks)]
        self.weights, self.biases = views[::2], views[1::2]
        self.gain = torch.ones(widths[0], device=device)
        self.shift = torch.zeros(widths[0], device=device)

    def parameters(self) -> List[torch.Tensor]:
        return [self.gain, self.shift] + [t for pair in zip(self.weights, self.biases) for t in pair]

    def normalised(self, obs: torch.Tensor) -> torch.Tensor:
        return vn.layer_norm(obs, self.gain, self.shift)[0]

    def __call__(self, obs: torch.Tensor) -> torch.Tensor:
        h = self.normalised(obs)
        for w, b in zip(self.weights[:-1], self.biases[:-1]):
            h = vn.linear(h, w, b, activation="tanh")
        return vn.linear(h, self.weights[-1], self.biases[-1])

    def gradients(self, obs: torch.Tensor, target: torch.Tensor):
        """(loss, gradients in ``parameters``' order): the mean squared distance to target."""
        h, mean, rstd = vn.layer_norm(obs, self.gain, self.shift)
        inputs, preacts = [], []
        for w, b in zip(self.weights[:-1], self.biases[:-1]):
            inputs.append(h)
            h, z = vn.linear(h, w, b, activation="tanh", preact=True)
            preacts.append(z)
        inputs.append(h)
        off = vn.linear(h, self.weights[-1], self.biases[-1], residual=-target)
        loss = (off * off).mean()
        grad = off * (2.0 / off.numel())
        grads: List[torch.Tensor] = []
        last = len(self.weights) - 1
        for l in range(last, -1, -1):
            act = None if l == last else "tanh"
            z = None if l == last else preacts[l]
            grad, gw, gb = vn.linear_backward(grad, inputs[l], self.weights[l], z, activation=act)
            grads = [gw, gb] + grads
        _, g_gain, g_shift = vn.layer_norm_backward(grad, obs, mean, rstd, self.gain)
        return loss, [g_gain, g_shift] + grads


def run(widths: Sequence[int] = (64, 256, 256, 8), *, batch: int = 1024, steps: int = 200, pop: int = 1024,
        generations: int = 30, sigma: float = 0.02, lr: float = 2e-3, es_lr: float = 1e-3, state_bits: int = 32,
        seed: int = 0, device="cuda"):
    """Both phases on synthetic data; returns (losses of the warm start, mean returns of the centre).

    The losses are one a step; the returns are the centre's on the episode's observations before
    the first generation and after each."""
    g = torch.Generator().manual_seed(seed)
    teacher = Policy(widths, device, g)
    policy = Policy(widths, device, g)

    optimizer = vn.AdamW(policy.parameters(), lr=lr, weight_decay=0.0, state_bits=state_bits)
    losses = []
    for _ in range(steps):
        obs = (torch.randn(batch, widths[0], generator=g) * 3 + 1).to(device)
        loss, grads = policy.gradients(obs, teacher(obs))
        optimizer.step(grads)
        losses.append(loss)

    # The episode: a few observations whose wanted actions differ from the teacher's.
    obs = (torch.randn(8, widths[0], generator=g) * 3 + 1).to(device)
    wanted = teacher(obs) + 0.3
    normalised = policy.normalised(obs)

    def centre_return():
        return -((policy(obs) - wanted) ** 2).mean()

    optimizer = vn.AdamW([policy.theta], lr=es_lr, weight_decay=0.0, state_bits=state_bits, maximize=True)
    returns = [centre_return()]
    for _ in range(generations):
        seeds = torch.randint(-2 ** 62, 2 ** 62, (pop,), generator=g).to(device)
        actions = vn.virtual_perturbed_mlp(normalised, policy.weights, policy.biases, seeds, sigma)
        fitness = vn.centered_ranks(-((actions - wanted) ** 2).mean(dim=(1, 2)))
        optimizer.step(vn.virtual_flat_gradient(fitness, seeds, policy.theta.numel(), sigma, pop))
        returns.append(centre_return())
    vn.device_status()
    return [float(v) for v in losses], [float(v) for v in returns]


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--generations", type=int, default=30)
    p.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    a = p.parse_args()
    losses, returns = run(steps=a.steps, generations=a.generations, state_bits=a.state_bits)
    print(f"warm start: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print(f"evolution:  return {returns[0]:.4f} -> {returns[-1]:.4f} in {len(returns) - 1} generations")


if __name__ == "__main__":
    main()
