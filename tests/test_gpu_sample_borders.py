"""Drawing an index next to the borders of min-p, and how exact it is on the longest rows, against float64."""

import math

import numpy as np
import pytest
import torch

from oracle import acting as ora
import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def neighbours(at, count):
    """fp32 values around a number, in order."""
    bits = np.float32(at).view(np.int32) + np.arange(-count, count + 1, dtype=np.int32)
    return bits.view(np.float32)


@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("n", [12, 60, 200, 401, 4096])
@pytest.mark.parametrize("min_p,t,top", [(0.999, 1.0, 0.0), (0.97, 0.5, 0.0), (0.7, 1.3, 1e-3), (0.02, 1.0, 3.0), (0.999, 1.0, -0.25)])
def test_logits_next_to_where_min_p_ends(min_p, t, top, n, each):
    """Logits around top + T ln(min_p). The promised 3e-11 decides: those nearer than 4e-11 to min_p are left out."""
    if each:
        min_p = float(np.float32(min_p))
    v = neighbours(top + t * math.log(min_p), 150)
    w = np.exp((v.astype(np.float64) - np.float32(top)) / t)
    v = v[np.abs(w - min_p) > 4e-11]
    assert (np.exp((v.astype(np.float64) - np.float32(top)) / t) >= min_p).any()
    g = torch.Generator().manual_seed(n)
    rows = 40
    x = torch.full((rows, n), top - 8 * t)  # below every min_p here
    x[:, 0] = top
    take = min(n - 1, 300)
    for r in range(rows):
        x[r, 1:1 + take] = torch.from_numpy(v)[torch.randint(0, len(v), (take,), generator=g)]
    u = torch.rand(rows, generator=g)
    arg = torch.full((rows,), min_p, device=DEV) if each else min_p
    tt = torch.full((rows,), t, device=DEV) if each else t
    got = vn.sample(x.to(DEV), u.to(DEV), temperature=tt, min_p=arg).cpu().numpy()
    t64 = float(np.float32(t)) if each else t
    want = [ora.sample(x[r].double().numpy(), float(u[r]), temperature=t64, min_p=min_p)[0] for r in range(rows)]
    assert got.tolist() == want


@pytest.mark.parametrize("n", [8, 100, 500])
def test_min_p_at_an_infinite_temperature(n):
    """All finite logits weigh as much as the largest, so none is filtered."""
    x = torch.arange(float(n)).expand(5, n).clone()
    u = torch.tensor([0.0, 0.3, 0.5, 0.77, 0.999])
    for p in (0.5, 1.0):
        got = vn.sample(x.to(DEV), u.to(DEV), temperature=torch.full((5,), math.inf, device=DEV), min_p=p)
        assert got.tolist() == [int(v * n) for v in u.double().tolist()]


@pytest.mark.parametrize("n", [5000, 131071, 524288])
@pytest.mark.parametrize("tail", [-29.2, -28.9, -20.0])
def test_long_flat_tails(n, tail):
    """By float64's sums u S lies between those at the index and before it, to within n 2^-43 of the largest weight, for the rounding of
    each weight to a whole unit of 2^-42, and 3e-11 of S."""
    x = torch.full((1, n), tail)
    x[0, 0] = 0.0
    w = np.exp(x[0].double().numpy())
    c = np.cumsum(w)
    us = [1.0 - 2.0 ** -24, 1.0 - 2.0 ** -23, 1.0 - 2.0 ** -20, 0.5, 0.0]
    index, logp = vn.sample(x.to(DEV).expand(len(us), n), torch.tensor(us).to(DEV), logprobs=True)
    bound = n * 2.0 ** -43 + 3e-11 * c[-1]
    for i, u in zip(index.tolist(), us):
        assert c[i] >= u * c[-1] - bound and (i == 0 or c[i - 1] <= u * c[-1] + bound), (u, i)
    # The share's logarithm: S is known to 2.2e-6 of what it has beyond the largest, then a few roundings.
    for i, l in zip(index.tolist(), logp.tolist()):
        want = math.log(w[i] / c[-1])
        assert abs(l - want) <= 2.2e-6 * (c[-1] - 1) / c[-1] + 8 * 2.0 ** -24 * (abs(want) + abs(tail)) + 1e-12


def test_logits_further_apart_than_fp32_reaches():
    """Beyond 3.4e38 below the largest a logit is never drawn, at any temperature."""
    for n in (6, 60, 600):
        x = torch.full((3, n), -3e38)
        x[:, 2] = 3e38
        got = vn.sample(x.to(DEV), torch.tensor([0.0, 0.5, 1 - 2.0 ** -24]).to(DEV), temperature=1e38)
        assert got.tolist() == [2, 2, 2]
