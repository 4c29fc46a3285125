"""The warm-start example with clipped gradients: a bound that no gradient reaches changes nothing, bit for bit; a small one
gives finite losses of the same count."""

import math

import pytest

from virtual_noise_perturbed_gb300.build import build
from virtual_noise_perturbed_gb300.examples import warm_start

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def test_clipped_warm_start():
    small = dict(widths=(16, 32, 4), batch=64, steps=5, pop=32, generations=2)
    plain = warm_start.run(**small)
    assert warm_start.run(**small, max_norm=1e9) == plain
    losses, returns = warm_start.run(**small, max_norm=1e-3)
    assert len(losses) == 5 and len(returns) == 3 and all(math.isfinite(v) for v in losses + returns)
    assert losses[0] == plain[0][0]
