"""Which kernels the linear layer's calls take, from the library's plan on the CPU: the sizes that the GPU
tests run reach every kernel that any call reaches."""

import random

import pytest

from tests.network_routes import SIZES, WIDTHS, kernels, plan
from virtual_noise_perturbed_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("backward", [False, True])
def test_the_sizes_of_the_gpu_tests_reach_every_kernel(kind, backward):
    reached = set().union(*(kernels(*s, kind, backward) for s in SIZES[kind, backward]))
    rng = random.Random(5)

    def size():
        v = int(2 ** rng.uniform(0, 15.5))
        return max(1, v - v % rng.choice((1, 1, 8, 64)))
    for _ in range(20000):
        s = size(), size(), size()
        if s[0] * s[1] * s[2] > 10 ** 12:
            continue
        missing = {k for k in kernels(*s, kind, backward, rng.random() < 0.8) if k[1] != "rows"} - reached
        assert not missing, (s, missing)


def test_plan_refusals(lib):
    f = lib.vn_testhook_linear_plan
    assert f(1, 1, 1, 2, 0, 1, 0, None) == 3
    assert f(-1, 1, 1, 0, 0, 1, 0, None) == 2
    assert f(1, 1, 1, 0, 7, 1, 0, None) == 4
    assert f(1, 1, 1, 0, 0, 1, 0, None) == 1
    assert plan(1, 64, 64, "fp32", False)[0] == 0 and plan(100, 64, 64, "fp32", False)[0] == 2


def test_the_widths_of_the_gpu_tests_are_all_widths():
    plans = [plan(*s, "bf16", True) for s in WIDTHS]
    assert [p[0] for p in plans] == [3] * len(WIDTHS) and [p[7] for p in plans] == [1] * len(WIDTHS)
    assert [p[8] for p in plans] == list(range(32, 257, 16))
    assert {plan(*s, "fp32", True)[8] for s in WIDTHS} >= set(range(64, 257, 16))


def test_every_cta_of_a_split_tile_has_a_share_of_k():
    rng = random.Random(7)
    for _ in range(20000):
        rows, n_in, n_out = (max(1, int(2 ** rng.uniform(0, 16))) for _ in range(3))
        kind, backward = rng.choice(("fp32", "bf16")), rng.random() < 0.5
        p = plan(rows, n_in, n_out, kind, backward)
        for (pair, _, split), nk in zip((p[4:7], p[7:10]), (n_out, rows) if backward else (n_in,)):
            assert pair or 1 << split <= -(-nk // 64) * (6 if kind == "fp32" else 1)
