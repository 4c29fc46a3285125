"""Layer norm's rows of odd lengths on both sides of every boundary of the kernels' choice."""

import pytest

from tests.test_gpu_network import check_norm_backward, test_layer_norm as check_norm
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n", (125, 129, 253, 259, 509, 515, 4099, 4999, 5001, 8189, 8195, 13999, 14001, 16385, 16391))
def test_lengths(n, kind):
    build()
    for rows in (1, 3, 157):
        check_norm(rows, n, kind, "fp32")
    check_norm_backward(157, n, kind, "fp32")
