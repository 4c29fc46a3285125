"""More rows than 32-bit coordinates reach, taken in slices: layer and grad_x, against plain arithmetic."""

import ctypes

import pytest
import torch

import virtual_noise_perturbed_gb300 as vn
from virtual_noise_perturbed_gb300 import _lib
from virtual_noise_perturbed_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = ctypes.c_void_p
ROWS = 2 ** 31 + 5


def test_rows_beyond_32_bits():
    build()
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(ROWS, 2, dtype=torch.bfloat16, device=DEV)
    block = torch.randn(1 << 20, 2, generator=g, device=DEV).bfloat16()
    for r in range(0, ROWS, 1 << 20):              # rows repeat every 2^20, but for a mark at the ends of slices
        x[r:r + (1 << 20)] = block[:min(1 << 20, ROWS - r)]
    marks = [0, 1, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31, ROWS - 1]
    for i, r in enumerate(marks):
        x[r] = torch.tensor([8.0 + i, -8.0 - i])
    w = torch.tensor([[0.5, -0.25]], device=DEV).bfloat16()
    b = torch.tensor([3.0], device=DEV).bfloat16()
    y = vn.linear(x, w, b, check_status=True)
    assert y.shape == (ROWS, 1)
    for r in range(0, ROWS, 1 << 26):
        p = x[r:r + (1 << 26)].float()
        want = (p[:, :1] * 0.5 - p[:, 1:] * 0.25 + 3.0).bfloat16()      # exact but for the last rounding
        assert torch.equal(y[r:r + (1 << 26)], want), r
    # grad_x = grad W of the same rows
    lib = _lib.load()
    gx = torch.empty_like(x)
    need = lib.vn_linear_backward_workspace(ROWS, 2, 1, 1, 0, 1)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    stream = P(torch.cuda.current_stream().cuda_stream)
    assert lib.vn_linear_backward(P(y.data_ptr()), P(x.data_ptr()), P(w.data_ptr()), P(0), 1, ROWS, 2, 1, 0, P(gx.data_ptr()),
                                  P(0), P(0), 1, P(ws.data_ptr()), need, stream) == 0
    vn.device_status()
    for r in range(0, ROWS, 1 << 26):
        assert torch.equal(gx[r:r + (1 << 26)], y[r:r + (1 << 26)] * w), r
    with pytest.raises(vn.VNError) as e:
        vn.linear_backward(y, x, w)
    assert e.value.status == 6
