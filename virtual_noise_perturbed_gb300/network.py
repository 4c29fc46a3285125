"""The centre network: what the population step perturbs, run unperturbed and trained.

``linear`` and ``layer_norm`` with their gradients, ``gradient_norm`` and ``clip_gradients``, and ``AdamW``, the
parameter step for any gradient: these, or the population's estimate (``virtual_flat_gradient`` and the others).
For acting ``pack4`` and ``linear4``, a layer's weights in 4 bits and ``linear`` on them, and ``sample``, an
index for each row of logits.

Like the rest of the package's Python, these functions only check and marshal arguments and
call ``libvn.so`` on the current CUDA stream; all arithmetic runs in the library's kernels.
They do it in a small extension module (``csrc/vn_torch.cpp``), since a call's time on the host is
what a small layer costs. Tensors must be on a CUDA device; there is no CPU path. Inputs that
are not contiguous are copied first. Nothing here is recorded by autograd: results carry no gradient function,
and gradients come from the ``..._backward`` calls. What a call writes over (``out``, the
parameters of a step) counts as changed in place, so autograd refuses to use what it has saved of it.
"""

from __future__ import annotations

import os
import struct
from array import array
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _lib
from ._lib import load
from .api import _device, _dt, device_status

_ACTS = {None: _lib.VN_ACT_NONE, "none": _lib.VN_ACT_NONE, "tanh": _lib.VN_ACT_TANH, "relu": _lib.VN_ACT_RELU,
         "gelu": _lib.VN_ACT_GELU, "silu": _lib.VN_ACT_SILU}


_binding = None


def _native():
    """The extension module over libvn.so; raise if it is missing (no fallback exists)."""
    global _binding
    if _binding is None:
        load()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; build it with `python -m virtual_noise_perturbed_gb300.build` "
                               "(needs nvcc)")
        from . import _binding as module
        _binding = module
    return _binding


def _act(activation: Optional[str]) -> int:
    try:
        return _ACTS[activation]
    except (KeyError, TypeError):
        raise ValueError("activation must be None, 'tanh', 'relu', 'gelu' or 'silu'") from None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           activation: Optional[str] = None, residual: Optional[torch.Tensor] = None, preact: bool = False,
           out: Optional[torch.Tensor] = None,
           check_status: bool = False) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """act(x W^T + b) + residual, shape (..., out), in one epilogue (``vn_linear``); not recorded by
    autograd.

    x is (..., in), weight (out, in), residual (..., out), all float32 or all bfloat16; bias
    (out,) of either type. ``activation``: None, "tanh", "relu", "gelu" (z times the normal
    distribution function of z) or "silu". With ``preact=True`` the result is (y, z), z the
    value before the activation that ``linear_backward`` needs. Activations are good to 2^-20 (1 + |z|),
    with up to 8 float32 rows to a few roundings. An infinity in x or weight gives NaN with more than 8
    float32 rows, whose products are sums over three bfloat16 terms. ``check_status=True`` calls
    ``device_status()`` before returning (it synchronises): the tensor-core kernels bound
    their waits, and a wait that ran out leaves y unwritten."""
    y = (_binding or _native()).linear(x, weight, bias, _act(activation), residual, preact, out)
    if check_status:
        device_status(x.device)
    return y


def linear_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                    preact: Optional[torch.Tensor] = None, *, activation: Optional[str] = None, bias: bool = True,
                    check_status: bool = False) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(grad_x, grad_weight, grad_bias) of ``linear`` (``vn_linear_backward``).

    grad is the gradient of y, (..., out); preact the z that ``linear(..., preact=True)``
    returned (not needed without an activation). The gradients have their tensors' shapes and
    dtypes, grad_bias the weight's (None with ``bias=False``). The residual's gradient is
    grad. With bfloat16 and an activation, grad times the activation's slope is rounded once to bfloat16
    before the two products (grad_bias sums it unrounded). Infinities are as for ``linear``; slopes are
    good to 2^-20."""
    grads = (_binding or _native()).linear_backward(grad, x, weight, preact, _act(activation), bias)
    if check_status:
        device_status(x.device)
    return grads


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5,
               out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): each row of x (..., n) to zero mean and unit variance, times weight plus
    bias (``vn_layer_norm``). x is float32 or bfloat16 and y like it; weight and bias (n,) are of
    either type, or None. mean and rstd are float32 of x's leading shape; ``layer_norm_backward``
    takes them. Not recorded by autograd."""
    return (_binding or _native()).layer_norm(x, weight, bias, eps, out)


def layer_norm_backward(grad: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None) \
        -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(grad_x, grad_weight, grad_bias) of ``layer_norm`` from its stored mean and rstd
    (``vn_layer_norm_backward``). The last two are (n,) of weight's dtype, None without a weight."""
    return (_binding or _native()).layer_norm_backward(grad, x, mean, rstd, weight)


Gradients = Union[torch.Tensor, Sequence[torch.Tensor]]


def _listed(tensors: Gradients) -> Union[torch.Tensor, list]:
    return tensors if isinstance(tensors, (list, torch.Tensor)) else list(tensors)


def gradient_norm(grads: Gradients, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The norm over all elements of ``grads``, a tensor or a sequence of them (float32 or bfloat16, one
    dtype), as a float32 tensor of shape () (``vn_gradient_norm``): the exact norm rounded once, but for
    a last bit next to a border."""
    return (_binding or _native()).clip_gradients(_listed(grads), None, None, out)


def clip_gradients(grads: Gradients, max_norm: float, *, out: Optional[Gradients] = None) -> torch.Tensor:
    """Scale ``grads`` to a norm of at most ``max_norm``, and return the norm that they had
    (``vn_clip_gradients``): each element times the float32 max_norm / norm where norm > max_norm, a float32 product
    rounded to the gradient's dtype.

    ``grads``: a tensor or a sequence of them, contiguous, of one dtype, written over in place, or with
    ``out``, tensors like them that take the result, only read. An infinite norm makes the factor 0 (NaN where the
    gradient is infinite), a NaN makes it NaN. Nothing synchronises: the norm stays on the device."""
    if max_norm is None:
        raise TypeError("max_norm must be a number")
    return (_binding or _native()).clip_gradients(_listed(grads), max_norm, None if out is None else _listed(out), None)


class AdamW:
    """AdamW over many tensors, one launch a step (``vn_adamw``).

    ``params``: contiguous CUDA tensors of one dtype (float32 or bfloat16) on one device that share no
    memory, updated in place by ``step``. ``weight_decay``: one number, or one for each tensor.
    ``maximize=True`` ascends: the direction of a fitness gradient. ``state_bits``: 32, or 8 for
    moments held as e4m3 codes with a float32 scale for each 256 elements of a tensor.

    ``state`` holds the moments in flat tensors: "m" and "v", and with 8 bits "m_scale" and
    "v_scale" (v's codes are of its root). Tensor i's moments are the ``params[i].numel()``
    elements from ``offsets[i]`` on, a multiple of 256. To resume, pass the saved ``state`` and
    ``steps``; the tensors passed are used and updated as they are. A deep copy, and a pickled handle,
    have parameters and moments of their own."""

    BLOCK = 256

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01, *, state_bits: int = 32,
                 maximize: bool = False, state: Optional[dict] = None, step: int = 0):
        self.params = tuple(params)
        if not self.params:
            raise ValueError("at least one tensor is needed")
        self._params = list(self.params)
        self._check_params()
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        n = len(self.params)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        if len(decay) != n:
            raise ValueError("one weight_decay for each tensor")
        self.lr, self.betas, self.eps, self.maximize = float(lr), (float(betas[0]), float(betas[1])), float(eps), bool(maximize)
        self.state_bits, self.steps = state_bits, int(step)
        self.sizes = [p.numel() for p in self.params]
        self.offsets, total = [], 0
        for s in self.sizes:
            self.offsets.append(total)
            total += -(-s // self.BLOCK) * self.BLOCK
        self._decay, self._total = decay, total
        self._tensors = self._state(total, state)
        self._lay_out()

    def _lay_out(self) -> None:
        """The table that the library reads: one row of eight words a tensor, as its struct has them:
        param, grad, both moments, their scales, the number of elements, the decay."""
        n = len(self.params)
        self._refuse_overlaps()
        self._table = t = array("Q", bytes(64 * n))
        held = self._tensors
        m, v, size = held["m"].data_ptr(), held["v"].data_ptr(), self.state_bits // 8
        t[2::8] = array("Q", [m + o * size for o in self.offsets])
        t[3::8] = array("Q", [v + o * size for o in self.offsets])
        if self.state_bits == 8:
            m, v = held["m_scale"].data_ptr(), held["v_scale"].data_ptr()
            t[4::8] = array("Q", [m + o // self.BLOCK * 4 for o in self.offsets])
            t[5::8] = array("Q", [v + o // self.BLOCK * 4 for o in self.offsets])
        t[6::8] = array("Q", self.sizes)
        t[7::8] = array("Q", struct.pack(f"{n}d", *self._decay))
        self._address = t.buffer_info()[0]

    def _refuse_overlaps(self) -> None:
        # Blocks of all tensors are updated at once: memory that two of them shared would hold either's result.
        named = [(f"params[{i}]", p) for i, p in enumerate(self.params)] + [(f"state['{k}']", t) for k, t in self._tensors.items()]
        end, last = 0, ""
        for start, size, name in sorted((t.data_ptr(), t.numel() * t.element_size(), name) for name, t in named):
            if size and start < end:
                raise ValueError(f"{last} and {name} share memory")
            if size:
                end, last = start + size, name

    def __getstate__(self) -> dict:
        kept = dict(self.__dict__)
        del kept["_table"], kept["_address"]
        # Codes travel as bytes: plain pickle does not know torch's 8-bit types.
        kept["_tensors"] = {k: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for k, t in self._tensors.items()}
        return kept

    def __setstate__(self, kept: dict) -> None:
        # A copy has tensors, and so addresses, of its own.
        self.__dict__.update(kept)
        self._tensors = {k: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for k, t in kept["_tensors"].items()}
        self._check_params()
        self._state(self._total, self._tensors)
        self._lay_out()

    def _check_params(self) -> None:
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor) or not p.is_cuda or not p.is_contiguous():
                raise ValueError(f"params[{i}] must be a contiguous CUDA tensor (updated in place)")
            if p.dtype != self.params[0].dtype:
                raise TypeError("the parameters must have one dtype")
        self.device = _device(*self.params)
        _dt(self.params[0], "params[0]")

    def _state(self, total: int, given: Optional[dict]) -> dict:
        kind = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        want = {"m": (total, kind), "v": (total, kind)}
        if self.state_bits == 8:
            want.update(m_scale=(total // self.BLOCK, torch.float32), v_scale=(total // self.BLOCK, torch.float32))
        if given is None:
            return {k: torch.zeros(size, dtype=torch.uint8 if d == torch.float8_e4m3fn else d, device=self.device).view(d)
                    for k, (size, d) in want.items()}
        if set(given) != set(want):
            raise ValueError(f"state must have {sorted(want)}, got {sorted(given)}")
        for k, (size, d) in want.items():
            t = given[k]
            if not isinstance(t, torch.Tensor) or t.shape != (size,) or t.dtype != d or t.device != self.device \
                    or not t.is_contiguous():
                raise ValueError(f"state['{k}'] must be a contiguous {d} tensor of shape ({size},) on {self.device}")
        return dict(given)

    @property
    def state(self) -> dict:
        """The moments' tensors (a new dict of them: their addresses are the handle's)."""
        return dict(self._tensors)

    def step(self, grads: Gradients, lr: Optional[float] = None, *, max_norm: Optional[float] = None) -> Optional[torch.Tensor]:
        """One step of every tensor. ``grads``: a gradient for each tensor, or one flat tensor with
        all of them one after another (as ``virtual_flat_gradient`` lays them out); float32 or
        bfloat16. ``lr`` replaces the learning rate for this step. A step cannot be captured in a graph
        (RuntimeError): replays would repeat the step number and learning rate of the capture.

        With ``max_norm`` the step takes the gradients scaled to a norm of at most that, as
        ``clip_gradients`` would leave them but in float32 (``vn_adamw_clipped``; the gradients themselves stay
        as they are), and returns the norm that they had, a float32 tensor of shape ()."""
        norm = (_binding or _native()).adamw(self._params, _listed(grads), self._address, self.state_bits,
                                             self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps,
                                             self.steps + 1, self.maximize, max_norm)
        self.steps += 1
        return norm

    def moments(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """The moments (m, v) as flat float32 tensors in ``offsets``' layout: the state itself with
        32 bits, with 8 the values that the codes stand for (``vn_adamw_moments``)."""
        s = self._tensors
        if self.state_bits == 32:
            return s["m"], s["v"]
        return (_binding or _native()).adamw_moments(s["m"], s["v"], s["m_scale"], s["v_scale"])


class Weight4:
    """A layer's weights in 4 bits with a scale for each ``group`` consecutive elements of a row, as ``pack4`` makes
    them and ``linear4`` takes them: ``codes`` (uint8, (out, bytes); their order is the library's own), ``scales`` of the weights'
    dtype, (out, ceil(in / group)), ``shape`` (out, in) and ``group``. A saved handle is made again from those four."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, in_features: int, group: int):
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        self.codes, self.scales, self.group = codes, scales, int(group)
        self.shape = torch.Size((codes.shape[0], int(in_features)))

    def dequantize(self, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The weights that the codes stand for, code times scale, each rounded once to the scales' dtype
        (``vn_unpack_weight``)."""
        return (_binding or _native()).unpack_weight(self.codes, self.scales, self.shape[1], self.group, out)


def pack4(weight: torch.Tensor, *, group: int = 64) -> Weight4:
    """``weight`` (out, in), float32 or bfloat16, in 4 bits (``vn_pack_weight``): of each ``group`` (32, 64 or 128) consecutive
    elements of a row the scale is their largest magnitude over 7, and a code the whole number of -7 .. 7 next to
    an element over it."""
    codes, scales = (_binding or _native()).pack_weight(weight, group)
    return Weight4(codes, scales, weight.shape[1], group)


def linear4(x: torch.Tensor, weight: Weight4, bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = None,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            check_status: bool = False) -> torch.Tensor:
    """``linear`` on packed weights, act(x V^T + b) + residual with V code times scale (``vn_linear_packed``): a layer
    that acts on few rows and is bound by reading its weights reads a quarter of them.

    x is (..., in) of the scales' dtype, the rest as for ``linear``. With more than 32 rows (float32: 10) V is
    unpacked first, and ``linear``'s kernels run; V is not rounded in bfloat16 (two terms each), and once in float32. An infinity in x gives NaN in float32.
    Not recorded by autograd. ``check_status`` as for ``linear``."""
    y = (_binding or _native()).linear_packed(x, weight.codes, weight.scales, weight.shape[1], weight.group, bias, _act(activation),
                                              residual, out)
    if check_status:
        device_status(x.device)
    return y


PerRow = Union[float, torch.Tensor, None]


def sample(logits: torch.Tensor, uniforms: torch.Tensor, *, temperature: PerRow = 1.0, top_k: Union[int, torch.Tensor, None] = None,
           top_p: PerRow = None, min_p: PerRow = None, logprobs: bool = False,
           out: Optional[torch.Tensor] = None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """An index for each row of ``logits`` (..., n), drawn with that row's random number of [0, 1) in
    ``uniforms`` (...), as int64 (...) (``vn_sample``): actions from a policy's logits.

    The weights are exp(logits / temperature). ``top_k`` keeps the k largest logits (of equal ones those with the lower
    index), ``top_p`` of those the largest ones until their sum reaches that share, ``min_p`` those whose weight is at
    least that share of the largest's. The index is the first at which the sum of the kept weights passes
    ``uniforms`` times the whole: float64's index, but where sums next to a border are closer than 3e-11 of the whole and
    n 2^-43 of the largest weight. Each parameter is a number, None (no filter) or a
    tensor of the leading shape (float32, ``top_k`` int64). A temperature of 0 takes the largest logit. With ``logprobs=True`` the result is
    (index, log of the kept weights' share that it has), the latter float32.

    logits are float32 or bfloat16, n up to 524,288. A row with a NaN, or with nothing above -infinity, gets
    the index -1 (and a NaN)."""
    return (_binding or _native()).sample(logits, uniforms, temperature, top_k, top_p, min_p, logprobs, out)


__all__ = ["AdamW", "Weight4", "clip_gradients", "gradient_norm", "layer_norm", "layer_norm_backward", "linear", "linear4",
           "linear_backward", "pack4", "sample"]
