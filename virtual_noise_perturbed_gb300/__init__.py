"""Virtual-noise evolution strategies on one GB300 (sm_103a).

The population ES step of the EvoX API page
"evox.triton_kernels.kernels.virtual_noise" -- the perturbed linear forward,
the weight / bias gradient estimates, the noise dump and the mean-abs metric --
as a C-ABI CUDA library (``libvn.so``, declared in ``include/vn.h``) with a thin
Python binding. The noise is regenerated on the fly from (seed, element index)
and never materialised. Beside it the centre network that the step perturbs, run
unperturbed and trained by its gradients: the linear layer with bias, activation and
residual, layer norm, gradient clipping and AdamW, the layer on weights in 4 bits, and
the drawing of an action from logits.
"""

from .api import (  # noqa: F401
    VNError,
    centered_ranks,
    compute_offsets,
    device_status,
    es_update,
    gradient_update,
    hash_probe,
    noise_dump,
    perturbed_linear_path,
    virtual_bias_gradient,
    virtual_flat_gradient,
    virtual_perturbed_linear,
    virtual_perturbed_mlp,
    virtual_reduce_metric,
    virtual_weight_gradient,
)
from .network import (  # noqa: F401
    AdamW,
    Weight4,
    clip_gradients,
    gradient_norm,
    layer_norm,
    layer_norm_backward,
    linear,
    linear4,
    linear_backward,
    pack4,
    sample,
)

__all__ = [
    "AdamW", "VNError", "Weight4", "centered_ranks", "clip_gradients", "compute_offsets", "device_status", "es_update", "gradient_norm", "gradient_update", "hash_probe", "layer_norm",
    "layer_norm_backward", "linear", "linear4", "linear_backward", "noise_dump", "pack4", "perturbed_linear_path", "sample",
    "virtual_bias_gradient", "virtual_flat_gradient", "virtual_perturbed_linear", "virtual_perturbed_mlp",
    "virtual_reduce_metric",
    "virtual_weight_gradient",
]
