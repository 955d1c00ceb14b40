"""B200-native bucketed gradient quantization for communication.

The hot path (error feedback, per-bucket level fit, Philox stochastic rounding, dense bit
packing, decode and worker average) runs in the CUDA library ``libgq.so`` behind the C ABI in
``include/gq.h``; ``gq`` is its Python binding and ``synth`` draws seeded synthetic gradients.

The gradients themselves can be made from activations kept in 8 bits: ``gq.gq_act_*`` (pack and
unpack, activation functions, a linear layer's weight gradient) and ``gq.gq_layer_norm_*``.
"""
from . import gq  # noqa: F401
