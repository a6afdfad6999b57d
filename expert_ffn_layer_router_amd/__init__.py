"""MI355X (gfx950) Mixture-of-Experts FFN layer forward.

The layer (router top-k, regroup by expert, int4 grouped GEMM with SwiGLU,
weighted scatter-back) and the grouped products of its experts run in
hand-written HIP kernels behind the C ABI of
include/moe.h and include/moe_ops.h; this package is its thin Python binding.
"""

from ._lib import MoeError, load, MOE_FLAG_BAD_SLOT  # noqa: F401
from .layer import DeviceWeights, ExpertCache, HostExpert, MoeLayer, hbm_read_probe, to_device  # noqa: F401
from .products import (expert_product, expert_product_backward, gated_product, gated_product_backward,  # noqa: F401
                       int8_gated, int8_product, product_workspace, quantize_rows)
