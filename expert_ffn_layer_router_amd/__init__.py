"""MI355X (gfx950) Mixture-of-Experts FFN layer forward.

The layer (router top-k, regroup by expert, int4 grouped GEMM with SwiGLU,
weighted scatter-back), the grouped products of its experts (also in 8-bit
floating point) and the step that trains them run in hand-written HIP kernels
behind the C ABI of include/moe.h, moe_ops.h, moe_fp8.h and moe_optim.h; this
package is its thin Python binding.
"""

from ._lib import MoeError, load, MOE_FLAG_BAD_SLOT  # noqa: F401
from .fp8 import (fp8_gated, fp8_gated_backward, fp8_product, fp8_product_backward, fp8_workspace,  # noqa: F401
                  quantize_blocks)
from .layer import DeviceWeights, ExpertCache, HostExpert, MoeLayer, hbm_read_probe, to_device  # noqa: F401
from .optim import adamw_states, adamw_step  # noqa: F401
from .products import (expert_product, expert_product_backward, gated_product, gated_product_backward,  # noqa: F401
                       int8_gated, int8_product, product_workspace, quantize_rows)
