"""MI355X-native PowerSGD gradient compression (the data-parallel hot path of DALL·E training).

The PowerSGD step runs in hand-written gfx950 HIP kernels inside libpsgd.so (C ABI:
include/psgd.h). This package is the thin Python binding over it:
  * binding  - ctypes wrappers with the ABI's names (psgd_create, psgd_compress, ...);
  * group    - convenience holders: one group of gradient matrices and their state, and a group
               of updates orthogonalised by Newton-Schulz products;
  * lowbit   - AdamW over a list of tensors, microscaled 4-bit matrices and a linear layer on them.
"""
from .binding import (  # noqa: F401
    LIB_PATH, PROFILE_SLOTS, PSGD_BF16, PSGD_F16, PSGD_F32, PSGD_NEAREST, PSGD_NS_ACCURATE, PSGD_NS_FAST, PSGD_STATE_BYTE, PSGD_STATE_F32,
    PSGD_STOCHASTIC, PsgdError, load_library,
    make_adam_matrix, make_adam_tensor, make_adamw_tensor, make_matrix, make_muon_matrix, make_ns_matrix, muon_hparams, ns_hparams, psgd_adam_attach, psgd_adam_prepare,
    psgd_adam_hparams, psgd_adam_update, psgd_adamw_moments, psgd_adamw_plan_create, psgd_adamw_plan_destroy, psgd_adamw_prepare,
    psgd_adamw_update, psgd_decompress_adam, psgd_block_grad_enter, psgd_block_grad_exit, psgd_block_grad_exit_enter,
    psgd_check_finite, psgd_compress, psgd_compress_p, psgd_compress_q,
    psgd_create, psgd_debug_buffer, psgd_decompress_update, psgd_destroy, psgd_embed_grad,
    psgd_embed_grad_workspace, psgd_embed_lookup, psgd_factor_buffer,
    psgd_last_error, psgd_mx_bytes, psgd_mx_dequantize, psgd_mx_product, psgd_mx_product_workspace, psgd_mx_quantize, psgd_muon_attach, psgd_muon_update, psgd_newton_schulz, psgd_ns_plan_create,
    psgd_ns_plan_destroy, psgd_orthogonalize, psgd_plan_counters, psgd_plan_create, psgd_plan_destroy,
    psgd_profile_events, psgd_refresh_q, psgd_reset_errors, psgd_step_noalloc, psgd_version,
)
from .group import NewtonSchulzGroup, PowerSGDGroup  # noqa: F401
from .lowbit import AdamWGroup, MxLinear, MxTensor  # noqa: F401
