"""B200-native batch-invariant token logprob + unclipped IS REINFORCE loss (sm_100a).

The compute path is the CUDA library ``libbi_isloss.so`` behind the C ABI in
``include/bi_isloss.h`` (the LM head, loss and diagnostics), ``include/bi_model.h`` (the
batch-invariant layers of the rest of the model) and ``include/bi_optim.h`` (the update); this
package only loads it and marshals tensors.
"""
from .api import (BiError, LossOutputs, check_status, d3_stats, decode_d3, debug_force_timeout_once,  # noqa: F401
                  gemm_bf16, is_loss_fwd_bwd, logprob_fwd, make_workspace, profile_enable, profile_read,
                  profile_reset, rmsnorm, workspace_bytes)
from .attention import attn_bwd, attn_fwd, qk_norm_rope, qk_norm_rope_bwd  # noqa: F401
from .optim import AdamWState, adamw_step  # noqa: F401
