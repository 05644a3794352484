"""Fusion groups on one GB300: a chain of up to 64 elementwise nodes in one
loop nest, the reduction-rooted softmax region, and the AdamW step over a
parameter tree, each one CUDA launch through a C ABI (include/psk.h); and
around them the operators a training step begins and ends with: the embedding
and its gradient, dropout, the norms' backward and the clipped policy loss.

    from reduction_groups_gb300 import psk_group_run, psk_softmax_region, psk_adamw_tree
"""

from .ops import (  # noqa: F401
    psk_adamw_clip_scale,
    psk_adamw_group_sqsums,
    psk_adamw_lr,
    psk_adamw_scalars,
    psk_adamw_tree,
    psk_adamw_tree_ex,
    psk_adamw_tree_scaled,
    psk_adamw_tree_static,
    psk_adamw_workspace,
    psk_device_status,
    psk_dropout,
    psk_embed,
    psk_embed_backward,
    psk_embed_workspace,
    psk_group_check,
    psk_group_prepare,
    psk_group_run,
    psk_group_run_interp,
    psk_norm_backward,
    psk_norm_backward_workspace,
    psk_norm_region,
    psk_policy_loss,
    psk_policy_loss_workspace,
    psk_softmax_backward,
    psk_softmax_masked,
    psk_softmax_region,
    psk_test_drop_row,
    psk_test_fast_exp,
    psk_token_logp,
)
from ._native import PskError  # noqa: F401
