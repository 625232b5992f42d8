"""The norm's backward takes a checkpoint, it makes none (no GPU)."""
import pytest
import torch


def test_backward_ckpt_is_given():
    import __graft_entry__
    __graft_entry__.build()
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    dy, rstd = torch.zeros(4, 128, dtype=torch.bfloat16), torch.ones(4)
    # True asks moe_layer_norm to make one; here it would be read before anything wrote it
    for ckpt in (True, False):
        with pytest.raises(TypeError):
            L.moe_layer_norm_backward(dy, rstd, ckpt=ckpt)
    with pytest.raises(ValueError):
        L.moe_layer_norm_backward(dy, rstd)
    with pytest.raises(ValueError):
        L.moe_layer_norm_backward(dy, rstd, x=dy, ckpt=(dy, rstd))
