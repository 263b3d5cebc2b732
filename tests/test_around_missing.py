"""Gradients' calls without what they need: refused by name, before anything is made."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv


@pytest.mark.parametrize("missing", ["dout", "out", "lse"])
def test_dense_attn_bwd_names_what_is_missing(missing):
    q = torch.zeros((1, 2, 4, 64))
    args = dict(dout=q, q=q, k=q, v=q, out=q, lse=torch.zeros((1, 2, 4)))
    args[missing] = None
    with pytest.raises(ValueError, match=f"^{missing} "):
        fv.dense_attn_bwd(**args)


@pytest.mark.parametrize("missing", ["dq_out", "dk_out"])
def test_qk_norm_rope_bwd_names_what_is_missing(missing):
    x = torch.zeros((1, 4, 2, 64))
    args = dict(dq_out=x.transpose(1, 2), dk_out=x.transpose(1, 2), q=x, k=x)
    args[missing] = None
    with pytest.raises(ValueError, match=f"^{missing} "):
        fv.qk_norm_rope_bwd(**args)
