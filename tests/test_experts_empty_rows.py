"""Weights and rows of no columns are refused like any other wrong size (CPU: no call gets as far as a GPU)."""
import pytest
import torch

import combine_moe_route_meta_gb300 as moe


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("mode", ["normal", "masked"])
def test_no_columns(mode, swiglu):
    u8 = dict(dtype=torch.uint8)
    args = [mode, torch.zeros((2, 4, 0), **u8), torch.zeros(0, **u8), torch.zeros(2, dtype=torch.int32),
            torch.zeros((2, 32, 0), **u8), torch.zeros(0, **u8)]
    kw = dict(seg_indptr=torch.zeros(3, dtype=torch.int64), max_tokens_per_expert=4)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        if swiglu:
            moe.moe_expert_gemm_swiglu(*args, torch.zeros(64, **u8), torch.zeros(128, **u8), st, 1.0, **kw)
        else:
            moe.moe_expert_gemm(*args, torch.zeros(256, dtype=torch.bfloat16), st, **kw)
