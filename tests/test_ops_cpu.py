"""Refusals of the permutation, quantiser and block-scaled products that stop
on the host: no call of this file gets as far as a launch, so they run without
a GPU."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe


def _plan(cap, block_m, experts):
    return dict(sorted_ids=torch.zeros(cap, dtype=torch.int32),
                inv_perm=torch.zeros(4, dtype=torch.int32),
                counts=torch.zeros(experts, dtype=torch.int32),
                block_info=torch.zeros((cap // block_m, 4), dtype=torch.int32),
                num_blocks=torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("experts", [4, 256])
def test_grouped_product_refuses_a_plan_over_more_experts(experts):
    cap, N, K, E = 64, 32, 128, 3
    a = torch.zeros((cap, K), dtype=torch.uint8)
    w = torch.zeros((E, N, K), dtype=torch.uint8)
    with pytest.raises(ValueError, match=f"over {experts} experts, w holds 3"):
        moe.grouped_gemm_fp8_block(a, torch.ones((cap, 1)), w, torch.ones((E, 1, 1)),
                                   _plan(cap, 16, experts), 16)
