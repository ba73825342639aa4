"""The token permutation's gradients where their sums are longest, and what a
set status word stops: against the formulas in 64 bits."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from test_gpu_permute import _case, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [4096, 4100, 4095, 16384])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient_of_one_large_term(H, dtype):
    """A term of 2^24 among terms of one: what is added to it later on its chain
    is lost.  A path of p additions loses at most p 2^-24 of the terms' sum; the
    longest has H / 128 on a lane's chain, 2 to join its chains and 5 across
    the lanes."""
    T, K, E = 9, 2, 4
    plan, slots, cap = _case(T, K, E, 16, seed=3)
    p = -(-H // 128) + 2 + 5
    for first in (0, 1, 130, H - 1):
        y = torch.ones((cap, H), dtype=dtype)
        y[:, first] = 2.0 ** 24
        g, w = torch.ones((T, H), dtype=dtype), _rand((T, K), torch.float32, 1)
        _, dw = moe.unpermute_tokens_backward(g.cuda(), y.cuda(), plan, w.cuda())
        total = 2.0 ** 24 + H - 1
        assert float((dw.double() - total).abs().max()) <= p * 2.0 ** -24 * total
