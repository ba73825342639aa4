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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [64, 61])
def test_a_set_status_word_stops_every_step(dtype, H):
    """Nothing is written, neither rows nor padding nor gradients."""
    T, K = 8, 2
    plan, slots, cap = _case(T, K, 4, 16)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    x, y = torch.ones((T, H), dtype=dtype).cuda(), torch.ones((cap, H), dtype=dtype).cuda()
    w = torch.ones((T, K), device="cuda")

    def sevens(rows):
        return torch.full((rows, H), 7.0, dtype=dtype, device="cuda")

    for out in (moe.permute_tokens(x, plan, sevens(cap), status),
                moe.permute_tokens_backward(y, plan, K, sevens(T), status),
                moe.unpermute_tokens(y, plan, w, sevens(T), status),
                moe.unpermute_tokens_backward(x, y, plan, w, sevens(cap), status)[0]):
        assert bool((out == 7).all())
    grad_w = torch.full((T, K), 7.0, device="cuda")
    moe._abi.moe_unpermute_tokens_backward(x, y, moe.dtype_code(dtype), T, H, K, w,
                                           plan["inv_perm"], plan["sorted_ids"], cap,
                                           sevens(cap), grad_w, status)
    assert bool((grad_w == 7).all())
