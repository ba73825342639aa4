"""The 128-block fp8 quantiser and products where their kernels hand data from
one warp to another, loop, or stop: against the formulas in 64 bits, with the
bounds of test_gpu_fp8_block.py unless a test derives its own."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import _abi
from test_gpu_fp8_block import _close, _codes, _dequant, _gen, _nblk, _scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", range(5))
@pytest.mark.parametrize("M,N,K", [(20, 1000, 7168), (400, 1000, 4608), (2500, 1096, 2048)])
def test_scales_change_with_every_slot(form, M, N, K):
    """Row scales from 2^-40 to 2^40 over many stages and tiles: a scale slot
    written before its last reader is done moves a sum by powers of two."""
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    e = torch.randint(-40, 41, (M, _nblk(K)), generator=_gen(5), device="cuda")
    sa, sw = torch.exp2(e.float()), _scales((_nblk(N), _nblk(K)), 4)
    outs = []
    for _ in range(3):
        out = torch.empty((M, N), dtype=torch.float32, device="cuda")
        _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_F32, form)
        outs.append(out)
    _close(outs[0], _dequant(a, sa), _dequant(w, sw, N), torch.float32)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("form", [2, 3, 4])
@pytest.mark.parametrize("K", [128, 256, 384])
def test_a_cluster_stores_nothing_when_one_of_its_ctas_gave_up(form, K):
    """Of the CTAs that share so short a K some have no scale block: with no
    copies in flight they finish, the others' waits run out.  The first ones must
    not store what the others left in shared memory."""
    M, N = 300, 400
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form, 2_000_000,
                                 status)
    assert moe.moe_get_device_status(status) == _abi.MOE_ERR_TIMEOUT
    assert bool((out == 7).all())
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), torch.bfloat16)


@pytest.mark.parametrize("form", range(5))
@pytest.mark.parametrize("K", [128, 512, 1024, 7168])
def test_waits_that_run_out_with_copies_in_flight(form, K):
    """With the scales held back the copies are issued and no stage is taken:
    the issuing thread gives up while the producer has either left (a K of few
    stages) or waits as well.  The kernel drains, reports MOE_ERR_TIMEOUT, writes
    nothing and leaves the device usable."""
    M, N = 300, 400
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form + 16, 2_000_000,
                                 status)
    assert moe.moe_get_device_status(status) == _abi.MOE_ERR_TIMEOUT
    assert bool((out == 7).all())
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), torch.bfloat16)


def test_held_back_scales_need_a_wait_limit():
    a, s = _codes((4, 128), 1), _scales((4, 1), 3)
    out = torch.empty((4, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoEError) as e:
        _abi.moe_test_gemm_fp8_block(a, s, a, s[:1], 4, 4, 128, out, _abi.MOE_BF16, 16)
    assert e.value.status == _abi.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gated_precision_over_all_gates(dtype):
    """The scale of a block of one value shows v itself.  The fast exponential
    is within 2 + 1.173 |gate| units of the last place (2^-23), the fast division
    within 2, three more operations and the scale's division are rounded once:
    (8 + 1.2 |gate|) 2^-23."""
    g = torch.cat([torch.linspace(-87, 87, 4001), torch.tensor([-87.25, -1e-3, 1e-30, 3e4])])
    x = torch.zeros((g.numel(), 256))
    x[:, 5], x[:, 133] = g, 2.0 ** 60
    x = x.to(dtype)
    q, s = moe.quantize_fp8_block(x.cuda(), gated=True)
    gate = x[:, 5].double()
    v = gate * torch.sigmoid(gate) * 2.0 ** 60
    err = (s[:, 0].double().cpu() * 448 - v.abs()).abs()
    seen = v.abs() > 2.0 ** -100
    assert bool((err <= (8 + 1.2 * gate.abs()) * 2.0 ** -23 * v.abs())[seen].all())
    assert int(seen.sum()) > 4000
    assert bool((q[:, 5].cpu().double()[seen].abs() == 448).all())


@pytest.mark.parametrize("T,block_m", [(20, 16), (300, 128), (300, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_set_status_word_stops_the_grouped_product(T, block_m, dtype):
    ids = torch.randint(0, 4, (T, 1), generator=_gen(1), device="cuda", dtype=torch.int32)
    plan = moe.align(ids, 4, block_m)
    cap = plan["sorted_ids"].numel()
    out = torch.full((cap, 72), 7.0, dtype=dtype, device="cuda")
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    moe.grouped_gemm_fp8_block(_codes((cap, 128), 1), _scales((cap, 1), 2), _codes((4, 72, 128), 3),
                               _scales((4, 1, 1), 4), plan, block_m, out=out, dev_status=status)
    assert bool((out == 7).all())


@pytest.mark.parametrize("T", [3, 300])
def test_an_id_out_of_range_leaves_the_layers_output(T):
    """align reports it; no step that reads the lists then runs, and the
    output keeps what it held."""
    E, K, H, I = 4, 2, 256, 128
    g = _gen(1)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[T - 1, 1] = E
    out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.forward_fp8_block(x, ids, torch.full((T, K), 0.5, device="cuda"),
                          _codes((E, 2 * I, H), 3), _scales((E, 2, 2), 4), _codes((E, H, I), 5),
                          _scales((E, 2, 1), 6), out=out, dev_status=status)
    assert moe.moe_get_device_status(status) == _abi.MOE_ERR_DEVICE_BAD_ID
    assert bool((out == 7).all())
