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


def _gated_ref(x):
    """(scales, values, block of each column) of gated rows in 64 bits."""
    H = x.shape[1] // 2
    v = x[:, :H].double() * torch.sigmoid(x[:, :H].double()) * x[:, H:].double()
    p = torch.zeros((x.shape[0], _nblk(H) * 128), dtype=torch.float64, device=x.device)
    p[:, :H] = v.abs()
    return p.view(x.shape[0], -1, 128).amax(-1) / 448, v


def _check_gated(x, q, s):
    """The scale within (8 + 1.2 * 16 + 2) 2^-23 < 2^-18 of the exact one for
    gates of at most 16; a code, half a step off, by 2^-4 of the value or half a
    subnormal step, 2^-10 of the scale."""
    sr, v = _gated_ref(x)
    sd = s.double()
    assert bool(((sd - sr).abs() <= 2.0 ** -18 * sr).all())
    se = sd.repeat_interleave(128, 1)[:, :v.shape[1]]
    err = (q.double() * se - v).abs()
    assert bool((err <= (2.0 ** -4 + 2.0 ** -15) * v.abs() + 2.0 ** -10 * 1.001 * se).all())


@pytest.mark.parametrize("T,H", [(3, 16), (1, 112), (7, 144), (50, 1008), (9, 128), (5000, 1040),
                                 (16411, 2048), (9800, 272)])
def test_gated_rows_of_words(T, H):
    """bf16 rows of a multiple of 16 columns, which are walked by teams with the
    next block's words in flight: one block to a team, several (from about 19,456
    blocks on), and rows that end inside a block.  The magnitude changes by up to
    2^30 from block to block, so a word of another block shows in the scale."""
    g = _gen(T)
    x = torch.randn(T, 2 * H, generator=g, device="cuda").clamp(-16, 16)
    e = torch.randint(-15, 16, (T, _nblk(H)), generator=g, device="cuda").float()
    x[:, H:] *= torch.exp2(2 * e).repeat_interleave(128, 1)[:, :H]
    x = x.to(torch.bfloat16)
    guard = torch.full((T + 2, H), 0x55, dtype=torch.uint8, device="cuda")
    q, s = moe.quantize_fp8_block(x, gated=True, out=(
        guard[1:-1], torch.full((T, _nblk(H)), float("nan"), device="cuda")))
    for t0 in range(0, T, 2048):
        r = slice(t0, t0 + 2048)
        _check_gated(x[r], q[r].view(torch.float8_e4m3fn), s[r])
    assert bool((guard[0] == 0x55).all()) and bool((guard[-1] == 0x55).all())


@pytest.mark.parametrize("T,H,gated", [(300001, 7168, False), (150001, 7168, True)])
def test_quantize_offsets_past_32_bits(T, H, gated):
    """More than 2^31 elements: sampled rows are those of a call of their own,
    which the other tests check, and of the formula."""
    x = torch.randn(T, (2 if gated else 1) * H, device="cuda", dtype=torch.bfloat16).clamp_(-16, 16)
    assert x.numel() > 2 ** 31
    q, s = moe.quantize_fp8_block(x, gated=gated)
    pick = torch.tensor([0, 1, T // 2, 2 ** 31 // x.shape[1] - 1, 2 ** 31 // x.shape[1],
                         2 ** 31 // x.shape[1] + 1, T - 2, T - 1], device="cuda")
    qp, sp = moe.quantize_fp8_block(x[pick], gated=gated)
    qs = q.view(torch.uint8)[pick]
    assert torch.equal(qs, qp.view(torch.uint8)) and torch.equal(s[pick], sp)
    if gated:
        _check_gated(x[pick], qp, sp)
    else:
        m = x[pick].double().abs().view(8, -1, 128).amax(-1)
        assert bool(((sp.double() * 448 - m).abs() <= 2.0 ** -22 * m).all())


@pytest.mark.parametrize("T,block_m", [(40, 16), (700, 128)])
def test_gradient_of_the_grouped_products_rows(T, block_m):
    """d a of sum(out * g): row s of expert e is g's row times w[e], the same
    call on each expert's transposed codes and block scales."""
    E, N, K = 4, 640, 400
    ids = torch.randint(0, E, (T, 1), generator=_gen(3), device="cuda", dtype=torch.int32)
    plan = moe.align(ids, E, block_m)
    cap = plan["sorted_ids"].numel()
    w, sw = _codes((E, N, K), 2), _scales((E, _nblk(N), _nblk(K)), 4)
    gq, gs = moe.quantize_fp8_block(
        torch.randn(cap, N, generator=_gen(7), device="cuda").to(torch.bfloat16))
    wt = w.view(torch.uint8).transpose(1, 2).contiguous()
    out = torch.full((cap, K), 777.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_gemm_fp8_block(gq, gs, wt, sw.transpose(1, 2).contiguous(), plan, block_m, out=out)
    seen = 0
    for e, _, first, n in plan["block_info"][:int(plan["num_blocks"])].tolist():
        r = slice(first, first + n)
        _close(out[r], _dequant(gq[r], gs[r]), _dequant(w[e], sw[e], N).t(), torch.bfloat16)
        seen += n
    assert seen == T


@pytest.mark.parametrize("M", [1, 8])
def test_a_status_word_that_is_set_meanwhile(M):
    """From another stream, while the CTAs of the kernel for few rows start: each stores
    its 16 columns whole and right, or leaves them alone."""
    N, K = 8192, 512
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    want = moe.gemm_fp8_block(a, sa, w, sw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for wait in range(0, 6000, 60):
        status.zero_()
        out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        moe.gemm_fp8_block(a, sa, w, sw, out=out, dev_status=status)
        with torch.cuda.stream(side):
            torch.cuda._sleep(wait)
            status.fill_(1)
        torch.cuda.synchronize()
        right, left = ((out == v).view(M, -1, 16) for v in (want, 7.0))
        # a CTA has its columns of every row
        assert bool((right.all(2).all(0) | left.all(2).all(0)).all())
    moe.gemm_fp8_block(a, sa, w, sw, out=out.fill_(7.0), dev_status=status)
    assert bool((out == 7.0).all())
