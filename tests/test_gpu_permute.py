"""Token permutation and its gradients on the GPU, against the formulas in 64
bits (and the oracle's align for the lists).  Tolerances, derived before any
run: rows that are only copied are equal; a sum of n products in fp32 is within
d = 2 n 2^-23 sum |terms| of the exact one, and is rounded once, so the output
lies between the output type's roundings of (exact - d) and (exact + d)."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
import oracle
from mixture_experts_grouped_02_gb300 import _abi

pytestmark = pytest.mark.gpu


def _ids(T, K, E, seed, skew=False):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g)
    if skew:
        logits += 3.0 * torch.randn(E, generator=g)
    return torch.topk(logits, K, dim=1).indices.to(torch.int32)


def _case(T, K, E, block_m, seed=0, skew=False, base=0, local=0):
    ids = _ids(T, K, E, seed, skew)
    plan = moe.align(ids.cuda(), E, block_m, expert_base=base, local_experts=local)
    al = oracle.align(ids.numpy(), E, block_m, expert_base=base, local_experts=local)
    slots = torch.from_numpy(np.asarray(al["inv_perm"], np.int64)).view(T, K)
    return plan, slots, plan["sorted_ids"].numel()


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def _permute_ref(x, slots, cap):
    out = torch.zeros((cap, x.shape[1]), dtype=x.dtype)
    for t in range(slots.shape[0]):
        for k in range(slots.shape[1]):
            if slots[t, k] >= 0:
                out[slots[t, k]] = x[t]
    return out


def _gathered(rows, slots):
    """(T, K, H) in 64 bits, zero for another shard's assignments."""
    v = rows.double()[slots.clamp(min=0)]
    return torch.where((slots >= 0)[..., None], v, 0.0)


def _between(got, ref, d, dtype):
    """got between the roundings to dtype of ref - d and ref + d."""
    got = got.cpu()
    assert got.dtype == dtype
    bad = (got < (ref - d).to(dtype)) | (got > (ref + d).to(dtype)) | got.isnan()
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


def _close_sum(got, terms, dtype, dim):
    ref, mag = terms.sum(dim), terms.abs().sum(dim)
    _between(got, ref, 2 * terms.shape[dim] * 2.0 ** -23 * mag, dtype)


SHAPES = [  # T, H, K, E, block_m
    (1, 7168, 8, 256, 16), (1, 1, 1, 1, 16), (5, 3, 2, 4, 32), (33, 129, 3, 8, 64),
    (64, 256, 2, 8, 128), (100, 2880, 4, 32, 128), (257, 1032, 6, 60, 256), (40, 2050, 9, 16, 16),
]


@pytest.mark.parametrize("T,H,K,E,block_m", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_permute_and_gradient(T, H, K, E, block_m, dtype):
    plan, slots, cap = _case(T, K, E, block_m, seed=T, skew=True)
    x = _rand((T, H), dtype, 1)
    out = torch.full((cap, H), float("nan"), dtype=dtype, device="cuda")
    got = moe.permute_tokens(x.cuda(), plan, out)
    assert torch.equal(got.cpu(), _permute_ref(x, slots, cap))
    g = _rand((cap, H), dtype, 2)
    pad = torch.ones(cap, dtype=torch.bool)
    pad[slots.flatten()] = False
    g[pad] = float("nan")  # padding rows are not read
    dx = moe.permute_tokens_backward(g.cuda(), plan, K)
    assert dx.dtype == dtype and dx.shape == (T, H)
    _close_sum(dx, _gathered(g, slots), dtype, 1)


@pytest.mark.parametrize("T,H,K,E,block_m", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unpermute_and_gradients(T, H, K, E, block_m, dtype):
    plan, slots, cap = _case(T, K, E, block_m, seed=T + 1)
    y = _rand((cap, H), dtype, 3)
    pad = torch.ones(cap, dtype=torch.bool)
    pad[slots.flatten()] = False
    y[pad] = float("nan")
    w = _rand((T, K), torch.float32, 4)
    out = moe.unpermute_tokens(y.cuda(), plan, w.cuda())
    _close_sum(out, w.double()[..., None] * _gathered(y, slots), dtype, 1)

    g = _rand((T, H), dtype, 5)
    buf = torch.full((cap, H), float("nan"), dtype=dtype, device="cuda")
    dy, dw = moe.unpermute_tokens_backward(g.cuda(), y.cuda(), plan, w.cuda(), buf)
    ref = torch.zeros((cap, H), dtype=torch.float64)
    ref[slots] = w.double()[..., None] * g.double()[:, None, :]
    _between(dy, ref, 2.0 ** -23 * ref.abs(), dtype)
    assert bool((dy.cpu()[pad] == 0).all())
    _close_sum(dw, g.double()[:, None, :] * _gathered(y, slots), torch.float32, 2)


@pytest.mark.parametrize("base,local", [(0, 3), (3, 5), (7, 1)])
def test_shard(base, local):
    T, K, E, H = 50, 3, 8, 136
    plan, slots, cap = _case(T, K, E, 16, seed=9, base=base, local=local)
    x, y = _rand((T, H), torch.bfloat16, 1), _rand((cap, H), torch.bfloat16, 2)
    w, g = _rand((T, K), torch.float32, 3), _rand((T, H), torch.bfloat16, 4)
    assert torch.equal(moe.permute_tokens(x.cuda(), plan).cpu(), _permute_ref(x, slots, cap))
    _close_sum(moe.permute_tokens_backward(y.cuda(), plan, K), _gathered(y, slots),
               torch.bfloat16, 1)
    _close_sum(moe.unpermute_tokens(y.cuda(), plan, w.cuda()),
               w.double()[..., None] * _gathered(y, slots), torch.bfloat16, 1)
    dy, dw = moe.unpermute_tokens_backward(g.cuda(), y.cuda(), plan, w.cuda())
    assert bool((dw.cpu()[slots < 0] == 0).all())
    _close_sum(dw, g.double()[:, None, :] * _gathered(y, slots), torch.float32, 2)
    held = torch.zeros(cap, dtype=torch.bool)
    held[slots[slots >= 0]] = True
    assert bool((dy.cpu()[~held] == 0).all())


def test_shard_without_a_token():
    T, K, E, H = 6, 1, 8, 64
    ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    plan = moe.align(ids, E, 16, expert_base=4, local_experts=2)
    cap = plan["sorted_ids"].numel()
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    w = torch.ones((T, K), device="cuda")
    y = torch.full((cap, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert bool((moe.permute_tokens(x, plan) == 0).all())
    assert bool((moe.permute_tokens_backward(y, plan, K) == 0).all())
    assert bool((moe.unpermute_tokens(y, plan, w) == 0).all())
    dy, dw = moe.unpermute_tokens_backward(x, y, plan, w)
    assert bool((dy == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn, torch.float32])
def test_codes_and_scales_are_copied(dtype):
    T, K, E = 30, 4, 16
    plan, slots, cap = _case(T, K, E, 32, seed=3)
    for H in (57, 112, 7168):
        x = torch.randint(0, 120, (T, H), generator=torch.Generator().manual_seed(H))
        x = x.to(torch.uint8).view(dtype) if dtype != torch.float32 else x.float()
        bits = torch.uint8 if dtype != torch.float32 else torch.float32
        got = moe.permute_tokens(x.cuda(), plan).cpu()
        assert torch.equal(got.view(bits), _permute_ref(x.view(bits), slots, cap))


def test_rows_off_the_vector_alignment():
    """Contiguous rows that start at any element of a buffer."""
    T, K, E, H = 21, 2, 8, 256
    plan, slots, cap = _case(T, K, E, 16, seed=5)
    for off in (1, 3, 8):
        flat = torch.randn(T * H + 16, device="cuda").to(torch.bfloat16)
        x = flat[off:off + T * H].view(T, H)
        yb = torch.randn(cap * H + 16, device="cuda").to(torch.bfloat16)
        y = yb[off:off + cap * H].view(cap, H)
        assert torch.equal(moe.permute_tokens(x, plan).cpu(), _permute_ref(x.cpu(), slots, cap))
        w = torch.rand((T, K), device="cuda")
        _close_sum(moe.unpermute_tokens(y, plan, w),
                   w.cpu().double()[..., None] * _gathered(y.cpu(), slots), torch.bfloat16, 1)
        dy, dw = moe.unpermute_tokens_backward(x, y, plan, w)
        _close_sum(dw, x.cpu().double()[:, None, :] * _gathered(y.cpu(), slots), torch.float32, 2)
        base = moe.unpermute_tokens_backward(x.clone(), y.clone(), plan, w)
        assert torch.equal(dy, base[0])


def test_gradients_against_differences():
    """Unpermute is linear in the rows and in the weights: a central difference
    of <out, g> along a direction is the gradient's product with it, up to the
    fp32 rounding of the two sums (relative 1e-4 at these sizes)."""
    T, K, E, H = 37, 3, 8, 96
    plan, slots, cap = _case(T, K, E, 16, seed=11)
    y, w = _rand((cap, H), torch.float32, 1).cuda(), _rand((T, K), torch.float32, 2).cuda()
    g = _rand((T, H), torch.float32, 3).cuda()
    dy, dw = moe.unpermute_tokens_backward(g, y, plan, w)
    vy, vw = _rand((cap, H), torch.float32, 4).cuda(), _rand((T, K), torch.float32, 5).cuda()
    loss = lambda yy, ww: float((moe.unpermute_tokens(yy, plan, ww).double() * g.double()).sum())
    h = 0.5
    num_y = (loss(y + h * vy, w) - loss(y - h * vy, w)) / (2 * h)
    num_w = (loss(y, w + h * vw) - loss(y, w - h * vw)) / (2 * h)
    scale_y = float((dy.double() * vy.double()).abs().sum())
    scale_w = float((dw.double() * vw.double()).abs().sum())
    assert abs(num_y - float((dy.double() * vy.double()).sum())) <= 1e-4 * scale_y
    assert abs(num_w - float((dw.double() * vw.double()).sum())) <= 1e-4 * scale_w
    x, gs = _rand((T, H), torch.float32, 6).cuda(), _rand((cap, H), torch.float32, 7).cuda()
    dx = moe.permute_tokens_backward(gs, plan, K)
    vx = _rand((T, H), torch.float32, 8).cuda()
    lossx = lambda xx: float((moe.permute_tokens(xx, plan).double() * gs.double()).sum())
    num_x = (lossx(x + h * vx) - lossx(x - h * vx)) / (2 * h)
    scale_x = float((dx.double() * vx.double()).abs().sum())
    assert abs(num_x - float((dx.double() * vx.double()).sum())) <= 1e-4 * scale_x


def test_infinities_and_nan_stay_in_their_rows():
    T, K, E, H = 20, 2, 8, 128
    plan, slots, cap = _case(T, K, E, 16, seed=13)
    y = _rand((cap, H), torch.bfloat16, 1)
    y[slots[3, 0], 5] = float("inf")
    y[slots[4, 1], 6] = float("nan")
    w = torch.rand((T, K), generator=torch.Generator().manual_seed(2)) + 0.1
    out = moe.unpermute_tokens(y.cuda(), plan, w.cuda()).float().cpu()
    assert out[3, 5] == float("inf") and bool(out[4, 6].isnan())
    bad = ~torch.isfinite(out)
    assert int(bad.sum()) == 2


def test_offsets_past_32_bits():
    """A list of more than 2^31 elements: the last rows against the formula."""
    T, K, E, H = 38000, 8, 64, 7168
    ids = _ids(T, K, E, 21)
    plan = moe.align(ids.cuda(), E, 16)
    cap = plan["sorted_ids"].numel()
    assert cap * H > 2 ** 31
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    xs = moe.permute_tokens(x, plan)
    inv = plan["inv_perm"].long().view(T, K)
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    for k in range(K):
        assert torch.equal(xs[inv[pick, k]], x[pick])
    last = int(plan["padded_offsets"][-1])
    top = plan["sorted_ids"][last - 64:last]
    rows = xs[last - 64:last]
    for s in range(64):
        i = int(top[s])
        want = x[i // K] if i < T * K else torch.zeros_like(x[0])
        assert torch.equal(rows[s], want)
    w = torch.rand((T, K), device="cuda")
    out = moe.unpermute_tokens(xs, plan, w)
    ref = x[pick].double() * w[pick].double().sum(1, keepdim=True)
    _between(out[pick], ref.cpu(), 2 * K * 2.0 ** -23 * ref.abs().cpu(), torch.bfloat16)
    dy, dw = moe.unpermute_tokens_backward(x, xs, plan, w)
    ref = (x[pick].double() ** 2).sum(1, keepdim=True).expand(-1, K)
    assert bool(((dw[pick].double() - ref).abs() <= H * 2.0 ** -23 * ref).all())
    s = inv[pick, K - 1]
    ref = (w[pick, K - 1:].double() * x[pick].double()).cpu()
    _between(dy[s], ref, 2.0 ** -23 * ref.abs(), torch.bfloat16)


def test_on_another_stream():
    T, K, E, H = 200, 2, 8, 512
    plan, slots, cap = _case(T, K, E, 16, seed=17)
    x = _rand((T, H), torch.bfloat16, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xd = x.cuda()
    side.wait_stream(torch.cuda.current_stream())
    a = moe.permute_tokens(xd, plan, stream=side)
    w = torch.ones((T, K), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    b = moe.unpermute_tokens(a, plan, w, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a.cpu(), _permute_ref(x, slots, cap))
    assert torch.equal(b.float().cpu(), K * x.float())


def test_nothing_to_do_and_skipped():
    plan = dict(inv_perm=torch.empty(0, dtype=torch.int32, device="cuda"),
                sorted_ids=torch.empty(0, dtype=torch.int32, device="cuda"))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert moe.permute_tokens(x, plan).shape == (0, 64)
    assert moe.permute_tokens_backward(x, plan, 2).shape == (0, 64)
    # a status word that already holds an error: nothing is written
    plan, slots, cap = _case(8, 2, 4, 16)
    x = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((cap, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    moe.permute_tokens(x, plan, out, dev_status=status)
    assert bool((out == 7).all())


def test_refusals():
    plan, _, cap = _case(8, 2, 4, 16)
    x = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.ones((cap, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((8, 2), device="cuda")
    for bad in (lambda: moe.permute_tokens(x.half(), plan),
                lambda: moe.permute_tokens(x[:7], plan),
                lambda: moe.permute_tokens(x.t().contiguous().t(), plan),
                lambda: moe.permute_tokens(x.cpu(), plan),
                lambda: moe.permute_tokens(x, plan, out=y[:-1]),
                lambda: moe.permute_tokens(x, dict(plan, inv_perm=plan["inv_perm"].long())),
                lambda: moe.permute_tokens_backward(y[:-1], plan, 2),
                lambda: moe.permute_tokens_backward(y, plan, 3),
                lambda: moe.permute_tokens_backward(y.to(torch.float8_e4m3fn), plan, 2),
                lambda: moe.unpermute_tokens(y[:-1], plan, w),
                lambda: moe.unpermute_tokens(y, plan, w.double()),
                lambda: moe.unpermute_tokens(y, plan, w[:-1]),
                lambda: moe.unpermute_tokens_backward(x.float(), y, plan, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError) as e:
        _abi.moe_permute_tokens(x, _abi.MOE_E2M1_MX, 8, 64, 2, plan["inv_perm"],
                                plan["sorted_ids"], cap, y)
    assert e.value.status == _abi.MOE_ERR_INVALID_ARG


def test_checked_build_skips_slots_outside_the_list():
    """The range-checked build reports a corrupt inverse permutation instead of
    reading or writing outside the rows."""
    L = _abi.checked_lib()
    T, K, H = 4, 2, 64
    plan, slots, cap = _case(T, K, 4, 16)
    inv = plan["inv_perm"].clone()
    inv[3] = cap + 5
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((T, K), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs = torch.zeros((cap, H), dtype=torch.bfloat16, device="cuda")
    out, dw = torch.zeros_like(x), torch.zeros_like(w)
    s = torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()
    ids = plan["sorted_ids"]
    for call in (lambda: L.moe_permute_tokens(p(x), _abi.MOE_BF16, T, H, K, p(inv), p(ids), cap,
                                              p(xs), p(st), s),
                 lambda: L.moe_permute_tokens_backward(p(xs), _abi.MOE_BF16, T, H, K, p(inv), cap,
                                                       p(out), p(st), s),
                 lambda: L.moe_unpermute_tokens(p(xs), _abi.MOE_BF16, T, H, K, p(w), p(inv), cap,
                                                p(out), p(st), s),
                 lambda: L.moe_unpermute_tokens_backward(p(x), p(xs), _abi.MOE_BF16, T, H, K, p(w),
                                                         p(inv), p(ids), cap, p(xs), p(dw), p(st),
                                                         s)):
        st.zero_()
        assert call() == _abi.MOE_OK
        assert int(st.item()) == _abi.MOE_ERR_BOUNDS
