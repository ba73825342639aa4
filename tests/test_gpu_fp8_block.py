"""The 128-block fp8 quantiser and products on the GPU, against the formulas
in 64 bits.  Tolerances, derived before any run:

 * quantiser of x itself: the same fp32 operations on the CPU, equal;
 * gated: the exact v is within 2^-17 of the fp32 one (fast exponential and
   division at |gate| <= 16), a code is half a step (2^-4 relative, or half a
   subnormal step 2^-10 of the scale) off, the scale within 2^-16;
 * products: each scale block is summed by the tensor core in fp32 or better
   (128 terms), the blocks by fp32 fused multiply-adds, the scale product is
   rounded once: the fp32 sum is within d = (128 + blocks + 4) 2^-23 sum
   |terms| of the exact one, and the output, rounded once, lies between the
   output type's roundings of (exact - d) and (exact + d).
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
import oracle
from mixture_experts_grouped_02_gb300 import _abi

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100


def _nblk(n):
    return -(-n // 128)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(shape, seed):
    v = torch.randn(shape, generator=_gen(seed), device="cuda") * 110
    return v.clamp(-448, 448).to(F8)


def _scales(shape, seed):
    return 0.01 * (0.1 + torch.rand(shape, generator=_gen(seed), device="cuda"))


def _dequant(q, s, rows=None):
    s = s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if rows is not None:
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    return q.double() * s


def _close(got, a, w, dtype):
    """got against a @ w.T (64-bit operands), by the derived bound."""
    ref, mag = a @ w.t(), a.abs() @ w.abs().t()
    d = (128 + _nblk(a.shape[1]) + 4) * 2.0 ** -23 * mag
    assert got.dtype == dtype
    bad = (got < (ref - d).to(dtype)) | (got > (ref + d).to(dtype)) | got.isnan()
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


# ------------------------------------------------------------- quantiser

def _quant_ref(x):
    T, H = x.shape
    nb = _nblk(H)
    p = torch.zeros((T, nb * 128))
    p[:, :H] = x.float()
    b = p.view(T, nb, 128)
    m = torch.from_numpy(np.fmax(np.fmax.reduce(np.abs(b.numpy()), axis=-1), np.float32(FLOOR)))
    c = torch.full_like(m, 448.0)  # a tensor: scalar / tensor is no IEEE division in torch
    q = (b * (c / m)[..., None]).clamp(-448, 448)
    return q.reshape(T, -1)[:, :H].to(F8), m / c


@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (3, 7168), (5, 130), (17, 129), (64, 2880),
                                 (200, 2048), (33, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(T, H, dtype):
    x = (torch.randn(T, H, generator=torch.Generator().manual_seed(T)) * 3).to(dtype)
    x[0] *= 1e-20
    if T > 2:
        x[1] = 0
        x[2] *= 1e20
    q, s = moe.quantize_fp8_block(x.cuda())
    qr, sr = _quant_ref(x)
    assert q.dtype == F8 and s.dtype == torch.float32
    assert torch.equal(s.cpu(), sr)
    assert torch.equal(q.cpu().view(torch.uint8) & 0x7f, qr.view(torch.uint8) & 0x7f)
    assert torch.equal(q.cpu().double(), qr.double())


def test_quantize_extremes():
    """Subnormals, the largest values, zeros, infinities and NaN, each in a
    block of its own: none reaches another block."""
    x = torch.ones((1, 128 * 6), dtype=torch.float32)
    x[0, :128] = 1e-40                     # subnormal: below the floor, zeros
    x[0, 128:256] = 3.4e38
    x[0, 256:384] = 0.0
    x[0, 384] = float("inf")
    x[0, 512] = float("nan")
    q, s = moe.quantize_fp8_block(x.cuda())
    q, s = q.cpu().double()[0], s.cpu().double()[0]
    assert bool((q[:128] == 0).all()) and float(s[0]) == float(np.float32(FLOOR) / np.float32(448))
    assert bool((q[128:256] == 448).all()) and abs(s[1] * 448 / 3.4e38 - 1) < 1e-6
    assert bool((q[256:384] == 0).all())
    assert bool(q[384].isnan()) and s[3] == float("inf")
    assert bool(q[512].isnan()) and bool((q[513:640] == 448).all()) and abs(s[4] * 448 - 1) < 1e-6
    assert bool((q[640:] == 448).all())


@pytest.mark.parametrize("T,H", [(1, 8), (4, 2048), (9, 129), (50, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_gated(T, H, dtype):
    x = (torch.randn(T, 2 * H, generator=torch.Generator().manual_seed(H)) * 3).to(dtype)
    x = x.clamp(-16, 16)
    q, s = moe.quantize_fp8_block(x.cuda(), gated=True)
    g, u = x[:, :H].double(), x[:, H:].double()
    v = g * torch.sigmoid(g) * u
    p = torch.zeros((T, _nblk(H) * 128), dtype=torch.float64)
    p[:, :H] = v.abs()
    sr = p.view(T, -1, 128).amax(-1) / 448
    sc = s.double().cpu()
    assert bool(((sc - sr).abs() <= 2.0 ** -16 * sr + 1e-30).all())
    se = sc.repeat_interleave(128, 1)[:, :H]
    err = (q.cpu().double() * se - v).abs()
    assert bool((err <= (2.0 ** -4 + 2.0 ** -15) * v.abs() + 2.0 ** -10 * 1.001 * se).all())


def test_gated_gate_of_any_size():
    """SiLU of very negative and very large gates: -0 and the gate itself."""
    x = torch.zeros((1, 256))
    x[0, :4] = torch.tensor([-1e30, -200.0, 200.0, 1e30])
    x[0, 128:] = 1.0
    q, s = moe.quantize_fp8_block(x.cuda(), gated=True)
    v = q.cpu().double()[0] * s.cpu().double()[0, 0]
    assert float(v[0]) == 0 and float(v[1]) == 0 and abs(float(v[3]) / 1e30 - 1) < 1e-5


# ---------------------------------------------------------------- product

GEMMS = [  # M, N, K
    (1, 1, 16), (1, 7168, 2048), (1, 256, 128), (2, 8, 48), (3, 24, 4096), (7, 72, 144),
    (8, 512, 1024), (9, 200, 2080), (16, 128, 128), (17, 136, 256), (33, 300, 400),
    (64, 1000, 512), (65, 257, 1040), (128, 256, 384), (129, 264, 640), (200, 520, 128),
    (333, 2880, 2880), (700, 1111, 528),
]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, dtype):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    guard = torch.full((M + 2, N), 777.0, dtype=dtype, device="cuda")
    out = guard[1:-1]
    moe.gemm_fp8_block(a, sa, w, sw, out=out)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), dtype)
    assert bool((guard[0] == 777).all()) and bool((guard[-1] == 777).all())


@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("N,K", [(1, 16), (17, 144), (520, 2064), (2500, 528), (6000, 7168)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_of_few_rows(M, N, K, dtype):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    guard = torch.full((M + 2, N), 777.0, dtype=dtype, device="cuda")
    out = guard[1:-1]
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, moe.dtype_code(dtype), 5)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), dtype)
    assert bool((guard[0] == 777).all()) and bool((guard[-1] == 777).all())
    with pytest.raises(moe.MoEError):  # nine rows
        _abi.moe_test_gemm_fp8_block(_codes((9, K), 1), _scales((9, _nblk(K)), 3), w, sw, 9, N, K,
                                     torch.empty((9, N), dtype=dtype, device="cuda"),
                                     moe.dtype_code(dtype), 5)


@pytest.mark.parametrize("form", range(5))
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (5, 136, 400), (40, 200, 1168), (129, 520, 2064),
                                   (300, 257, 640), (2100, 392, 144)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_in_every_form(form, M, N, K, dtype):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    guard = torch.full((M + 2, N), 777.0, dtype=dtype, device="cuda")
    out = guard[1:-1]
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, moe.dtype_code(dtype), form)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), dtype)
    assert bool((guard[0] == 777).all()) and bool((guard[-1] == 777).all())


# sizes on the sides of the choice between the forms: 128 and 64 weight rows to
# a CTA, a split K
@pytest.mark.parametrize("M,N,K", [(1300, 2000, 400), (100, 12800, 256), (2, 64, 7168),
                                   (257, 576, 4096), (20000, 128, 272), (8, 9000, 7168), (8, 9600, 7168)])
def test_gemm_across_the_choice_of_form(M, N, K):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    got = moe.gemm_fp8_block(a, sa, w, sw)
    _close(got, _dequant(a, sa), _dequant(w, sw, N), torch.bfloat16)


@pytest.mark.parametrize("form", range(5))
def test_waits_are_bounded(form):
    """With no copies in flight every form's first wait runs out: it reports
    MOE_ERR_TIMEOUT, writes nothing and leaves the device usable."""
    M, N, K = 300, 400, 1024
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, 8), 3), _scales((4, 8), 4)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form, 2_000_000,
                                 status)
    assert moe.moe_get_device_status(status) == _abi.MOE_ERR_TIMEOUT
    assert bool((out == 7).all())
    got = moe.gemm_fp8_block(a, sa, w, sw)
    _close(got, _dequant(a, sa), _dequant(w, sw, N), torch.bfloat16)


def test_gemm_is_deterministic_and_takes_uint8():
    M, N, K = 48, 640, 1536 + 16
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    one = moe.gemm_fp8_block(a, sa, w, sw, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(moe.gemm_fp8_block(a.view(torch.uint8), sa, w.view(torch.uint8), sw,
                                              out_dtype=torch.float32), one)


@pytest.mark.parametrize("M", [1, 5, 40, 150])
def test_gemm_row_with_nan_or_infinite_scale(M):
    """A NaN code or an infinite scale of one row reaches that row only."""
    N, K = 200, 512
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, _nblk(K)), 3), _scales((_nblk(N), _nblk(K)), 4)
    clean = moe.gemm_fp8_block(a, sa, w, sw)
    a.view(torch.uint8)[M - 1, 130] = 0x7f
    got = moe.gemm_fp8_block(a, sa, w, sw)
    assert bool(got[M - 1].isnan().all())
    assert torch.equal(got[:M - 1], clean[:M - 1])
    a.view(torch.uint8)[M - 1, 130] = 0
    sa[0, 1] = float("inf")
    got = moe.gemm_fp8_block(a, sa, w, sw)
    assert not bool(torch.isfinite(got[0]).any())
    assert torch.equal(got[1:M - 1], clean[1:M - 1])


def test_gemm_scales_of_wide_range():
    """Block scales from 2^-60 to 2^60: the products of a block meet only
    after their scales are applied."""
    M, N, K = 20, 256, 1024
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    e = torch.randint(-60, 61, (M, _nblk(K)), generator=_gen(5), device="cuda")
    sa = torch.exp2(e.float())
    sw = _scales((_nblk(N), _nblk(K)), 4)
    for dtype in (torch.bfloat16, torch.float32):
        got = moe.gemm_fp8_block(a, sa, w, sw, out_dtype=dtype)
        _close(got, _dequant(a, sa), _dequant(w, sw, N), dtype)


@pytest.mark.parametrize("M,N,K", [(300, 4096, 1024), (6, 4096, 1024), (70, 2880, 2880)])
def test_gradient_of_the_activations(M, N, K):
    """d a of sum(out * g) is g times w: the same product on the transposed
    codes and block scales, here against the formula on the quantised g."""
    w, sw = _codes((N, K), 2), _scales((_nblk(N), _nblk(K)), 4)
    g = torch.randn(M, N, generator=_gen(7), device="cuda").to(torch.bfloat16)
    gq, gs = moe.quantize_fp8_block(g)
    wt = w.view(torch.uint8).t().contiguous()
    da = moe.gemm_fp8_block(gq, gs, wt, sw.t().contiguous())
    _close(da, _dequant(gq, gs), _dequant(w, sw, N).t(), torch.bfloat16)
    # and the quantisation itself moves it by at most half a code per term
    # (2^-4 relative, or half a subnormal step)
    wd = _dequant(w, sw, N)
    se = gs.double().repeat_interleave(128, 1)[:, :N]
    lim = (2.0 ** -4 * g.double().abs() + 2.0 ** -10 * se) @ wd.abs()
    ref = g.double() @ wd
    assert bool(((da.double() - ref).abs() <= 1.01 * lim + 2.0 ** -8 * ref.abs()).all())


def test_gemm_offsets_past_32_bits():
    """An output of more than 2^31 elements: sampled rows."""
    M, N, K = 540001, 4096, 128
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sa, sw = _scales((M, 1), 3), _scales((_nblk(N), 1), 4)
    out = moe.gemm_fp8_block(a, sa, w, sw)
    assert out.numel() > 2 ** 31
    pick = torch.tensor([0, 127, 128, M // 2, M - 130, M - 1], device="cuda")
    sub = a.view(torch.uint8)[pick].view(F8)
    _close(out[pick], _dequant(sub, sa[pick]), _dequant(w, sw, N), torch.bfloat16)


# ---------------------------------------------------------------- grouped

def _ids(T, K, E, seed, skew):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g)
    if skew:
        logits += 3.0 * torch.randn(E, generator=g)
    return torch.topk(logits, K, dim=1).indices.to(torch.int32)


def _grouped(T, K, E, N, Kd, block_m, dtype, seed=0, skew=True, ids=None, base=0, local=0):
    ids = _ids(T, K, E, seed, skew) if ids is None else ids
    L = local or E
    plan = moe.align(ids.cuda(), E, block_m, expert_base=base, local_experts=local)
    al = oracle.align(ids.numpy(), E, block_m, expert_base=base, local_experts=local)
    cap = plan["sorted_ids"].numel()
    a, w = _codes((cap, Kd), 1), _codes((L, N, Kd), 2)
    sa, sw = _scales((cap, _nblk(Kd)), 3), _scales((L, _nblk(N), _nblk(Kd)), 4)
    valid = torch.zeros(cap, dtype=torch.bool)
    for b in range(al["num_blocks"]):
        _, _, first, n = (int(v) for v in al["block_info"][b])
        valid[first:first + n] = True
    a.view(torch.uint8)[(~valid).cuda()] = 0x7f  # padding rows hold NaN codes
    out = torch.full((cap, N), 777.0, dtype=dtype, device="cuda")
    moe.grouped_gemm_fp8_block(a, sa, w, sw, plan, block_m, out=out)
    for b in range(al["num_blocks"]):
        e, _, first, n = (int(v) for v in al["block_info"][b])
        r = slice(first, first + n)
        _close(out[r], _dequant(a[r], sa[r]), _dequant(w[e], sw[e], N), dtype)
    assert bool((out[(~valid).cuda()] == 777).all())  # padding rows untouched
    return out


@pytest.mark.parametrize("T,K,E,N,Kd,block_m", [
    (1, 8, 256, 128, 256, 16), (1, 1, 1, 40, 16, 16), (8, 2, 8, 512, 1024, 16),
    (8, 8, 32, 264, 400, 16), (20, 4, 8, 300, 272, 32), (60, 2, 4, 520, 384, 64),
    (100, 3, 5, 256, 2080, 128), (300, 2, 8, 1000, 640, 128), (700, 2, 3, 260, 256, 256),
    (513, 1, 2, 128, 128, 256), (3000, 2, 3, 1200, 400, 128), (2500, 1, 2, 2000, 272, 256),
    (2000, 2, 2, 1000, 144, 64), (40, 2, 4, 64, 6400, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped(T, K, E, N, Kd, block_m, dtype):
    _grouped(T, K, E, N, Kd, block_m, dtype, seed=T)


@pytest.mark.parametrize("block_m", [16, 32, 64, 128, 256])
def test_grouped_one_expert_takes_all(block_m):
    """Every token to the same expert, the others empty."""
    ids = torch.full((290, 1), 2, dtype=torch.int32)
    _grouped(290, 1, 4, 320, 272, block_m, torch.bfloat16, ids=ids)


@pytest.mark.parametrize("base,local", [(0, 3), (5, 3)])
def test_grouped_shard(base, local):
    _grouped(90, 3, 8, 264, 256, 16, torch.bfloat16, seed=5, base=base, local=local)


def test_grouped_shard_without_a_token():
    ids = torch.zeros((6, 1), dtype=torch.int32)
    out = _grouped(6, 1, 8, 64, 128, 16, torch.bfloat16, ids=ids, base=4, local=2)
    assert bool((out == 777).all())


def test_grouped_weights_past_32_bits():
    """More than 2^31 bytes of weights: the last experts' rows."""
    E, N, Kd, T = 80, 4096, 7168, 4
    ids = torch.tensor([[78], [79], [0], [79]], dtype=torch.int32)
    plan = moe.align(ids.cuda(), E, 16)
    cap = plan["sorted_ids"].numel()
    a = _codes((cap, Kd), 1)
    w = torch.empty((E, N, Kd), dtype=torch.uint8, device="cuda")
    for e in (0, 78, 79):
        w[e] = _codes((N, Kd), e).view(torch.uint8)
    sa, sw = _scales((cap, 56), 3), _scales((E, 32, 56), 4)
    out = moe.grouped_gemm_fp8_block(a, sa, w, sw, plan, 16)
    for t in range(T):
        s = int(plan["inv_perm"][t])
        e = int(ids[t, 0])
        _close(out[s:s + 1], _dequant(a[s:s + 1], sa[s:s + 1]),
               _dequant(w[e].view(F8), sw[e], N), torch.bfloat16)


# ------------------------------------------------------- together, refusals

def _ffn_ref(x, ids, tw, w13, s13, w2, s2, base=0):
    """The layer of exact (unquantised) activations in 64 bits."""
    T, H = x.shape
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    I = w13.shape[1] // 2
    for e in range(w13.shape[0]):
        t, k = (ids == e + base).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gu = x[t].double() @ _dequant(w13[e], s13[e], 2 * I).t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y = h @ _dequant(w2[e], s2[e], H).t()
        out.index_add_(0, t, tw[t, k].double()[:, None] * y)
    return out


@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (16, 16, 4), (300, 4, 2)])
def test_expert_ffn(T, E, K):
    """The whole layer.  Each activation code is at most 2^-4 off relatively,
    uniformly over a step about 0.018 rms of the value; two roundings through
    products of many terms keep the relative L2 distance below 0.06."""
    H, I = 512, 384
    ids = _ids(T, K, E, 3, False).cuda()
    tw = torch.softmax(torch.randn(T, K, generator=_gen(1), device="cuda"), 1)
    x = torch.randn(T, H, generator=_gen(2), device="cuda").to(torch.bfloat16)
    w13, w2 = _codes((E, 2 * I, H), 3), _codes((E, H, I), 4)
    s13, s2 = 0.04 * _scales((E, 6, 4), 5), 0.04 * _scales((E, 4, 3), 6)
    got = moe.forward_fp8_block(x, ids, tw, w13, s13, w2, s2)
    ref = _ffn_ref(x, ids, tw, w13, s13, w2, s2)
    assert float((got.double() - ref).norm() / ref.norm()) <= 0.06
    # two shards add up to the layer (bf16 rounding of each share)
    h = E // 2
    parts = [moe.forward_fp8_block(x, ids, tw, w13[b:b + h], s13[b:b + h].contiguous(),
                                   w2[b:b + h], s2[b:b + h].contiguous(), num_experts=E,
                                   expert_base=b) for b in (0, h)]
    total = parts[0].double() + parts[1].double()
    assert float((total - got.double()).norm() / ref.norm()) <= 2.0 ** -7
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = moe.forward_fp8_block(x, ids, tw, w13, s13, w2, s2, stream=side)
    side.synchronize()
    assert torch.equal(again, got)
    assert moe.forward_fp8_block(x[:0], ids[:0], tw[:0], w13, s13, w2, s2).shape == (0, H)


def test_expert_ffn_with_an_id_out_of_range():
    """Reported in the status word; the lists are unspecified then, so no later
    step may read them."""
    T, E, K, H, I = 20, 4, 2, 256, 128
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids = _ids(T, K, E, 1, False).cuda()
    ids[7, 1] = E
    tw = torch.full((T, K), 0.5, device="cuda")
    args = (_codes((E, 2 * I, H), 3), _scales((E, 2, 2), 4), _codes((E, H, I), 5),
            _scales((E, 2, 1), 6))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.forward_fp8_block(x, ids, tw, *args, dev_status=status)
    assert moe.moe_get_device_status(status) == _abi.MOE_ERR_DEVICE_BAD_ID
    moe.forward_fp8_block(x, ids, tw, *args)  # with a status word of its own
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        moe.forward_fp8_block(x, ids.long(), tw, *args)


def test_example():
    """The example runs, its fp8 layer is near the bf16 one (the bound of
    test_expert_ffn, doubled for bf16's own rounding) and its loss falls."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_expert_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    distances, losses = example.main(["--hidden", "512", "--inter", "256", "--experts", "16",
                                      "--topk", "4", "--tokens", "1", "40", "300"])
    assert max(distances) <= 0.12
    assert losses[-1] < losses[0]


def test_skipped_when_the_status_is_set():
    a, w = _codes((4, 128), 1), _codes((64, 128), 2)
    sa, sw = _scales((4, 1), 3), _scales((1, 1), 4)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.gemm_fp8_block(a, sa, w, sw, out=out, dev_status=status)
    assert bool((out == 7).all())
    big = torch.full((300, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.gemm_fp8_block(_codes((300, 128), 1), _scales((300, 1), 3), w, sw, out=big,
                       dev_status=status)
    assert bool((big == 7).all())


def test_refusals():
    a, w = _codes((4, 128), 1), _codes((64, 128), 2)
    sa, sw = _scales((4, 1), 3), _scales((1, 1), 4)
    for bad in (lambda: moe.gemm_fp8_block(a.float(), sa, w, sw),
                lambda: moe.gemm_fp8_block(a, sa[:3], w, sw),
                lambda: moe.gemm_fp8_block(a, sa, w, sw.half()),
                lambda: moe.gemm_fp8_block(a, sa, w[:, :64], sw),
                lambda: moe.gemm_fp8_block(a, sa, w, sw, out_dtype=torch.float16),
                lambda: moe.gemm_fp8_block(a, sa, w, sw, out=torch.empty((4, 63), device="cuda")),
                lambda: moe.gemm_fp8_block(a.cpu(), sa, w, sw),
                lambda: moe.quantize_fp8_block(a),
                lambda: moe.quantize_fp8_block(torch.ones((2, 7), device="cuda"), gated=True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError) as e:  # K not a multiple of 16
        moe.gemm_fp8_block(_codes((4, 24), 1), sa, _codes((64, 24), 2), sw)
    assert e.value.status == _abi.MOE_ERR_UNSUPPORTED
    off = torch.empty(4 * 128 + 16, dtype=torch.uint8, device="cuda")[1:1 + 4 * 128].view(4, 128)
    with pytest.raises(moe.MoEError) as e:  # codes off the 16-byte alignment
        moe.gemm_fp8_block(off, sa, w, sw)
    assert e.value.status == _abi.MOE_ERR_INVALID_ARG
    assert moe.gemm_fp8_block(a[:0], sa[:0], w, sw).shape == (0, 64)
    ids = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    plan = moe.align(ids, 1, 16)
    cap = plan["sorted_ids"].numel()
    with pytest.raises(ValueError):  # another block size than the plan's
        moe.grouped_gemm_fp8_block(_codes((cap, 128), 1), _scales((cap, 1), 3), w[None], sw[None],
                                   plan, 32)
    with pytest.raises(ValueError):
        moe.grouped_gemm_fp8_block(a, sa, w[None], sw[None], plan, 16)


def test_checked_build_skips_blocks_outside_the_weights():
    L = _abi.checked_lib()
    plan = moe.align(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 1, 16)
    cap = plan["sorted_ids"].numel()
    a, w = _codes((cap, 128), 1), _codes((1, 64, 128), 2)
    sa, sw = _scales((cap, 1), 3), _scales((1, 1, 1), 4)
    info = plan["block_info"].clone()
    info[0, 0] = 3  # an expert that is not held
    out = torch.full((cap, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: t.data_ptr()
    assert L.moe_grouped_gemm_fp8_block(p(a), p(sa), p(w), p(sw), 1, 64, 128, cap, 16, p(info),
                                        p(plan["num_blocks"]), p(out), _abi.MOE_BF16, p(st),
                                        torch.cuda.current_stream().cuda_stream) == _abi.MOE_OK
    assert int(st.item()) == _abi.MOE_ERR_BOUNDS
    assert bool((out == 7).all())


# a multiple of four scale blocks to a row (loaded four at a time where rows
# start on 16 bytes)
@pytest.mark.parametrize("form", range(6))
@pytest.mark.parametrize("off", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", [(7, 264, 1536), (8, 200, 3584), (1, 64, 512)])
def test_gemm_scales_on_any_alignment(form, off, M, N, K):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sw = _scales((_nblk(N), _nblk(K)), 4)
    sa = torch.empty(M * _nblk(K) + off, device="cuda")[off:].view(M, _nblk(K))
    sa.copy_(_scales((M, _nblk(K)), 3))
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_BF16, form)
    _close(out, _dequant(a, sa), _dequant(w, sw, N), torch.bfloat16)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("M,N,K", [(130, 392, 2048), (300, 1000, 4608)])
def test_gemm_of_many_rows_with_scales_on_any_alignment(off, M, N, K):
    a, w = _codes((M, K), 1), _codes((N, K), 2)
    sw = _scales((_nblk(N), _nblk(K)), 4)
    sa = torch.empty(M * _nblk(K) + off, device="cuda")[off:].view(M, _nblk(K))
    sa.copy_(_scales((M, _nblk(K)), 3))
    for form in range(5):
        out = torch.empty((M, N), dtype=torch.float32, device="cuda")
        _abi.moe_test_gemm_fp8_block(a, sa, w, sw, M, N, K, out, _abi.MOE_F32, form)
        _close(out, _dequant(a, sa), _dequant(w, sw, N), torch.float32)
