"""The bf16 products over very long sums, at the ends of their activations and
beside a status word that is set while they start: against the formulas in 64 bits,
with the bounds of test_gpu_linear.py unless a test derives its own."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import _abi
from test_gpu_linear import _act, _between, _rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _long(x, w):
    """(x w^T, its tolerance) in 64 bits: accumulators of at most 65536 terms, taken 16
    at a time, each time cutting off at most 2^-23 of the largest magnitude they
    meet, and additions of what 32768 terms or more each sum to."""
    K = x.shape[1]
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    return z, (min(K, 65536) / 16 + 48 + K / 32768) * 2.0 ** -23 * mag


@pytest.mark.parametrize("form", [0, 1, 2, 4, 6, 7])
@pytest.mark.parametrize("layout", [0, 1, 2, "swiglu"])
@pytest.mark.parametrize("K", [65536, 65544, 458_760, 1 << 20])
def test_long_sums(form, layout, K):
    """Sums whose terms all have one sign, where one accumulator over all of K would
    end up 1.1e-9 K short: a quarter of a bf16 step for the longest."""
    gated, layout = layout == "swiglu", 0 if layout == "swiglu" else layout
    M, N = 136, 72
    x, w = _rand((M, K), 1).abs(), _rand((2 * N if gated else N, K), 2, scale=1 / K).abs()
    y, d = _long(x, w)
    if gated:
        y, d = _act(y, d, "swiglu")
    a = x.t().contiguous() if layout == 2 else x
    b = w.t().contiguous() if layout else w
    for dtype in (BF16, F32):
        out = torch.full((M, N), NAN, dtype=dtype, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _abi.moe_test_linear(a, b, M, N, K, layout, 3 if gated else 0, out, moe.dtype_code(dtype),
                             form, 0, status)
        assert int(status) == 0
        _between(out, y, d, dtype)


@pytest.mark.parametrize("T", [1 << 20, 1 << 22])
def test_weight_gradient_over_many_rows(T):
    """T rows of 64 columns: one accumulator would be 1.2e-3 and 4.6e-3 short, where a
    bf16 value is off by 2^-9 at most."""
    dy, x, w = _rand((T, 64), 1).abs(), _rand((T, 64), 2).abs(), _rand((64, 64), 3)
    _, dw, _ = moe.linear_backward(dy, x, w, need_x=False)
    ref, d = _long(dy.t(), x.t())
    _between(dw, ref, d, BF16)
    # with a sum of its own added in fp32, once
    held = _rand((64, 64), 4)
    buf = held.clone()
    moe.linear_backward(dy, x, w, need_x=False, grad_w=buf, accumulate=True)
    ref = ref + held.double()
    _between(buf, ref, d + 2.0 ** -24 * ref.abs(), BF16)


def test_tiles_of_224_columns_have_one_accumulator():
    x, w = _rand((8, 65544), 1), _rand((8, 65544), 2)
    out = torch.empty((8, 8), dtype=BF16, device="cuda")
    _abi.moe_test_linear(x[:, :65536].contiguous(), w[:, :65536].contiguous(), 8, 8, 65536, 0, 0,
                         out, _abi.MOE_BF16, 224)
    with pytest.raises(moe.MoEError) as e:
        _abi.moe_test_linear(x, w, 8, 8, 65544, 0, 0, out, _abi.MOE_BF16, 224)
    assert e.value.status == _abi.MOE_ERR_UNSUPPORTED


# z, SiLU(z) and its slope there
ENDS = [(INF, INF, 1.0), (-INF, 0.0, 0.0), (NAN, NAN, NAN), (1e38, 1e38, 1.0), (-1e38, 0.0, 0.0),
        (-100.0, 0.0, 0.0), (0.0, 0.0, 0.5), (-0.0, 0.0, 0.5)]


def _same(got, want):
    want = torch.tensor(want, device="cuda").to(got.dtype).expand_as(got)
    return torch.equal(got.nan_to_num(7.0, 3e38, -3e38), want.nan_to_num(7.0, 3e38, -3e38))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("n", [8, 7])
@pytest.mark.parametrize("M", [1, 300])
def test_silu_at_the_ends(dtype, act, n, M):
    """Infinities take the limits, inf and 0, in rows of words and of single elements."""
    x = torch.ones((M, 8), dtype=BF16, device="cuda")
    rows = 2 * n if act == "swiglu" else n
    for z, y, _ in ENDS:
        bias = torch.ones(rows, device="cuda")
        bias[:n] = torch.tensor(z).to(BF16).float()
        got = moe.linear(x, torch.zeros((rows, 8), dtype=BF16, device="cuda"), bias, act,
                         out_dtype=dtype)
        assert _same(got, torch.tensor(y).to(BF16).item()), z


@pytest.mark.parametrize("n", [8, 7])
def test_silus_slope_at_the_ends(n):
    """1 and 0 at the infinities; SwiGLU's gradients have SiLU and its slope."""
    for z, y, slope in ENDS:
        pre = torch.full((1, n), z, device="cuda").to(BF16)
        grad = torch.ones((1, n), dtype=BF16, device="cuda")
        dz = torch.empty((1, n), dtype=BF16, device="cuda")
        _abi.moe_linear_backward_act(grad, pre, 1, n, _abi.MOE_LINEAR_SILU, dz, None, None)
        assert _same(dz, slope), z
        both = torch.cat([pre, torch.full_like(pre, 2.0)], 1)
        dz = torch.empty((1, 2 * n), dtype=BF16, device="cuda")
        _abi.moe_linear_backward_act(grad, both, 1, n, _abi.MOE_LINEAR_SWIGLU, dz, None, None)
        assert _same(dz[:, :n], 2 * slope) and _same(dz[:, n:], torch.tensor(y).to(BF16).item()), z


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_a_status_word_that_is_set_meanwhile(M, act):
    """From another stream, while the CTAs of the kernel for few rows start: each stores
    its columns (16, SwiGLU: 8) whole and right, or leaves them alone."""
    N, K, each = 8192, 512, 8 if act else 16
    x, w = _rand((M, K), 1), _rand((2 * N if act else N, K), 2, scale=K ** -0.5)
    want = moe.linear(x, w, activation=act)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for wait in range(0, 6000, 60):
        status.zero_()
        out = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        moe.linear(x, w, activation=act, out=out, dev_status=status)
        with torch.cuda.stream(side):
            torch.cuda._sleep(wait)
            status.fill_(1)
        torch.cuda.synchronize()
        right, left = ((out == v).view(M, -1, each) for v in (want, 7.0))
        # a CTA has its columns of every row
        assert bool((right.all(2).all(0) | left.all(2).all(0)).all())
    moe.linear(x, w, activation=act, out=out.fill_(7.0), dev_status=status)
    assert bool((out == 7.0).all())
