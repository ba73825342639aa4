"""Refusals of the norm, the routing and the bf16 products that stop on the host: no
call of this file gets as far as a launch, so they run without a GPU."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import _abi

INVALID, UNSUPPORTED = _abi.MOE_ERR_INVALID_ARG, _abi.MOE_ERR_UNSUPPORTED
WORKSPACE = _abi.MOE_ERR_WORKSPACE
BF16, F32, E4M3 = _abi.MOE_BF16, _abi.MOE_F32, _abi.MOE_E4M3

# Pointers of the C entry points, none of which is followed: the calls below are
# refused by their argument checks.
A = 1 << 20
NORM = dict(x=A, residual=A, weight=A, dtype=BF16, weight_dtype=F32, T=4, H=64, eps=1e-6,
            sum_out=A, out=A, codes=A, scale=A, rstd=A, stream=0)
NORM_BACKWARD = dict(grad_out=A, h=A, weight=A, rstd=A, grad_sum=A, dtype=BF16, weight_dtype=BF16,
                     T=4, H=64, grad_x=A, grad_weight=A, scratch=A, scratch_bytes=1 << 30, stream=0)
ROUTE = dict(logits=A, logit_dtype=F32, bias=A, T=4, E=64, K=4, scores=0, num_groups=8,
             topk_groups=4, group_scores=0, renormalize=True, scale=1.0, topk_ids=A,
             topk_weights=A, dev_status=A, stream=0)
ROUTE_BACKWARD = dict(grad_weights=A, logits=A, logit_dtype=F32, topk_ids=A, T=4, E=64, K=4,
                      scores=0, renormalize=True, scale=1.0, grad_logits=A, dev_status=A, stream=0)
LINEAR = dict(x=A, w=A, bias=A, residual=A, M=40, N=64, K=128, activation=1, out=A, out_dtype=BF16,
              preact=A, dev_status=A, stream=0)
BACK_ACT = dict(grad_out=A, preact=A, M=40, N=64, activation=1, grad_preact=A, grad_bias=A,
                scratch=A, scratch_bytes=1 << 30, stream=0)
BACK_INPUT = dict(grad_preact=A, w=A, M=40, N=64, K=128, grad_x=A, out_dtype=BF16, dev_status=A,
                  stream=0)
BACK_WEIGHT = dict(grad_preact=A, x=A, M=40, N=64, K=128, grad_w=A, out_dtype=F32,
                   accumulate=True, dev_status=A, stream=0)
CALLS = dict(moe_rms_norm=NORM, moe_rms_norm_backward=NORM_BACKWARD, moe_route_tokens=ROUTE,
             moe_route_tokens_backward=ROUTE_BACKWARD, moe_linear=LINEAR,
             moe_linear_backward_act=BACK_ACT, moe_linear_backward_input=BACK_INPUT,
             moe_linear_backward_weight=BACK_WEIGHT)


def _refused(name, **changed):
    with pytest.raises(moe.MoEError) as e:
        getattr(_abi, name)(**{**CALLS[name], **changed})
    return e.value.status


WORDS = {"scale", "rstd", "grad_weight", "scratch", "bias", "topk_ids", "topk_weights",
         "grad_weights", "dev_status", "grad_bias"}
TILES = {("moe_linear", "x"), ("moe_linear", "w"), ("moe_linear_backward_input", "grad_preact"),
         ("moe_linear_backward_input", "w"), ("moe_linear_backward_weight", "grad_preact"),
         ("moe_linear_backward_weight", "x")}


@pytest.mark.parametrize("name,arg", [(n, a) for n, c in CALLS.items() for a in c
                                      if c[a] == A and a != "codes"])
def test_pointers_off_their_alignment_are_refused(name, arg):
    """One byte off for every argument, two for 4-byte words, eight for the tiles
    that TMA reads."""
    offs = [1] + ([2] if arg in WORDS else []) + ([2, 8] if (name, arg) in TILES else [])
    for off in offs:
        assert _refused(name, **{arg: A + off}) == INVALID


@pytest.mark.parametrize("name,arg", [
    ("moe_rms_norm", "x"), ("moe_rms_norm", "weight"), ("moe_rms_norm", "scale"),
    ("moe_rms_norm", "codes"), ("moe_rms_norm_backward", "grad_out"),
    ("moe_rms_norm_backward", "h"), ("moe_rms_norm_backward", "weight"),
    ("moe_rms_norm_backward", "rstd"), ("moe_rms_norm_backward", "grad_x"),
    ("moe_route_tokens", "logits"), ("moe_route_tokens", "topk_ids"),
    ("moe_route_tokens", "topk_weights"), ("moe_route_tokens_backward", "grad_weights"),
    ("moe_route_tokens_backward", "logits"), ("moe_route_tokens_backward", "topk_ids"),
    ("moe_route_tokens_backward", "grad_logits"), ("moe_linear", "x"), ("moe_linear", "w"),
    ("moe_linear", "out"), ("moe_linear_backward_act", "grad_out"),
    ("moe_linear_backward_act", "preact"), ("moe_linear_backward_act", "grad_preact"),
    ("moe_linear_backward_input", "grad_preact"), ("moe_linear_backward_input", "w"),
    ("moe_linear_backward_input", "grad_x"), ("moe_linear_backward_weight", "grad_preact"),
    ("moe_linear_backward_weight", "x"), ("moe_linear_backward_weight", "grad_w")])
def test_missing_pointers_are_refused(name, arg):
    assert _refused(name, **{arg: None}) == INVALID


def test_a_norm_without_an_output_is_refused():
    assert _refused("moe_rms_norm", out=None, codes=None, scale=None) == INVALID


@pytest.mark.parametrize("name", ["moe_rms_norm_backward", "moe_linear_backward_act"])
def test_a_small_or_missing_scratch_is_refused(name):
    assert _refused(name, scratch=None) == WORKSPACE
    assert _refused(name, scratch_bytes=4) == WORKSPACE


SIZES = [(n, a, v, s) for n, c in CALLS.items() for a, v, s in (
    ("T", -1, INVALID), ("H", 0, INVALID), ("H", -3, INVALID), ("H", 2 ** 31 - 4095, UNSUPPORTED),
    ("H", 2 ** 31 - 1, UNSUPPORTED), ("E", 0, INVALID), ("E", 1032, UNSUPPORTED),
    ("K", 0, INVALID), ("M", -1, INVALID), ("N", 0, INVALID),
    ("eps", -1e-6, INVALID), ("eps", float("nan"), INVALID), ("eps", float("inf"), INVALID),
    ("scale", float("nan"), INVALID), ("scores", 2, INVALID), ("group_scores", 2, INVALID),
    ("dtype", E4M3, INVALID), ("weight_dtype", E4M3, INVALID), ("logit_dtype", E4M3, INVALID),
    ("out_dtype", E4M3, INVALID), ("activation", 4, INVALID), ("activation", -1, INVALID)) if a in c
    and not (a == "scale" and "codes" in c)]


@pytest.mark.parametrize("name,arg,value,status", SIZES)
def test_sizes_and_choices_are_refused(name, arg, value, status):
    assert _refused(name, **{arg: value}) == status


def test_routing_refusals():
    r = "moe_route_tokens"
    assert _refused(r, K=33, num_groups=1, topk_groups=1) == UNSUPPORTED
    assert _refused("moe_route_tokens_backward", K=33) == UNSUPPORTED
    assert _refused(r, num_groups=0) == INVALID
    assert _refused(r, num_groups=7) == INVALID  # no divisor of 64
    assert _refused(r, topk_groups=0) == INVALID
    assert _refused(r, topk_groups=9) == INVALID
    assert _refused(r, num_groups=64, topk_groups=64) == UNSUPPORTED
    assert _refused(r, topk_groups=1, K=9) == INVALID  # a group has 8
    assert _refused(r, num_groups=1, topk_groups=1, E=3, K=4) == INVALID


def test_product_refusals():
    """Rows that do not start on 16 bytes, and sizes past what TMA and tile indexes
    count."""
    for k in (129, 132, 4):
        assert _refused("moe_linear", K=k) == UNSUPPORTED
        assert _refused("moe_linear_backward_input", K=k) == UNSUPPORTED
        assert _refused("moe_linear_backward_weight", K=k) == UNSUPPORTED
        assert _refused("moe_linear_backward_input", N=k) == UNSUPPORTED
        assert _refused("moe_linear_backward_weight", N=k) == UNSUPPORTED
    big = 2 ** 30 - 4088
    assert _refused("moe_linear", K=big) == UNSUPPORTED
    assert _refused("moe_linear", N=big // 2) == UNSUPPORTED
    assert _refused("moe_linear", M=2 ** 31 - 512) == UNSUPPORTED
    assert _refused("moe_linear", M=2 ** 31 - 1024, N=2 ** 29 - 4096) == UNSUPPORTED
    assert _refused("moe_linear_backward_input", K=big // 2) == UNSUPPORTED
    assert _refused("moe_linear_backward_weight", M=big) == UNSUPPORTED
    longer = 2 ** 27 + 8  # sums that a bounded wait would not outlast
    assert _refused("moe_linear", K=longer) == UNSUPPORTED
    assert _refused("moe_linear_backward_input", N=longer) == UNSUPPORTED
    assert _refused("moe_linear_backward_weight", M=longer) == UNSUPPORTED
    for form in (-1, 8):
        with pytest.raises(moe.MoEError):
            _abi.moe_test_linear(A, A, 8, 8, 64, 0, 0, A, BF16, form, 0, None, 0)


# ------------------------------------------------------ what the helpers refuse

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


X, W32 = _t(4, 64), _t(64, dtype=torch.float32)
REFUSED = [
    (lambda: moe.rms_norm(X.half(), W32), "unsupported dtype"),
    (lambda: moe.rms_norm(X, _t(63)), "weight"),
    (lambda: moe.rms_norm(X, W32.half()), "unsupported dtype"),
    (lambda: moe.rms_norm(X, W32, residual=_t(4, 63)), "residual"),
    (lambda: moe.rms_norm(X, W32, residual=X.float()), "residual"),
    (lambda: moe.rms_norm(X, W32, sum_out=X), "sum_out without a residual"),
    (lambda: moe.rms_norm(X, W32, rstd=_t(4)), "rstd"),
    (lambda: moe.rms_norm(X, W32, out=_t(3, 64)), "out"),
    (lambda: moe.rms_norm_fp8_block(X, W32, normed=X.float()), "normed"),
    (lambda: moe.rms_norm_fp8_block(X, W32, out=(X, W32)), "out codes"),
    (lambda: moe.rms_norm_backward(X, X, W32, None), "rstd"),
    (lambda: moe.rms_norm_backward(X.float(), X, W32, _t(4, dtype=torch.float32)), "grad_out"),
    (lambda: moe.rms_norm_backward(X, X, W32, _t(4, dtype=torch.float32), grad_weight=_t(64)),
     "grad_weight"),
    (lambda: moe.route_tokens(_t(4, 8), 2, scores="relu"), "scores"),
    (lambda: moe.route_tokens(_t(4, 8), 2, group_scores="mean"), "group_scores"),
    (lambda: moe.route_tokens(_t(4, 8), 2, bias=_t(8)), "bias"),
    (lambda: moe.route_tokens(_t(4, 8).half(), 2), "unsupported dtype"),
    (lambda: moe.route_tokens_backward(_t(4, 2), _t(4, 8), _t(4, 2, dtype=torch.int32)),
     "grad_weights"),
    (lambda: moe.route_tokens_backward(_t(4, 2, dtype=torch.float32), _t(4, 8), _t(4, 2)),
     "topk_ids"),
    (lambda: moe.linear(X.float(), _t(8, 64)), "x: expected a 2-D bfloat16"),
    (lambda: moe.linear(X, _t(8, 63)), "w: expected 64 columns"),
    (lambda: moe.linear(X, _t(8, 64), activation="tanh"), "activation"),
    (lambda: moe.linear(X, _t(9, 64), activation="swiglu"), "gate and up"),
    (lambda: moe.linear(X, _t(8, 64), bias=_t(8)), "bias"),
    (lambda: moe.linear(X, _t(8, 64), residual=_t(4, 8, dtype=torch.float32)), "residual"),
    (lambda: moe.linear(X, _t(8, 64), out_dtype=torch.float16), "unsupported dtype"),
    (lambda: moe.linear(X, _t(8, 64), activation="silu", preact=_t(4, 9)), "preact"),
    (lambda: moe.linear_backward(_t(4, 8), X, _t(8, 64), "silu"), "preact"),
    (lambda: moe.linear_backward(_t(4, 9), X, _t(8, 64)), "grad_out"),
    (lambda: moe.linear_backward(_t(4, 8), X, _t(8, 64), accumulate=True), "accumulate"),
    (lambda: moe.linear_backward(_t(4, 8), X, _t(8, 64), grad_w=_t(8, 63)), "grad_w"),
]


@pytest.mark.parametrize("call", range(len(REFUSED)))
def test_helpers_refuse(call):
    with pytest.raises(ValueError, match=REFUSED[call][1]):
        REFUSED[call][0]()


# ------------------------------------------------------------- other devices

class _On(torch.Tensor):
    """A CPU tensor that claims a GPU, and memory there."""
    gpu = 0

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return True


def _at(gpu, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_On)
    t.gpu = gpu
    return t


def _device_calls(gpu, other):
    """Every call with its first tensor on `gpu` and one later one on `other`."""
    f32, i32 = torch.float32, torch.int32
    x, w = _at(gpu, 4, 64), _at(other, 64, dtype=f32)
    logits, k2 = _at(gpu, 4, 8, dtype=f32), _at(gpu, 4, 2, dtype=f32)
    return [
        lambda: moe.rms_norm(x, w),
        lambda: moe.rms_norm_fp8_block(x, _at(gpu, 64), residual=_at(other, 4, 64)),
        lambda: moe.rms_norm_backward(x, x, w, _at(gpu, 4, dtype=f32), grad_weight=False),
        lambda: moe.route_tokens(logits, 2, bias=_at(other, 8, dtype=f32)),
        lambda: moe.route_tokens_backward(k2, logits, _at(other, 4, 2, dtype=i32)),
        lambda: moe.linear(x, _at(other, 8, 64)),
        lambda: moe.linear_backward(_at(gpu, 4, 8), x, _at(other, 8, 64)),
        lambda: moe.linear_backward(_at(gpu, 4, 8), x, _at(gpu, 8, 64), "silu", _at(other, 4, 8)),
    ]


@pytest.mark.parametrize("call", range(8))
def test_tensors_of_other_devices_are_refused(call, monkeypatch):
    class Library:
        def __getattr__(self, name):
            if name.endswith("_scratch_bytes"):
                return lambda *args: 0
            return lambda *args: pytest.fail(f"{name} was called")

    monkeypatch.setattr(_abi, "_device", lambda: 0)
    monkeypatch.setattr(_abi, "lib", Library)
    for first in (0, 1):
        with pytest.raises(ValueError, match="current device cuda:0, got one on cuda:1"):
            _device_calls(first, 1)[call]()


def test_other_layouts_are_refused(monkeypatch):
    """Rows that are not dense are no rows of these calls."""
    monkeypatch.setattr(_abi, "_device", lambda: 0)
    x = _at(0, 64, 4)
    with pytest.raises(ValueError, match="contiguous"):
        moe.rms_norm(x.t(), _at(0, 64))


def test_scratch_sizes_without_rows():
    assert _abi.moe_rms_norm_backward_scratch_bytes(0, 64) == 0
    assert _abi.moe_linear_backward_act_scratch_bytes(0, 64, 1) == 0
    assert _abi.moe_linear_backward_act_scratch_bytes(8, 64, 9) == 0


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_columns_of_grad_preact_past_what_tma_counts_are_refused(out_dtype, accumulate):
    """They lie along the operand's rows, whose TMA coordinate is of 2 N bytes and the
    tile's past them, in 32 bits."""
    for n in (2 ** 30 - 4088, 2 ** 30, 2 ** 30 + 8, 2 ** 31 - 1024):
        assert _refused("moe_linear_backward_weight", N=n, K=8, M=1, out_dtype=out_dtype,
                        accumulate=accumulate) == UNSUPPORTED
        for form in (0, 7):
            with pytest.raises(moe.MoEError) as e:
                _abi.moe_test_linear(A, A, n, 8, 8, 2, 0, A, out_dtype, form, 0, None, 0)
            assert e.value.status == UNSUPPORTED
