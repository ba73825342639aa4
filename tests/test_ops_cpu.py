"""Refusals of the permutation, quantiser and block-scaled products that stop
on the host: no call of this file gets as far as a launch, so they run without
a GPU."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import _abi


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


# Pointers of the C entry points, none of which is followed: the calls below
# are refused by their argument checks.
A = 1 << 20
PERMUTE = dict(x=A, dtype=_abi.MOE_BF16, T=4, H=64, K=2, inv_perm=A, sorted_ids=A, cap=8,
               x_sorted=A, dev_status=A, stream=0)
PERMUTE_BACKWARD = dict(grad_sorted=A, dtype=_abi.MOE_BF16, T=4, H=64, K=2, inv_perm=A, cap=8,
                        grad_x=A, dev_status=A, stream=0)
UNPERMUTE = dict(y=A, dtype=_abi.MOE_BF16, T=4, H=64, K=2, topk_weights=A, inv_perm=A, cap=8,
                 out=A, dev_status=A, stream=0)
UNPERMUTE_BACKWARD = dict(grad_out=A, y=A, dtype=_abi.MOE_BF16, T=4, H=64, K=2, topk_weights=A,
                          inv_perm=A, sorted_ids=A, cap=8, grad_y=A, grad_weights=A, dev_status=A,
                          stream=0)
QUANTIZE = dict(x=A, x_dtype=_abi.MOE_BF16, T=4, H=64, gated=0, xq=A, scale=A, stream=0)
GEMM = dict(a=A, a_scale=A, w=A, w_scale=A, M=4, N=64, K=128, out=A, out_dtype=_abi.MOE_BF16,
            dev_status=A, stream=0)
GROUPED = dict(a=A, a_scale=A, w=A, w_scale=A, E=2, N=64, K=128, cap=32, block_m=16,
               block_info=A, num_blocks=A, out=A, out_dtype=_abi.MOE_BF16, dev_status=A, stream=0)
CALLS = dict(moe_permute_tokens=PERMUTE, moe_permute_tokens_backward=PERMUTE_BACKWARD,
             moe_unpermute_tokens=UNPERMUTE, moe_unpermute_tokens_backward=UNPERMUTE_BACKWARD,
             moe_quantize_fp8_block=QUANTIZE, moe_gemm_fp8_block=GEMM,
             moe_grouped_gemm_fp8_block=GROUPED)


def _refused(name, **changed):
    with pytest.raises(moe.MoEError) as e:
        getattr(_abi, name)(**{**CALLS[name], **changed})
    return e.value.status


WORDS = ("inv_perm", "sorted_ids", "topk_weights", "grad_weights", "scale", "a_scale", "w_scale",
         "block_info", "num_blocks", "dev_status")


@pytest.mark.parametrize("name,arg", [(n, a) for n, c in CALLS.items() for a in c
                                      if c[a] == A and a not in ("xq",)])
def test_pointers_off_their_alignment_are_refused(name, arg):
    """One byte off for every argument, two for the 4-byte words."""
    for off in (1, 2) if arg in WORDS else (1,):
        assert _refused(name, **{arg: A + off}) == _abi.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", CALLS)
def test_rows_near_2_31_columns_are_refused(name):
    """A CTA steps past a row's last column by up to its own width: column
    indexes of the widest rows would not stay in 32 bits."""
    arg = "K" if "gemm" in name else "H"
    for n in (2 ** 31 - 16, 2 ** 31 - 2048, 2 ** 31 - 4080):
        assert _refused(name, **{arg: n}) == _abi.MOE_ERR_UNSUPPORTED


class _On(torch.Tensor):
    """A CPU tensor that claims a GPU, and memory there."""
    gpu = 0

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return True


def _at(gpu, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_On)
    t.gpu = gpu
    return t


def _device_calls(gpu, other):
    """Every call with its first tensor on `gpu` and one later one on `other`."""
    i32, u8 = torch.int32, torch.uint8

    def plan(where):
        return dict(sorted_ids=_at(where, 32, dtype=i32), inv_perm=_at(where, 8, dtype=i32),
                    block_info=_at(where, 2, 4, dtype=i32), num_blocks=_at(where, 1, dtype=i32))

    x, y, w = _at(gpu, 4, 64), _at(gpu, 32, 64), _at(other, 4, 2)
    a, s = _at(gpu, 32, 128, dtype=u8), _at(gpu, 32, 1)
    weights, ws = _at(other, 2, 48, 128, dtype=u8), _at(gpu, 2, 1, 1)
    return [
        lambda: moe.permute_tokens(x, plan(other)),
        lambda: moe.permute_tokens_backward(y, plan(other), 2),
        lambda: moe.unpermute_tokens(y, plan(gpu), w),
        lambda: moe.unpermute_tokens_backward(x, y, plan(gpu), w),
        lambda: moe.quantize_fp8_block(x, out=(_at(other, 4, 64, dtype=u8), _at(gpu, 4, 1))),
        lambda: moe.gemm_fp8_block(a, s, _at(other, 48, 128, dtype=u8), _at(gpu, 1, 1)),
        lambda: moe.grouped_gemm_fp8_block(a, s, weights, ws, plan(gpu), 16),
        lambda: moe.forward_fp8_block(_at(gpu, 4, 128), _at(other, 4, 2, dtype=i32), w,
                                      _at(gpu, 2, 256, 128, dtype=u8), _at(gpu, 2, 2, 1),
                                      _at(gpu, 2, 128, 128, dtype=u8), _at(gpu, 2, 1, 1)),
    ]


@pytest.mark.parametrize("call", range(8))
def test_tensors_of_other_devices_are_refused(call, monkeypatch):
    """A launch takes the current device's kernels and stream: tensors that do
    not share it are refused before it."""
    class Library:
        def __getattr__(self, name):
            return lambda *args: pytest.fail(f"{name} was called")

    monkeypatch.setattr(_abi, "_device", lambda: 0)
    monkeypatch.setattr(_abi, "lib", Library)
    for first in (0, 1):
        with pytest.raises(ValueError, match="current device cuda:0, got one on cuda:1"):
            _device_calls(first, 1)[call]()


def test_pointers_of_an_int_subclass_are_taken():
    """A handle type of the caller's own, as every entry point has taken."""
    class Pointer(int):
        pass

    assert _abi._p(Pointer(A)) == A and _abi._p(A) == A and _abi._p(None) is None
    assert _refused("moe_quantize_fp8_block", x=Pointer(A + 1)) == _abi.MOE_ERR_INVALID_ARG
