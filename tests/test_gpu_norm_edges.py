"""The RMS norm's gradients over many rows and over values of any magnitude:
against the formulas in 64 bits, with the bounds of test_gpu_norm.py unless a test
derives its own."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import _abi
from test_gpu_norm import U, _grad_ref, _path, _rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _between(got, ref, d, dtype):
    assert got.dtype == dtype and got.shape == ref.shape
    bad = (got < (ref - d).to(dtype)) | (got > (ref + d).to(dtype)) | got.isnan()
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("H", [40, 257, 264, 1500, 1999, 2880, 2883, 4096, 8192])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stream_grad", [False, True])
def test_gradients_of_many_rows(H, dtype, stream_grad):
    """Seven rows or more to every team that is resident, and a remainder: rows fetched
    ahead at every depth, the slots gone round, and the weight gradient's terms
    carried from row to row.  That takes fewer additions on a path than rows there are:
    the team's rows, 8 in its CTA, the parts in 32 chains or more, 8 to join them."""
    parts = _abi.moe_rms_norm_backward_scratch_bytes(1 << 20, H) // (4 * H)
    teams = parts * (8 if H <= 512 else 1)
    T = 7 * teams + 3
    g = torch.Generator(device="cuda").manual_seed(H)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dy, h = rand(T, H).to(dtype), rand(T, H).to(dtype)
    ds = rand(T, H).to(dtype) if stream_grad else None
    w = 1 + 0.2 * rand(H)
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = moe.rms_norm_backward(dy, h, w, rstd, ds)
    ref, mag, terms = _grad_ref(dy, h, w, rstd, ds)
    _between(dx, ref, (_path(H) + 10) * U * mag, dtype)
    # CTAs may hold half as many rows at once in the other type or layout
    path = 2 * 8 + 8 + parts / 32 + 1 + 8 + 4
    _between(dw, terms.sum(0), path * U * terms.abs().sum(0), F32)
    if ds is not None:
        buf = ds.clone()
        again = moe.rms_norm_backward(dy, h, w, rstd, buf, out=buf)
        assert torch.equal(buf, dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("H", [200, 1999, 2880, 8192, 9000])
def test_gradients_of_values_of_any_magnitude(H):
    """Products of a row's values and their gradients that fp32 does not hold, or holds
    with few bits, of which the results have nothing."""
    for h_scale, dy_scale in ((1e25, 1e14), (1e-22, 1e-20), (1e30, 1e9), (1e-15, 1e-30),
                              (1e-10, 1e25), (1e25, 1e-10), (1e25, 1e-12)):
        h, dy = _rand((4, H), F32, 1, h_scale), _rand((4, H), F32, 2, dy_scale)
        w = _rand((H,), F32, 3)
        rstd = h.double().square().mean(1).rsqrt().float()
        dx, dw = moe.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
        ref, mag, terms = _grad_ref(dy, h, w, rstd, None)
        # results below 2^-126 have the bits of fp32's small numbers
        least = 2.0 ** -148
        _between(dx.cpu(), ref, (_path(H) + 10) * U * mag + least, F32)
        _between(dw.cpu(), terms.sum(0), 72 * U * terms.abs().sum(0) + least, F32)
