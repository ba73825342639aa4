"""The RMS norm's gradients over values of any magnitude: against the formulas in 64
bits, with the bounds of test_gpu_norm.py unless a test derives its own."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from test_gpu_norm import U, _grad_ref, _path, _rand

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _between(got, ref, d, dtype):
    assert got.dtype == dtype and got.shape == ref.shape
    bad = (got < (ref - d).to(dtype)) | (got > (ref + d).to(dtype)) | got.isnan()
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("H", [200, 1999, 2880, 8192, 9000])
def test_gradients_of_values_of_any_magnitude(H):
    """Products of a row's values and their gradients that fp32 does not hold, or holds
    with few bits, of which the results have nothing."""
    for h_scale, dy_scale in ((1e25, 1e14), (1e-22, 1e-20), (1e30, 1e9), (1e-15, 1e-30),
                              (1e-10, 1e25), (1e25, 1e-10)):
        h, dy = _rand((4, H), F32, 1, h_scale), _rand((4, H), F32, 2, dy_scale)
        w = _rand((H,), F32, 3)
        rstd = h.double().square().mean(1).rsqrt().float()
        dx, dw = moe.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda())
        ref, mag, terms = _grad_ref(dy, h, w, rstd, None)
        # results below 2^-126 have the bits of fp32's small numbers
        least = 2.0 ** -148
        _between(dx.cpu(), ref, (_path(H) + 10) * U * mag + least, F32)
        _between(dw.cpu(), terms.sum(0), 72 * U * terms.abs().sum(0) + least, F32)
