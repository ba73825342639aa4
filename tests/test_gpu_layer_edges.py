"""The norm, the router and the products on a stream that is given to them while
another one is current."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from test_gpu_layer import _rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("T", [5, 300])
def test_a_given_stream_beside_another_current_one(how, T):
    """Inputs that arrive late on the given stream: a launch, or a buffer's reuse, that
    went to the current one would meet zeros or be met too early."""
    H, E, K, I = 512, 16, 4, 136
    inputs = dict(x=_rand((T, H), 1), r=_rand((T, H), 2), norm=_rand((H,), 3, F32),
                  router=_rand((E, H), 4), w13=_rand((2 * I, H), 5, scale=0.05),
                  dl=_rand((T, E), 6), dh=_rand((T, I), 7), bias=_rand((2 * I,), 8, F32),
                  dw=_rand((T, K), 9, F32))

    def steps(v, stream=None):
        rstd, pre = v["rstd"], v["pre"]
        y, s = moe.rms_norm(v["x"], v["norm"], residual=v["r"], rstd=rstd, stream=stream)
        codes, scales, s2 = moe.rms_norm_fp8_block(v["x"], v["norm"], residual=v["r"],
                                                   stream=stream)
        logits = moe.linear(y, v["router"], out_dtype=F32, stream=stream)
        ids, tw = moe.route_tokens(logits, K, stream=stream)
        dl = moe.route_tokens_backward(v["dw"], logits, ids, stream=stream)
        h = moe.linear(y, v["w13"], v["bias"], "swiglu", preact=pre, stream=stream)
        back = moe.linear_backward(v["dh"], y, v["w13"], "swiglu", pre, bias=True, stream=stream)
        plain = moe.linear_backward(v["dl"], y, v["router"], bias=True, stream=stream)
        grads = moe.rms_norm_backward(back[0], s, v["norm"], rstd, plain[0], stream=stream)
        return (y, s, codes.view(torch.uint8), scales, s2, logits, ids, tw, dl, h, *back, *plain,
                *grads)

    def made(v):
        return {**v, "rstd": torch.zeros(T, device="cuda"),
                "pre": torch.zeros((T, 2 * I), dtype=BF16, device="cuda")}

    want = steps(made(inputs))
    late = made({k: torch.zeros_like(v) for k, v in inputs.items()})
    given, current = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(given):
        torch.cuda._sleep(50_000_000)
        for k, v in inputs.items():
            late[k].copy_(v)
    with torch.cuda.stream(current):
        got = steps(late, given if how == "stream" else given.cuda_stream)
        # what the given stream's buffers may not be reused for
        for t in want:
            torch.full_like(t, 1)
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
