"""The permutation, quantiser and products on the streams and in the graphs a
caller has."""
import pytest
import torch

import mixture_experts_grouped_02_gb300 as moe
from mixture_experts_grouped_02_gb300 import permute

pytestmark = pytest.mark.gpu

# handles of the default stream: torch's (0) and the runtime's name for it (1)
DEFAULT = (0, 1)


@pytest.mark.parametrize("handle", DEFAULT)
def test_the_default_stream_by_its_handle(handle):
    """Buffers and inner calls of a call on the default stream's handle belong
    to that stream, and not to one of torch's pool."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with permute._on(handle):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        assert torch.cuda.current_stream() == side


def _layer(T, E, K, H, I):
    g = torch.Generator(device="cuda").manual_seed(0)

    def codes(*shape):
        v = torch.randn(shape, generator=g, device="cuda") * 110
        return v.clamp(-448, 448).to(torch.float8_e4m3fn)

    def scales(*shape):
        return 4e-4 * (0.1 + torch.rand(shape, generator=g, device="cuda"))

    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.topk(torch.randn(T, E, generator=g, device="cuda"), K).indices.to(torch.int32)
    tw = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    return x, ids, tw, (codes(E, 2 * I, H), scales(E, 2 * I // 128, H // 128), codes(E, H, I),
                        scales(E, H // 128, I // 128))


@pytest.mark.parametrize("handle", DEFAULT)
def test_a_layer_on_the_default_streams_handle_waits_for_its_input(handle):
    """The input arrives on the default stream some milliseconds after the
    call: a layer given that stream's handle computes the new one."""
    x, ids, tw, weights = _layer(40, 8, 2, 512, 256)
    want = moe.forward_fp8_block(x, ids, tw, *weights)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    late.copy_(x)
    got = moe.forward_fp8_block(late, ids, tw, *weights, stream=handle)
    assert torch.equal(got, want)
    torch.cuda._sleep(20_000_000)
    late.zero_()
    rows = moe.permute_tokens(late, moe.align(ids, 8, 16, stream=handle), stream=handle)
    assert bool((rows == 0).all())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_layer_and_its_permutation_in_a_graph(T):
    """Captured once and replayed on new inputs, as a caller does who cannot
    spend the host's time on every call."""
    E, K, H, I = 8, 2, 512, 256
    x, ids, tw, weights = _layer(T, E, K, H, I)
    g = torch.Generator(device="cuda").manual_seed(5)
    inputs = [(torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16),
               torch.topk(torch.randn(T, E, generator=g, device="cuda"), K).indices.int())
              for _ in range(3)]

    def step():
        out = moe.forward_fp8_block(x, ids, tw, *weights)
        plan = moe.align(ids, E, 16)
        rows = moe.permute_tokens(x, plan)
        dx = moe.permute_tokens_backward(rows, plan, K)
        y = moe.unpermute_tokens(rows, plan, tw)
        dy, dw = moe.unpermute_tokens_backward(y, rows, plan, tw)
        q, s = moe.quantize_fp8_block(x)
        gemm = moe.gemm_fp8_block(q, s, weights[0][0], weights[1][0])
        return out, rows, dx, y, dy, dw, q.view(torch.uint8), s, gemm

    step()  # what is looked up once per device
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for nx, nids in inputs:
        x.copy_(nx)
        ids.copy_(nids)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
