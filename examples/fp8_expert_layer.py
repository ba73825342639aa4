"""The token permutation, the 128-block fp8 quantiser and the block-scaled fp8
products used together, on a GB300:

* serving: an MoE layer whose expert weights are e4m3 with a scale per 128 x
  128 block (DeepSeek-V3's checkpoint format), compared with moe_forward on
  the same weights in bf16, from one token to a prefill batch;
* training: a step through experts of the user's own, with the permutation
  and its gradients around them as autograd functions.

    python examples/fp8_expert_layer.py [--hidden 7168 --inter 2048 --experts 32 --topk 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_grouped_02_gb300 as moe  # noqa: E402


def quantize_weights(w):
    """(codes, scales) of w (E, N, K) in 128 x 128 blocks."""
    E, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.zeros((E, nb * 128, kb * 128), device=w.device)
    p[:, :N, :K] = w
    b = p.view(E, nb, 128, kb, 128)
    scale = b.abs().amax((2, 4)).clamp(min=2.0 ** -100) / 448.0
    q = (b / scale[:, :, None, :, None]).clamp(-448, 448).reshape(E, nb * 128, kb * 128)
    return q[:, :N, :K].to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def dequantize_weights(q, scale):
    full = scale.repeat_interleave(128, 1).repeat_interleave(128, 2)
    return (q.float() * full[:, :q.shape[1], :q.shape[2]]).to(torch.bfloat16)


def route(logits, K):
    v, ids = torch.topk(logits, K, dim=1)
    return ids.to(torch.int32), torch.softmax(v.float(), 1)


def us_per_call(f, n=20):
    for _ in range(3):
        f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(n):
        f()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) * 1e3 / n


def serve(H, I, E, K, tokens):
    """Relative L2 distance of the fp8 layer from the bf16 one, per batch size."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    w13, s13 = quantize_weights(rand(E, 2 * I, H) / H ** 0.5)
    w2, s2 = quantize_weights(rand(E, H, I) / I ** 0.5)
    w13_bf16, w2_bf16 = dequantize_weights(w13, s13), dequantize_weights(w2, s2)
    distances = []
    for T in tokens:
        x = rand(T, H).to(torch.bfloat16)
        ids, weights = route(rand(T, E), K)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fp8 = lambda: moe.forward_fp8_block(x, ids, weights, w13, s13, w2, s2, dev_status=status)
        bf16 = lambda: moe.forward(x, ids, weights, w13_bf16, w2_bf16)
        a, b = fp8().float(), bf16().float()
        if moe.moe_get_device_status(status) != 0:
            raise RuntimeError("the fp8 layer reported an error")
        distances.append(float((a - b).norm() / b.norm()))
        print(f"T={T:5d}: fp8 {us_per_call(fp8):8.1f} us, bf16 {us_per_call(bf16):8.1f} us, "
              f"relative L2 distance {distances[-1]:.3f}")
    return distances


class Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan, K):
        ctx.plan, ctx.K = plan, K
        return moe.permute_tokens(x, plan)

    @staticmethod
    def backward(ctx, grad):
        return moe.permute_tokens_backward(grad.contiguous(), ctx.plan, ctx.K), None, None


class Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, plan):
        ctx.plan = plan
        ctx.save_for_backward(y, weights)
        return moe.unpermute_tokens(y, plan, weights)

    @staticmethod
    def backward(ctx, grad):
        y, weights = ctx.saved_tensors
        gy, gw = moe.unpermute_tokens_backward(grad.contiguous(), y, ctx.plan, weights)
        return gy, gw, None


def train(H, I, E, K, T, steps=3):
    """Loss before each of a few steps of SGD on the router and on experts of
    one matrix each, towards a random target."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda")
    target = torch.randn(T, I, generator=g, device="cuda")
    router = (torch.randn(H, E, generator=g, device="cuda") / H ** 0.5).requires_grad_()
    experts = (torch.randn(E, H, I, generator=g, device="cuda") / H ** 0.5).requires_grad_()
    losses = []
    for _ in range(steps):
        v, ids = torch.topk(x @ router, K, dim=1)
        weights = torch.softmax(v, 1)
        plan = moe.align(ids.to(torch.int32), E, 16)
        rows = Permute.apply(x, plan, K)
        # every block of 16 slots belongs to one expert
        expert = plan["block_info"][:, 0].clamp(min=0).long()
        blocks = rows[:expert.numel() * 16].view(-1, 16, H)
        y = torch.bmm(blocks, experts[expert]).view(-1, I)
        pad = rows.shape[0] - y.shape[0]
        y = torch.nn.functional.pad(y, (0, 0, 0, pad))
        out = Unpermute.apply(y, weights, plan)
        loss = (out - target).square().mean()
        loss.backward()
        losses.append(float(loss.detach()))
        with torch.no_grad():
            for p in (router, experts):
                p -= 20.0 * p.grad
                p.grad = None
    print("training loss:", " ".join(f"{v:.4f}" for v in losses))
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 8, 128, 2048])
    a = ap.parse_args(argv)
    distances = serve(a.hidden, a.inter, a.experts, a.topk, a.tokens)
    losses = train(256, 128, a.experts, a.topk, 512)
    return distances, losses


if __name__ == "__main__":
    main()
