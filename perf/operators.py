"""Cases of the token permutation and of the block-scaled fp8 products.

Operators (``op`` of a case):

``permute``    token rows to the expert-sorted, block-padded list, padding rows
               zero; ``train`` adds its gradient (the sum of a token's copies).
``unpermute``  sorted rows back to tokens with the routing weights applied;
               ``train`` adds the gradients of the rows and of the weights.
``quantize``   rows to e4m3 codes with one fp32 scale per 128 columns, of the
               input itself or of SiLU(gate) * up.
``gemm``       a product of e4m3 operands with fp32 scales per 128 columns of
               a row (activations) and per 128 x 128 block (weights).
``grouped``    the same product for every expert of a sorted list.

``run`` computes a case in elementary torch operations, or, with ``own`` set,
by the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128
AMAX_FLOOR = 2.0 ** -100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a DeepSeek-V3-shaped layer on its way to 8 of 256 experts
        dict(name="permute_decode", op="permute", mode="fwd", T=1, H=7168, K=8, E=256, block_m=16,
             dtype="bf16", routing="zipf"),
        # the same layer's training batch, forward and gradient
        dict(name="permute_train", op="permute", mode="train", T=8192, H=7168, K=8, E=256,
             block_m=128, dtype="bf16", routing="zipf"),
        # a decode batch of a Mixtral-shaped layer, back to its tokens
        dict(name="unpermute_decode", op="unpermute", mode="fwd", T=32, H=4096, K=2, E=8,
             block_m=16, dtype="bf16", routing="normal"),
        # training batches: fp32 rows with an odd token count, and bf16 rows
        dict(name="unpermute_train_f32", op="unpermute", mode="train", T=4095, H=4096, K=2, E=8,
             block_m=256, dtype="f32", routing="normal"),
        dict(name="unpermute_train", op="unpermute", mode="train", T=8192, H=7168, K=8, E=256,
             block_m=128, dtype="bf16", routing="zipf"),
        # a decode batch's activations, and the hidden activation of a prefill shard
        dict(name="quantize_decode", op="quantize", gated=False, T=8, H=7168, dtype="bf16"),
        dict(name="quantize_silu_prefill", op="quantize", gated=True, T=16411, H=2048,
             dtype="bf16"),
        # a shared expert's down projection for one token
        dict(name="gemm_single_token", op="gemm", M=1, N=7168, K=2048),
        # odd row count, and widths that end inside a scale block
        dict(name="gemm_ragged", op="gemm", M=333, N=2880, K=2880),
        # a shared expert's gate/up projection over a prefill batch
        dict(name="gemm_prefill", op="gemm", M=8192, N=4096, K=7168),
        # gate/up of eight tokens over 256 experts: the active experts' weights are streamed
        dict(name="grouped_decode", op="grouped", T=8, TopK=8, E=256, N=4096, K=7168, block_m=16,
             routing="zipf"),
        # gate/up of an expert shard's share of a prefill batch, skewed over 32 experts
        dict(name="grouped_prefill", op="grouped", T=1024, TopK=8, E=32, N=4096, K=7168,
             block_m=128, routing="zipf"),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n if n % 1536 else n + 1


def _width(rng, lo, hi, step):
    """A multiple of `step`, but none of 1536; half of the time one of 128."""
    step = BLOCK if rng.random() < 0.5 else step
    n = max(lo, min(hi, _log_int(rng, lo, hi) // step * step))
    return n if n % 1536 else n + step


def draw(rng):
    op = rng.choice(["permute", "unpermute", "quantize", "gemm", "gemm", "grouped", "grouped"])
    if op in ("permute", "unpermute"):
        E = rng.choice([4, 8, 32, 60, 128, 256])
        # rows of an odd number of elements among them
        H = rng.randrange(129, 2001, 2) if rng.random() < 0.15 else _width(rng, 128, 7168, 8)
        return dict(op=op, mode=rng.choice(["fwd", "train"]), T=_log_int(rng, 1, 8192), H=H,
                    K=rng.randint(1, min(8, E)), E=E, block_m=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    routing=rng.choice(["normal", "zipf"]))
    if op == "quantize":
        H = rng.randrange(129, 2001, 2) if rng.random() < 0.15 else _width(rng, 128, 7168, 8)
        return dict(op=op, gated=rng.random() < 0.5, T=_log_int(rng, 1, 16384), H=H,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gemm":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_width(rng, 64, 4096, 8),
                    K=_width(rng, 128, 7168, 16))
    return dict(op=op, T=_log_int(rng, 1, 1024), TopK=rng.randint(1, 8),
                E=rng.choice([8, 16, 32]), N=_width(rng, 64, 4096, 8),
                K=_width(rng, 128, 7168, 16), block_m=rng.choice([16, 32, 64, 128]),
                routing=rng.choice(["normal", "zipf"]))


# ----------------------------------------------------------------- inputs

def _popularity(E, routing):
    """Expert probabilities by rank: equal, or proportional to rank^-1.1."""
    p = torch.ones(E, dtype=torch.float64)
    if routing == "zipf":
        p = torch.arange(1, E + 1, dtype=torch.float64).pow(-1.1)
    return p / p.sum()


def _route(T, K, E, routing, g):
    """Top-k ids (T, K) and renormalised weights of random router logits."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = _popularity(E, routing).log().to("cuda", torch.float32)
    logits += bias[torch.randperm(E, generator=g, device="cuda")]
    v, ids = torch.topk(logits, K, dim=1)
    return ids, torch.softmax(v, dim=1)


def _plan(ids, E, block_m):
    """The expert-sorted, block-padded list of the ids (T, K): for flat index
    i = t*K + k, inv_perm[i] is its slot and sorted_ids[slot] = i (T*K in
    padding slots); block_info holds {expert, block, first slot, valid rows}."""
    flat = ids.reshape(-1)
    n, dev = flat.numel(), flat.device
    cap = n + min(E, n) * (block_m - 1)
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + block_m - 1) // block_m * block_m
    first = torch.cumsum(counts, 0) - counts
    pfirst = torch.cumsum(padded, 0) - padded
    order = torch.argsort(flat, stable=True)
    e = flat[order]
    slots = pfirst[e] + torch.arange(n, device=dev) - first[e]
    inv = torch.empty(n, dtype=torch.int32, device=dev)
    inv[order] = slots.to(torch.int32)
    sorted_ids = torch.full((cap,), n, dtype=torch.int32, device=dev)
    sorted_ids[slots] = order.to(torch.int32)
    nb = padded.sum() // block_m
    row = torch.arange(cap // block_m, device=dev) * block_m
    be = torch.searchsorted(pfirst + padded, row, right=True).clamp(max=E - 1)
    m = (row - pfirst[be]) // block_m
    info = torch.stack([be, m, row, (counts[be] - m * block_m).clamp(max=block_m)], 1)
    info[row >= nb * block_m] = torch.tensor([-1, 0, 0, 0], device=dev)
    return dict(sorted_ids=sorted_ids, inv_perm=inv,
                block_info=info.to(torch.int32).contiguous(),
                num_blocks=nb.to(torch.int32).reshape(1))


def _codes(shape, g):
    """e4m3 codes of normal values whose block maximum sits near the largest code."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(110.0)
    return v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)


def _scales(shape, g, k):
    """Positive fp32 scales that make products of `k` terms of the order of one."""
    u = torch.rand(shape, generator=g, device="cuda")
    return (0.5 + u) / (110.0 * k ** 0.25)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    s = dict(case=c)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(DTYPES[c["dtype"]])

    if c["op"] in ("permute", "unpermute"):
        ids, weights = _route(c["T"], c["K"], c["E"], c["routing"], g)
        s["plan"] = _plan(ids, c["E"], c["block_m"])
        rows = s["plan"]["sorted_ids"].numel()
        if c["op"] == "permute":
            s["x"] = rand(c["T"], c["H"])
            if c["mode"] == "train":
                s["grad"] = rand(rows, c["H"])
        else:
            s["y"] = rand(rows, c["H"])
            s["weights"] = weights.contiguous()
            if c["mode"] == "train":
                s["grad"] = rand(c["T"], c["H"])
    elif c["op"] == "quantize":
        x = rand(c["T"], (2 if c["gated"] else 1) * c["H"])
        # some channels are far larger than the rest, as in trained models
        hot = torch.rand(x.shape[1], generator=g, device="cuda") < 0.01
        s["x"] = torch.where(hot, x * 8, x)
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["a"], s["b"] = _codes((M, K), g), _codes((N, K), g)
        s["a_scale"] = _scales((M, -(-K // BLOCK)), g, K)
        s["b_scale"] = _scales((-(-N // BLOCK), -(-K // BLOCK)), g, K)
    else:
        N, K, E = c["N"], c["K"], c["E"]
        ids, _ = _route(c["T"], c["TopK"], E, c["routing"], g)
        s["plan"] = _plan(ids, E, c["block_m"])
        rows = s["plan"]["sorted_ids"].numel()
        s["a"] = _codes((rows, K), g)
        s["a_scale"] = _scales((rows, -(-K // BLOCK)), g, K)
        s["b"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            s["b"][e] = _codes((N, K), g)
        s["b_scale"] = _scales((E, -(-N // BLOCK), -(-K // BLOCK)), g, K)
        # the layer's output buffer; rows of padding slots stay zero
        s["out"] = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _slot_rows(plan, n):
    """Which slots hold an assignment, and their flat index (0 elsewhere)."""
    valid = plan["sorted_ids"] < n
    return valid[:, None], torch.where(valid, plan["sorted_ids"], 0).long()


def _permute(x, plan, K):
    valid, i = _slot_rows(plan, x.shape[0] * K)
    return torch.where(valid, x.float()[i // K], 0.0).to(x.dtype)


def _gathered(rows, plan, K):
    """The rows of every token's K assignments, (T, K, H) in fp32."""
    return rows.float()[plan["inv_perm"].long()].view(-1, K, rows.shape[1])


def _unpermute_backward(grad, y, plan, w):
    T, K = w.shape
    valid, i = _slot_rows(plan, T * K)
    dy = torch.where(valid, w.reshape(-1)[i][:, None] * grad.float()[i // K], 0.0).to(y.dtype)
    dw = (grad.float()[:, None, :] * _gathered(y, plan, K)).sum(-1)
    return dy, dw


def _blocks(x):
    """(T, H) as (T, blocks, 128), zero past H."""
    T, H = x.shape
    nb = -(-H // BLOCK)
    p = torch.zeros((T, nb * BLOCK), dtype=x.dtype, device=x.device)
    p[:, :H] = x
    return p.view(T, nb, BLOCK)


def _quantize(x, gated):
    x = x.float()
    if gated:
        gate, up = x.chunk(2, dim=1)
        x = gate / (1.0 + torch.exp(-gate)) * up
    b = _blocks(x)
    amax = b.abs().amax(-1).clamp(min=AMAX_FLOOR)
    q = (b * (448.0 / amax)[..., None]).clamp(-448.0, 448.0)
    q = q.reshape(x.shape[0], -1)[:, :x.shape[1]].to(torch.float8_e4m3fn)
    return q.contiguous(), amax / 448.0


def _spread(scale, rows, cols):
    """Scales per 128 columns (and, with `rows`, per 128 rows) as one per element."""
    scale = scale.repeat_interleave(BLOCK, dim=-1)[..., :cols]
    if rows is not None:
        scale = scale.repeat_interleave(BLOCK, dim=-2)[..., :rows, :]
    return scale


def _gemm(a, a_scale, b, b_scale):
    af = a.float().mul_(_spread(a_scale, None, a.shape[1]))
    bf = b.float().mul_(_spread(b_scale, b.shape[0], b.shape[1]))
    return (af @ bf.t()).to(torch.bfloat16)


def _grouped(a, a_scale, b, b_scale, plan, block_m, out):
    info = plan["block_info"].long()
    nb = info.shape[0]
    expert = info[:, 0].clamp(min=0)
    rows = info[:, 2:3] + torch.arange(block_m, device=a.device)
    live = torch.arange(block_m, device=a.device) < info[:, 3:4]
    rows = torch.where(live, rows, 0)
    af = a.float().mul_(_spread(a_scale, None, a.shape[1]))[rows.reshape(-1)]
    bf = b.view(torch.uint8)[expert].view(torch.float8_e4m3fn).float()
    bf.view(torch.float32).mul_(_spread(b_scale[expert], b.shape[1], b.shape[2]))
    y = torch.bmm(af.view(nb, block_m, -1), bf.transpose(1, 2))
    y = torch.where(live[..., None], y, 0.0).to(out.dtype).view(nb * block_m, -1)
    # blocks lie one behind the other in the list; past the last one there are no rows
    out.zero_()
    out[:nb * block_m] = y
    return out


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _run_own(s, c, op)
    if op == "permute":
        out = dict(rows=_permute(s["x"], s["plan"], c["K"]))
        if c["mode"] == "train":
            out["dx"] = _gathered(s["grad"], s["plan"], c["K"]).sum(1).to(s["x"].dtype)
        return out
    if op == "unpermute":
        w = s["weights"]
        g = _gathered(s["y"], s["plan"], c["K"])
        out = dict(out=(w[..., None] * g).sum(1).to(s["y"].dtype))
        if c["mode"] == "train":
            out["dy"], out["dw"] = _unpermute_backward(s["grad"], s["y"], s["plan"], w)
        return out
    if op == "quantize":
        q, scale = _quantize(s["x"], c["gated"])
        return dict(codes=q, scale=scale)
    if op == "gemm":
        return dict(out=_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"]))
    return dict(out=_grouped(s["a"], s["a_scale"], s["b"], s["b_scale"], s["plan"],
                             c["block_m"], s["out"]))


def _run_own(s, c, op):
    import mixture_experts_grouped_02_gb300 as moe
    if op == "permute":
        out = dict(rows=moe.permute_tokens(s["x"], s["plan"]))
        if c["mode"] == "train":
            out["dx"] = moe.permute_tokens_backward(s["grad"], s["plan"], c["K"])
        return out
    if op == "unpermute":
        out = dict(out=moe.unpermute_tokens(s["y"], s["plan"], s["weights"]))
        if c["mode"] == "train":
            out["dy"], out["dw"] = moe.unpermute_tokens_backward(s["grad"], s["y"], s["plan"],
                                                                 s["weights"])
        return out
    if op == "quantize":
        q, scale = moe.quantize_fp8_block(s["x"], gated=c["gated"])
        return dict(codes=q, scale=scale)
    if op == "gemm":
        return dict(out=moe.gemm_fp8_block(s["a"], s["a_scale"], s["b"], s["b_scale"]))
    return dict(out=moe.grouped_gemm_fp8_block(s["a"], s["a_scale"], s["b"], s["b_scale"],
                                               s["plan"], c["block_m"], out=s["out"]))


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] in ("permute", "unpermute"):
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["K"]
        cap = n + min(c["E"], n) * (c["block_m"] - 1)
        token, list_, kept = c["T"] * c["H"] * es, cap * c["H"] * es, n * c["H"] * es
        if c["op"] == "permute":
            b = token + list_ + 4 * (n + cap)
            f = 0
            if c["mode"] == "train":
                b, f = b + kept + token + 4 * n, f + n * c["H"]
        else:
            b, f = kept + token + 8 * n, 2 * n * c["H"]
            if c["mode"] == "train":
                b += token + kept + list_ + 12 * n + 4 * cap
                f += 3 * n * c["H"]
        return dict(bytes=b, flops=f)
    if c["op"] == "quantize":
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["H"]
        return dict(bytes=n * es * (2 if c["gated"] else 1) + n + 4 * c["T"] * -(-c["H"] // BLOCK),
                    flops=n * (8 if c["gated"] else 3))
    N, K = c["N"], c["K"]
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    if c["op"] == "gemm":
        M = c["M"]
        return dict(bytes=M * K + N * K + 4 * kb * (M + nb) + 2 * M * N, flops=2 * M * N * K)
    n = c["T"] * c["TopK"]
    # experts that receive a row, in expectation
    active = float((1 - (1 - _popularity(c["E"], c["routing"])).pow(n)).sum())
    return dict(bytes=n * K + active * N * K + 4 * kb * (n + active * nb) + 2 * n * N,
                flops=2 * n * N * K)


# -------------------------------------------------- the definitions in 64 bits

def _exact_product(a, a_scale, b, b_scale):
    """sum over the scale blocks along K of a_scale * b_scale * (a . b)."""
    col = torch.arange(a.shape[1], device=a.device) // BLOCK
    row = torch.arange(b.shape[0], device=a.device) // BLOCK
    x = a.double() * a_scale.double()[:, col]
    w = b.double() * b_scale.double()[row][:, col]
    return x @ w.t()


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("permute", "unpermute"):
        K, T = c["K"], c["T"]
        slots = s["plan"]["inv_perm"].long().view(T, K)
        rows = s["plan"]["sorted_ids"].numel()
        if c["op"] == "permute":
            x = s["x"].double()
            xs = torch.zeros((rows, c["H"]), dtype=torch.float64, device="cuda")
            for k in range(K):
                xs[slots[:, k]] = x
            out = dict(rows=xs)
            if c["mode"] == "train":
                out["dx"] = sum(s["grad"][slots[:, k]].double() for k in range(K))
            return out
        y, w = s["y"], s["weights"].double()
        out = dict(out=sum(w[:, k:k + 1] * y[slots[:, k]].double() for k in range(K)))
        if c["mode"] == "train":
            grad = s["grad"].double()
            dy = torch.zeros((rows, c["H"]), dtype=torch.float64, device="cuda")
            dw = torch.empty((T, K), dtype=torch.float64, device="cuda")
            for k in range(K):
                dy[slots[:, k]] = w[:, k:k + 1] * grad
                dw[:, k] = (grad * y[slots[:, k]].double()).sum(1)
            out["dy"], out["dw"] = dy, dw
        return out
    if c["op"] == "quantize":
        x = s["x"].double()
        H = c["H"]
        if c["gated"]:
            x = x[:, :H] * torch.sigmoid(x[:, :H]) * x[:, H:]
        codes = torch.empty((c["T"], H), dtype=torch.float64, device="cuda")
        scale = torch.empty((c["T"], -(-H // BLOCK)), dtype=torch.float64, device="cuda")
        for j in range(scale.shape[1]):
            part = x[:, j * BLOCK:(j + 1) * BLOCK]
            scale[:, j] = part.abs().amax(1).clamp(min=AMAX_FLOOR) / 448.0
            v = (part / scale[:, j:j + 1]).clamp(-448.0, 448.0)
            codes[:, j * BLOCK:(j + 1) * BLOCK] = v.to(torch.float8_e4m3fn).double()
        return dict(codes=codes, scale=scale)
    if c["op"] == "gemm":
        return dict(out=_exact_product(s["a"], s["a_scale"], s["b"], s["b_scale"]))
    out = torch.zeros((s["a"].shape[0], c["N"]), dtype=torch.float64, device="cuda")
    for e, _, first, valid in s["plan"]["block_info"].tolist():
        if e >= 0:
            r = slice(first, first + valid)
            out[r] = _exact_product(s["a"][r], s["a_scale"][r], s["b"][e], s["b_scale"][e])
    return dict(out=out)
