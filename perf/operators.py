"""What the experts' products and the gradient of dispatch and combine cost.

Four operators of the path, each in a plain form of elementary torch
operations (``own`` false) and as a user calls it (``own`` true):

* ``product``           moe_grouped_gemm_fp8: expert rows times expert weights, both e4m3
                        with a scale per 128 channels (weights: per 128 x 128 block);
* ``gated``             moe_grouped_gemm_silu_fp8: the first product of an expert with
                        silu(gate) * up and the e4m3 quantisation of the result;
* ``combine_backward``  the gradient of the weighted gather-sum;
* ``dispatch_backward`` the gradient of the scatter of token rows.

Sizes are the path's own (hidden 7168, 256 or 512 experts, top-8, batches of
128, 4096 and 16384 tokens, the tiny line's 16 x 128 x 8 x 2) with an expert
width of 2048, and odd ones.
"""

import math

import torch

own = False

ALIGN = 128
BLOCK = 128
E4M3_MAX = 448.0
DEV = "cuda"


def listed():
    return [
        # One token's second product: 8 experts of one row each, where latency counts.
        dict(name="product one token", op="product", tokens=1, experts=256, topk=8, hidden=7168,
             inter=2048, alpha=0.0, dropped=0.0, dense=False),
        # A decode batch: about 4 rows an expert, so the weights' bytes bound it.
        dict(name="product decode", op="product", tokens=128, experts=256, topk=8, hidden=7168,
             inter=2048, alpha=0.0, dropped=0.0, dense=False),
        # A prefill batch under skewed routing: tens to hundreds of rows an expert.
        dict(name="product prefill skewed", op="product", tokens=4096, experts=256, topk=8,
             hidden=7168, inter=2048, alpha=0.6, dropped=0.0, dense=False),
        # The shared expert's second product on a prefill batch: one dense product.
        dict(name="product shared expert", op="product", tokens=4096, experts=1, topk=1,
             hidden=7168, inter=2048, alpha=0.0, dropped=0.0, dense=True),
        # The tiny line: the smallest call of the fused first product.
        dict(name="gated tiny", op="gated", tokens=16, experts=8, topk=2, hidden=128, inter=128,
             alpha=0.0, dropped=0.0, dense=False),
        # A decode batch's first product on all 256 experts.
        dict(name="gated decode", op="gated", tokens=128, experts=256, topk=8, hidden=7168,
             inter=2048, alpha=0.0, dropped=0.0, dense=False),
        # An odd batch on a small model, some pairs dropped, a few hot experts.
        dict(name="gated odd", op="gated", tokens=777, experts=60, topk=6, hidden=1408, inter=896,
             alpha=1.2, dropped=0.05, dense=False),
        # One expert-parallel rank's share: 32 experts with about 1000 rows each.
        dict(name="gated rank share", op="gated", tokens=4096, experts=32, topk=8, hidden=7168,
             inter=2048, alpha=0.0, dropped=0.0, dense=False),
        # A training micro-batch small enough that launches count.
        dict(name="combine_backward small", op="combine_backward", tokens=128, experts=256,
             topk=8, hidden=7168, inter=0, alpha=0.0, dropped=0.0, dense=False),
        # A training micro-batch under skewed routing.
        dict(name="combine_backward skewed", op="combine_backward", tokens=4096, experts=256,
             topk=8, hidden=7168, inter=0, alpha=0.6, dropped=0.0, dense=False),
        # The scatter's gradient on an odd batch with dropped pairs.
        dict(name="dispatch_backward odd", op="dispatch_backward", tokens=1023, experts=100,
             topk=6, hidden=2080, inter=0, alpha=0.0, dropped=0.05, dense=False),
        # The scatter's gradient on the large line: 16384 tokens, a few hot experts of 512.
        dict(name="dispatch_backward large", op="dispatch_backward", tokens=16384, experts=512,
             topk=8, hidden=7168, inter=0, alpha=1.2, dropped=0.0, dense=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "gated", "combine_backward", "dispatch_backward"])
    alpha = rng.choice([0.0, 0.0, 0.6, 1.2])
    dropped = rng.choice([0.0, 0.0, 0.05])
    if op in ("combine_backward", "dispatch_backward"):
        experts = _spread(rng, 2, 512)
        topk = min(rng.randint(1, 16), experts)
        hidden = 32 * _spread(rng, 2, 256)
        tokens = _spread(rng, 1, min(16384, int(9.0e8 / (topk * hidden))))
        return dict(op=op, tokens=tokens, experts=experts, topk=topk, hidden=hidden, inter=0,
                    alpha=alpha, dropped=dropped, dense=False)
    dense = op == "product" and rng.random() < 0.25
    inter = 128 * _spread(rng, 1, 32)
    hidden = 128 * _spread(rng, 1, 64) if op == "gated" else 32 * _spread(rng, 2, 256)
    width = (2 if op == "gated" else 1) * inter * hidden  # weights of one expert
    experts = 1 if dense else _spread(rng, 2, min(512, int(7.4e9 / width)))
    topk = 1 if dense else min(rng.randint(1, 16), experts)
    tokens = _spread(rng, 1, max(1, min(16384, int(9.0e11 / (width * topk)))))
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, hidden=hidden, inter=inter,
                alpha=0.0 if dense else alpha, dropped=0.0 if dense else dropped, dense=dense)


# ---------------------------------------------------------------- inputs

def _route(case, gen):
    """Top-k ids (a dropped pair's is -1), and the layout a dispatch makes of
    them: counts, 128-padded offsets, within-expert ranks."""
    bs, e, k = case["tokens"], case["experts"], case["topk"]
    keys = torch.rand((bs, e), generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
    keys = -torch.log(-torch.log(keys))
    if case["alpha"]:
        order = torch.randperm(e, generator=gen, device=DEV).float()
        keys = keys - case["alpha"] * torch.log(order + 1)
    ids = keys.topk(k, dim=1).indices
    if case["dropped"]:
        keep = torch.rand((bs, k), generator=gen, device=DEV) >= case["dropped"]
        ids = torch.where(keep, ids, torch.full_like(ids, -1))
    flat = ids.reshape(-1)
    hot = torch.nn.functional.one_hot(flat.clamp(min=0), e) * (flat >= 0)[:, None]
    counts = hot.sum(0)
    rank = (hot.cumsum(0) - hot).gather(1, flat.clamp(min=0)[:, None])[:, 0]
    rank = torch.where(flat >= 0, rank, torch.full_like(rank, -1))
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    send = torch.zeros(e + 1, dtype=torch.int64, device=DEV)
    send[1:] = padded.cumsum(0)
    n = bs * k
    cap = ALIGN * ((n + (ALIGN - 1) * min(n, e)) // ALIGN)
    return dict(ids=ids.int(), idx=rank.int(), counts=counts.int(), send=send.int(), cap=cap)


def _quantised(x):
    """e4m3 codes and fp32 scales of rows, one scale per 128 channels."""
    rows, cols = x.shape
    b = x.view(rows, cols // BLOCK, BLOCK)
    s = b.abs().amax(2) / E4M3_MAX
    q = (b / s.clamp(min=1e-30)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(rows, cols).view(torch.uint8), s


def _weights(e, n, k, gen):
    """e4m3 codes [e, n, k] and a scale per 128 x 128 block."""
    nb, kb = -(-n // BLOCK), k // BLOCK
    codes = torch.empty((e, n, k), dtype=torch.uint8, device=DEV)
    scales = torch.empty((e, nb, kb), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 29) // (nb * BLOCK * k))
    for e0 in range(0, e, step):
        c = min(step, e - e0)
        w = torch.randn((c, nb * BLOCK, k), generator=gen, device=DEV).mul_(k ** -0.5)
        b = w.view(c, nb, BLOCK, kb, BLOCK)
        s = b.abs().amax((2, 4)) / E4M3_MAX
        b.div_(s[:, :, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        codes[e0:e0 + c] = w.to(torch.float8_e4m3fn).view(torch.uint8)[:, :n]
        scales[e0:e0 + c] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, bs, e, k = case["op"], case["tokens"], case["experts"], case["topk"]
    hidden, inter = case["hidden"], case["inter"]
    s = dict(op=op, experts=e, topk=k, dense=case["dense"])
    if case["dense"]:
        s.update(counts=None, send=None, cap=bs, rows=bs)
    else:
        s.update(_route(case, gen), rows=bs * k)
    cap = s["cap"]
    if op in ("product", "gated"):
        n, kdim = (hidden, inter) if op == "product" else (2 * inter, hidden)
        x = torch.randn((cap, kdim), generator=gen, device=DEV)
        if op == "product":  # rows that a gated activation made
            x = x * torch.sigmoid(x) * torch.randn((cap, kdim), generator=gen, device=DEV)
        s["x"], s["x_scales"] = _quantised(x)
        s["w"], s["w_scales"] = _weights(e, n, kdim, gen)
        # The buffers a serving loop keeps; rows of no token stay as they are.
        if op == "product":
            s["out"] = torch.zeros((cap, n), dtype=torch.bfloat16, device=DEV)
        else:
            s["out"] = torch.zeros((cap, inter), dtype=torch.uint8, device=DEV)
            s["out_scales"] = torch.zeros((cap, inter // BLOCK), dtype=torch.float32, device=DEV)
        if not case["dense"]:
            # What a host that knows the routing would loop over: the experts with rows.
            s["active"] = s["counts"].nonzero()[:, 0]
            s["longest"] = int(s["counts"].max())
    elif op == "combine_backward":
        s["grad"] = torch.randn((bs, hidden), generator=gen, device=DEV).bfloat16()
        s["y"] = torch.randn((cap, hidden), generator=gen, device=DEV).bfloat16()
        logits = torch.randn((bs, k), generator=gen, device=DEV)
        s["scales"] = torch.softmax(logits, 1)
        s["out"] = torch.zeros((cap, hidden), dtype=torch.bfloat16, device=DEV)
    else:
        s["grad"] = torch.randn((cap, hidden), generator=gen, device=DEV).bfloat16()
        s["add"] = torch.randn((bs, hidden), generator=gen, device=DEV).bfloat16()
    return s


# ---------------------------------------------------------------- the operators

def _call(s):
    """The calls a user makes of the framework."""
    import combine_moe_dispatch_layout_amd as moe
    op = s["op"]
    if op == "product":
        return moe.moe_grouped_gemm_fp8(s["x"], s["x_scales"], s["w"], s["w_scales"],
                                        s["counts"], s["send"], expected_rows=s["rows"],
                                        out=s["out"])
    if op == "gated":
        codes, scales = moe.moe_grouped_gemm_silu_fp8(
            s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], s["send"],
            expected_rows=s["rows"], out=s["out"], out_scales=s["out_scales"])
        return codes.view(torch.float8_e4m3fn), scales
    if op == "combine_backward":
        return moe.moe_combine_backward(s["grad"], s["y"], s["ids"], s["idx"], s["send"],
                                        s["scales"], s["experts"], grad_expand_x=s["out"])
    return moe.moe_dispatch_backward(s["grad"], s["ids"], s["idx"], s["send"], s["experts"],
                                     grad_x_add=s["add"])


def _dequantised(codes, scales):
    """fp32 values of e4m3 codes [.., rows, cols] with scales [.., rows, cols / 128]."""
    v = codes.view(torch.float8_e4m3fn).float()
    v.view(*scales.shape, BLOCK).mul_(scales[..., None])
    return v


def _plain_product(s):
    """fp32 products of the experts' rows [active, longest, n], with the row
    each belongs to ([active, longest], cap where there is none)."""
    cap = s["cap"]
    n = s["w"].shape[1]
    if s["dense"]:
        rows = torch.arange(cap, device=DEV)[None]
        w, ws = s["w"], s["w_scales"]
    else:
        at = torch.arange(s["longest"], device=DEV)[None]
        act = s["active"]
        start, count = s["send"][act].long()[:, None], s["counts"][act].long()[:, None]
        rows = torch.where(at < count, start + at, torch.full_like(start + at, cap))
        w, ws = s["w"][act], s["w_scales"][act]
    x = _dequantised(s["x"], s["x_scales"])
    xt = x[rows.clamp(max=cap - 1)].transpose(1, 2).contiguous()
    wf = _dequantised(w, ws.repeat_interleave(BLOCK, 1)[:, :n])
    return torch.bmm(wf, xt).transpose(1, 2), rows


def _by_row(values, rows, cap):
    """values [.., cols] put at their rows of a [cap, cols] buffer of zeros."""
    out = torch.zeros((cap + 1, values.shape[-1]), dtype=values.dtype, device=DEV)
    out[rows.reshape(-1)] = values.reshape(-1, values.shape[-1])
    return out[:cap]


def _plain(s):
    op = s["op"]
    if op == "product":
        y, rows = _plain_product(s)
        return _by_row(y.bfloat16(), rows, s["cap"])
    if op == "gated":
        y, rows = _plain_product(s)
        gate, up = y.chunk(2, 2)
        h = gate / (1 + torch.exp(-gate)) * up
        b = h.reshape(*h.shape[:2], -1, BLOCK)
        scales = b.abs().amax(3) / E4M3_MAX
        q = torch.where(scales[..., None] > 0, b / scales[..., None], torch.zeros_like(b))
        codes = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        return (_by_row(codes.reshape(h.shape), rows, s["cap"]).view(torch.float8_e4m3fn),
                _by_row(scales, rows, s["cap"]))
    ids, bs, k = s["ids"].long(), s["ids"].shape[0], s["topk"]
    real = (ids >= 0).reshape(-1)
    slots = s["send"].long()[ids.clamp(min=0)].reshape(-1) + s["idx"]
    if op == "combine_backward":
        cap, h = s["y"].shape
        g = s["grad"].float()
        dy = (s["scales"][:, :, None] * g[:, None]).bfloat16()
        dy = _by_row(dy, torch.where(real, slots, torch.full_like(slots, cap)), cap)
        y = torch.where(real[:, None], s["y"][slots.clamp(0, cap - 1)].float(), 0.0)
        return dy, (y.view(bs, k, h) * g[:, None]).sum(2)
    cap, h = s["grad"].shape
    g = torch.where(real[:, None], s["grad"][slots.clamp(0, cap - 1)].float(), 0.0)
    return (g.view(bs, k, h).sum(1) + s["add"].float()).bfloat16()


def run(state):
    return _call(state) if own else _plain(state)


# ---------------------------------------------------------------- what they cannot do without

def work(case):
    bs, e, k = case["tokens"], case["experts"], case["topk"]
    hidden, inter = case["hidden"], case["inter"]
    rows = bs * k * (1 - case["dropped"])
    if case["op"] in ("product", "gated"):
        active = e * (1 - (1 - k / e) ** bs) if e > 1 else 1
        n, kdim = (hidden, inter) if case["op"] == "product" else (2 * inter, hidden)
        written = n * 2 if case["op"] == "product" else inter * (1 + 4 / BLOCK)
        return {"bytes": rows * (kdim * (1 + 4 / BLOCK) + written)
                + active * n * kdim * (1 + 4 / BLOCK ** 2),
                "flops": 2 * rows * n * kdim}
    if case["op"] == "combine_backward":
        return {"bytes": 2 * hidden * (bs + 2 * rows) + 16 * bs * k, "flops": 3 * rows * hidden}
    return {"bytes": 2 * hidden * (rows + 2 * bs) + 8 * bs * k, "flops": rows * hidden}


# ---------------------------------------------------------------- by the definition, in 64 bits

def _exact_expert(s, e, lo, hi):
    """Rows [lo, hi) of expert e's product, in 64 bits."""
    x = s["x"][lo:hi].view(torch.float8_e4m3fn).double()
    x *= torch.repeat_interleave(s["x_scales"][lo:hi].double(), BLOCK, dim=1)
    n = s["w"].shape[1]
    w = s["w"][e].view(torch.float8_e4m3fn).double()
    ws = s["w_scales"][e].double()
    w *= ws.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)
    return x @ w.t().contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("product", "gated"):
        cap, n = s["cap"], s["w"].shape[1]
        if case["dense"]:
            parts = [(0, 0, cap)]
        else:
            counts, send = s["counts"].tolist(), s["send"].tolist()
            parts = [(e, send[e], send[e] + c) for e, c in enumerate(counts) if c]
        cols = n if op == "product" else n // 2
        out = torch.zeros((cap, cols), dtype=torch.float64, device=DEV)
        scales = torch.zeros((cap, -(-cols // BLOCK)), dtype=torch.float64, device=DEV)
        for e, lo, hi in parts:
            y = _exact_expert(s, e, lo, hi)
            if op == "gated":
                y = torch.nn.functional.silu(y[:, :cols]) * y[:, cols:]
                y = y.view(hi - lo, -1, BLOCK)
                scales[lo:hi] = y.abs().max(2).values / E4M3_MAX
                y = (y / scales[lo:hi, :, None]).view(hi - lo, cols)
            out[lo:hi] = y
        return out if op == "product" else (out, scales)
    ids, idx, send = s["ids"].tolist(), s["idx"].tolist(), s["send"].tolist()
    bs, k = case["tokens"], case["topk"]
    pairs = [(t, j, send[ids[t][j]] + idx[t * k + j]) for t in range(bs) for j in range(k)
             if ids[t][j] >= 0]
    token, choice, slot = (torch.tensor(v, dtype=torch.int64, device=DEV)
                           for v in (zip(*pairs) if pairs else ((), (), ())))
    if op == "combine_backward":
        dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros((bs, k), dtype=torch.float64, device=DEV)
        for i in range(0, len(pairs), 16384):
            t, j, r = token[i:i + 16384], choice[i:i + 16384], slot[i:i + 16384]
            g = s["grad"][t].double()
            dy[r] = g * s["scales"][t, j].double()[:, None]
            dw[t, j] = torch.linalg.vecdot(g, s["y"][r].double())
        return dy, dw
    dx = s["add"].double()
    for j in range(k):
        of = choice == j
        dx[token[of]] += s["grad"][slot[of]].double()
    return dx
