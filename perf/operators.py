"""The layer's 8-bit expert products and its balance loss, as they are measured.

Each case is one call (or one training step) of these operators:

  rows      quantise activations to e4m3, one power-of-two scale per row and 128 columns
  weights   quantise expert weights to e4m3, one power-of-two scale per 128 x 128 block (also transposed)
  product   ragged grouped product of quantised rows with quantised weights
  ffn       the expert FFN on quantised weights (SwiGLU or GELU)
  balance   balance loss over sequences, counts, and the gradient of the router's logits

``run`` computes them in elementary torch operations (``own`` false) or through the package (``own`` true).
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_MIN = E4M3_MAX * 2.0 ** -126   # keeps a block's scale a normal number
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # activations of one long prompt chunk at the DeepSeek-V3 width, and of a few fp32 tokens of odd width
        dict(name="rows_prompt", op="rows", rows=32768, cols=7168, dtype="bf16"),
        dict(name="rows_tokens_f32", op="rows", rows=33, cols=2064, dtype="f32"),
        # one matrix of the Mixtral experts, transposed for the input gradient; a small odd fp32 one
        dict(name="weights_mixtral_t", op="weights", E=8, rows=14336, cols=4096, transpose=True, dtype="bf16"),
        dict(name="weights_odd_f32", op="weights", E=5, rows=1104, cols=720, transpose=False, dtype="f32"),
        # decoding 16 tokens, and the fp32 input gradient at the Qwen3 shape with its skewed slices
        dict(name="product_decode", op="product", tokens=16, k=2, E=8, n=4096, kdim=14336, skew=0.0, out="bf16"),
        dict(name="product_skew_f32", op="product", tokens=16384, k=8, E=128, n=2048, kdim=768, skew=1.0, out="f32"),
        # one token of DeepSeek-V3; its 4096-token batch (weight bound); Mixtral's (compute bound); odd GELU experts with biases
        dict(name="ffn_token", op="ffn", tokens=1, k=8, E=256, d=7168, F=2048, act="swiglu", skew=0.0),
        dict(name="ffn_deepseek", op="ffn", tokens=4096, k=8, E=256, d=7168, F=2048, act="swiglu", skew=0.0),
        dict(name="ffn_mixtral", op="ffn", tokens=4096, k=2, E=8, d=4096, F=14336, act="swiglu", skew=0.0),
        dict(name="ffn_gelu_ragged", op="ffn", tokens=1999, k=2, E=6, d=784, F=2000, act="gelu", skew=0.6),
        # the router's loss: a small padded batch of eight experts, and a training batch of DeepSeek-V3
        dict(name="balance_small", op="balance", tokens=1000, k=2, E=8, seqs=4, scores="softmax", padded=True, dtype="f32"),
        dict(name="balance_batch", op="balance", tokens=131072, k=8, E=256, seqs=32, scores="sigmoid", padded=False, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of16(rng, lo, hi):
    return max(16, _spread(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["rows", "weights", "product", "ffn", "balance"])
    if op == "rows":
        cols = _of16(rng, 64, 14336)
        return dict(op=op, rows=_spread(rng, 1, max(2, 200_000_000 // cols)), cols=cols, dtype=rng.choice(["bf16", "f32"]))
    if op == "weights":
        rows, cols = _of16(rng, 128, 14336), _of16(rng, 128, 8192)
        return dict(op=op, E=_spread(rng, 1, max(1, min(256, 400_000_000 // (rows * cols)))), rows=rows, cols=cols,
                    transpose=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
    if op == "balance":
        E = rng.choice([4, 6, 8, 16, 24, 60, 64, 100, 128, 160, 256])
        tokens = _spread(rng, 16, 131072)
        return dict(op=op, tokens=tokens, k=rng.choice([1, 2, 4]) if E < 16 else rng.choice([4, 6, 8]), E=E,
                    seqs=_spread(rng, 1, max(1, min(512, tokens // 8))), scores=rng.choice(["softmax", "sigmoid"]),
                    padded=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))
    E, k = rng.choice([(6, 2), (8, 2), (16, 2), (32, 4), (64, 6), (128, 8)])
    tokens, skew = _spread(rng, 1, 8192), rng.choice([0.0, 0.5, 1.0])
    if op == "product":
        return dict(op=op, tokens=tokens, k=k, E=E, n=_of16(rng, 128, 4096), kdim=_of16(rng, 128, 4096), skew=skew,
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, tokens=tokens, k=k, E=E, d=_of16(rng, 128, 4096), F=_of16(rng, 128, 4096),
                act=rng.choice(["swiglu", "swiglu", "gelu"]), skew=skew)


def _active(case):
    """Experts that receive a row, as expected of tokens that choose evenly."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["tokens"])


def work(case):
    op, size = case["op"], {"bf16": 2, "f32": 4}.get(case.get("dtype"), 0)
    if op == "rows":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size + 1) + 4 * case["rows"] * -(-case["cols"] // BLOCK), "flops": 3 * n}
    if op == "weights":
        n = case["E"] * case["rows"] * case["cols"]
        return {"bytes": n * (size + 1) + 4 * case["E"] * -(-case["rows"] // BLOCK) * -(-case["cols"] // BLOCK), "flops": 3 * n}
    if op == "balance":
        n = case["tokens"] * case["E"]
        # forward: logits and ids; backward: logits again, the gradient written
        return {"bytes": n * (2 * size + 4) + 4 * case["tokens"] * case["k"], "flops": 20 * n}
    rows, active = case["tokens"] * case["k"], _active(case)
    if op == "product":
        n, k = case["n"], case["kdim"]
        return {"bytes": rows * k * (1 + 4 / BLOCK) + active * n * k + rows * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * rows * n * k}
    mats = 3 if case["act"] == "swiglu" else 2
    return {"bytes": 4 * rows * case["d"] + active * mats * case["d"] * case["F"], "flops": 2 * mats * rows * case["d"] * case["F"]}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _offsets(case, g):
    """Slice starts of tokens that choose k of E experts each; skew: a Zipf-like preference."""
    E = case["E"]
    rank = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).log()
    noise = -torch.empty(case["tokens"], E, device="cuda").exponential_(generator=g).log()
    ids = (noise - case["skew"] * rank).topk(case["k"], dim=1).indices
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, int(counts.max()), counts.nonzero().view(-1)


def _made_weights(E, rows, cols, g):
    """Quantised N(0, 0.02) weights, some experts at a time."""
    q = torch.empty((E, rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((E, -(-rows // BLOCK), -(-cols // BLOCK)), device="cuda")
    step = max(1, 400_000_000 // (rows * cols))
    for e in range(0, E, step):
        w = torch.randn((min(step, E - e), rows, cols), generator=g, device="cuda").mul_(0.02)
        q[e:e + step], s[e:e + step] = _weights_plain(w, False)
    return q, s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    state = dict(case)
    if op == "rows":
        # activations: per-row sizes differ by an order of magnitude, as hidden states do
        x = torch.randn((case["rows"], case["cols"]), generator=g, device="cuda")
        x *= torch.rand((case["rows"], 1), generator=g, device="cuda").mul_(2.3).exp_()
        state["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "weights":
        state["W"] = torch.empty((case["E"], case["rows"], case["cols"]), dtype=DTYPES[case["dtype"]], device="cuda")
        for e in range(case["E"]):
            state["W"][e] = torch.randn((case["rows"], case["cols"]), generator=g, device="cuda").mul_(0.02)
    elif op == "balance":
        N, E, S = case["tokens"], case["E"], case["seqs"]
        z = torch.randn((N, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        state["logits"] = z.to(DTYPES[case["dtype"]])
        state["topk_ids"] = state["logits"].topk(case["k"], dim=1).indices.to(torch.int32)
        cuts = torch.randint(1, N, (S - 1,), generator=g, device="cuda").sort().values if S > 1 else torch.empty(0, device="cuda")
        ends = torch.tensor([0, N], device="cuda")
        state["seq_offsets"] = torch.cat([ends[:1], cuts.to(ends.dtype), ends[1:]]).to(torch.int32)
        # padding: about an eighth of the tokens count for nothing
        state["token_mask"] = torch.rand(N, generator=g, device="cuda") > 0.125 if case["padded"] else None
    else:
        state["offsets"], state["longest"], state["active"] = _offsets(case, g)
        rows = case["tokens"] * case["k"]
        if op == "product":
            x = torch.randn((rows, case["kdim"]), generator=g, device="cuda")
            state["a"] = _rows_plain(x)
            state["w"] = _made_weights(case["E"], case["n"], case["kdim"], g)
        else:
            E, d, F = case["E"], case["d"], case["F"]
            state["x_sorted"] = torch.randn((rows, d), generator=g, device="cuda").to(torch.bfloat16)
            state["W1"], state["W2"] = _made_weights(E, F, d, g), _made_weights(E, d, F, g)
            state["W3"] = _made_weights(E, F, d, g) if case["act"] == "swiglu" else None
            small = lambda n: torch.randn((E, n), generator=g, device="cuda").mul_(0.02).to(torch.bfloat16)  # noqa: E731
            state["b1"], state["b2"] = (small(F), small(d)) if case["act"] == "gelu" else (None, None)
    return state


# -------------------------------------------------------------- plain forms


def _scale(amax):
    """The smallest power of two s with amax / s <= 448 (amax = m 2^x, 1/2 <= m < 1, and 448 = 7/8 2^9)."""
    m, x = torch.frexp(amax.clamp(min=AMAX_MIN))
    e = x - 9 + (m > 0.875)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _rows_plain(x):
    """(q [rows, cols] e4m3, scales [ceil(cols / 128), rows])."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    s = _scale(x.abs().amax(2))
    q = (x * (1.0 / s)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :cols].contiguous(), s.t().contiguous()


def _weights_plain(W, transpose):
    """(q [E, rows, cols] e4m3, scales [E, ceil(rows / 128), ceil(cols / 128)]), both with the last two axes exchanged if asked for."""
    E, rows, cols = W.shape
    x = torch.nn.functional.pad(W.float(), (0, -cols % BLOCK, 0, -rows % BLOCK))
    x = x.view(E, x.shape[1] // BLOCK, BLOCK, x.shape[2] // BLOCK, BLOCK)
    s = _scale(x.abs().amax((2, 4)))
    q = (x * (1.0 / s)[:, :, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(E, x.shape[1] * BLOCK, x.shape[3] * BLOCK)[:, :rows, :cols]
    if transpose:
        q, s = q.transpose(1, 2), s.transpose(1, 2)
    return q.contiguous(), s.contiguous()


def _rows_values(q, s):
    return q.float() * s.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _weights_values(w, experts):
    """The values of some experts' weights."""
    q, s = w
    w, s = q.view(torch.uint8)[experts].view(q.dtype).float(), s[experts]
    return w * s.repeat_interleave(BLOCK, 1)[:, :w.shape[1]].repeat_interleave(BLOCK, 2)[:, :, :w.shape[2]]


def _grouped_plain(x, w, s):
    """Rows offsets[e] .. offsets[e+1]-1 of x times w[e]^T for the experts that have rows, every slice padded to the longest."""
    start = s["offsets"].long()[s["active"]]
    row = torch.arange(x.shape[0], device=x.device)
    at = torch.searchsorted(start, row, right=True) - 1
    rows = (start[:, None] + torch.arange(s["longest"], device=x.device)).clamp(max=x.shape[0] - 1)
    y = torch.bmm(x[rows], _weights_values(w, s["active"]).transpose(1, 2))
    return y[at, row - start[at]], s["active"][at]


def _ffn_plain(s):
    x = _rows_values(*_rows_plain(s["x_sorted"]))
    h, expert = _grouped_plain(x, s["W1"], s)
    if s["act"] == "swiglu":
        up, _ = _grouped_plain(x, s["W3"], s)
        h = h * (1.0 / (1.0 + torch.exp(-h))) * up
    else:
        h = h + s["b1"].float()[expert]
        h = 0.5 * h * (1.0 + torch.erf(h * 0.5 ** 0.5))
    y, _ = _grouped_plain(_rows_values(*_rows_plain(h)), s["W2"], s)
    return (y if s["b2"] is None else y + s["b2"].float()[expert]).to(torch.bfloat16)


def _balance_plain(s):
    z, E, S = s["logits"].float(), s["E"], s["seqs"]
    N, k = z.shape[0], s["k"]
    seq = torch.searchsorted(s["seq_offsets"].long(), torch.arange(N, device=z.device), right=True) - 1
    valid = torch.ones(N, dtype=torch.bool, device=z.device) if s["token_mask"] is None else s["token_mask"]
    if s["scores"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        m = 1.0
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
        m = 1.0 - p
    p = p / p.sum(1, keepdim=True) * valid[:, None]
    place = (seq[:, None] * E + s["topk_ids"].long())[valid]
    counts = torch.bincount(place.reshape(-1), minlength=S * E).view(S, E)
    tokens = torch.bincount(seq[valid], minlength=S).double()
    P = torch.zeros((S, E), dtype=torch.float64, device=z.device).index_add_(0, seq, p.double())
    weight = torch.where(tokens > 0, E / (tokens.clamp(min=1) ** 2 * (tokens > 0).sum()), 0.0)
    loss = (weight * (counts * P).sum(1)).sum()
    c = (weight[:, None] * counts).float()[seq]
    dz = p * m * (c - (p * c).sum(1, keepdim=True))
    return {"loss": loss.float().view(1), "counts": counts.int(), "dlogits": dz}


def run(state):
    op = state["op"]
    if own:
        import mixture_experts_layer_53_b200 as M
        if op == "rows":
            return M.moe_quantize_rows(state["x"])
        if op == "weights":
            return M.moe_quantize_weights(state["W"], transpose=state["transpose"])
        if op == "product":
            return M.moe_expert_matmul_fp8(state["a"], state["offsets"], state["w"], out_dtype=DTYPES[state["out"]])
        if op == "ffn":
            cfg = M.make_config(state["tokens"], state["d"], state["F"], state["E"], state["k"], act=state["act"], dtype="bf16")
            return M.moe_expert_ffn_fp8(cfg, state["x_sorted"], state["offsets"], state["W1"], state["W2"], W3=state["W3"],
                                        b1=state["b1"], b2=state["b2"])
        kw = dict(seq_offsets=state["seq_offsets"], token_mask=state["token_mask"], scores=state["scores"])
        fwd = M.moe_balance_loss(state["logits"], state["topk_ids"], **kw)
        dz = M.moe_balance_loss_backward(state["logits"], fwd, **kw)
        return {"loss": fwd["loss"], "counts": fwd["counts"], "dlogits": dz}
    if op == "rows":
        return _rows_plain(state["x"])
    if op == "weights":
        return _weights_plain(state["W"], state["transpose"])
    if op == "product":
        y, _ = _grouped_plain(_rows_values(*state["a"]), state["w"], state)
        return y.to(DTYPES[state["out"]])
    return _ffn_plain(state) if op == "ffn" else _balance_plain(state)


# ------------------------------------------------------- the same in 64 bits


def _exact_scale(amax):
    """2^e with the smallest whole e such that amax <= 448 2^e."""
    a = amax.double().clamp(min=AMAX_MIN)
    e = torch.ceil(torch.log2(a / E4M3_MAX))
    e = e + (a > E4M3_MAX * torch.exp2(e)).double()
    return torch.exp2(e - (a <= E4M3_MAX * torch.exp2(e - 1)).double())


def _exact_rows(x):
    """Values of x rounded to e4m3 under a scale for each row and 128 columns: (q, scales), in 64 bits."""
    q, scales = torch.empty_like(x, dtype=torch.float64), []
    for c in range(0, x.shape[1], BLOCK):
        part = x[:, c:c + BLOCK].double()
        s = _exact_scale(part.abs().max(1).values)
        q[:, c:c + BLOCK] = (part / s[:, None]).float().to(torch.float8_e4m3fn).double()
        scales.append(s)
    return q, torch.stack(scales)


def _exact_slice(x, w, e, lo, hi):
    """x[lo:hi] w[e]^T, block of 128 columns after block."""
    (xq, xs), (wq, ws) = x, w
    y = torch.zeros((hi - lo, wq.shape[1]), dtype=torch.float64, device=xq.device)
    for b in range(xs.shape[0]):
        c = slice(b * BLOCK, (b + 1) * BLOCK)
        scale = ws[e, :, b].double().repeat_interleave(BLOCK)[:wq.shape[1]]
        y += (xq[lo:hi, c].double() * xs[b, lo:hi, None].double()) @ (wq[e, :, c].double() * scale[:, None]).t()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        return list(_exact_rows(s["x"]))
    if op == "weights":
        q, scales = [], []
        for W in s["W"]:
            W = W.t() if case["transpose"] else W
            a = torch.stack([torch.stack([W[r:r + BLOCK, c:c + BLOCK].abs().max() for c in range(0, W.shape[1], BLOCK)])
                             for r in range(0, W.shape[0], BLOCK)])
            a = _exact_scale(a)
            each = a.repeat_interleave(BLOCK, 0)[:W.shape[0]].repeat_interleave(BLOCK, 1)[:, :W.shape[1]]
            q.append((W.double() / each).float())
            scales.append(a)
        return [torch.stack(q).to(torch.float8_e4m3fn).float(), torch.stack(scales)]
    if op == "balance":
        z, E, k = s["logits"].double(), case["E"], case["k"]
        cut = s["seq_offsets"].tolist()
        valid = torch.ones(z.shape[0], dtype=torch.bool, device="cuda") if s["token_mask"] is None else s["token_mask"]
        score = torch.softmax(z, 1) if case["scores"] == "softmax" else torch.sigmoid(z)
        p = score / score.sum(1, keepdim=True)
        dz, loss = torch.zeros_like(z), torch.zeros(1, dtype=torch.float64, device="cuda")
        full = [(a, b) for a, b in zip(cut, cut[1:]) if bool(valid[a:b].any())]
        for a, b in full:
            ok = valid[a:b]
            f = torch.bincount(s["topk_ids"][a:b][ok].reshape(-1).long(), minlength=E).double() / ok.sum()
            part = p[a:b][ok]
            loss += E * (f * part.mean(0)).sum() / len(full)
            c = E * f / ok.sum() / len(full)
            slope = 1.0 if case["scores"] == "softmax" else 1.0 - score[a:b][ok]
            dz[a:b][ok] = part * slope * (c - (part @ c)[:, None])
        return {"loss": loss, "counts": None, "dlogits": dz}
    cut = s["offsets"].tolist()
    parts = [(e, a, b) for e, (a, b) in enumerate(zip(cut, cut[1:])) if b > a]
    if op == "product":
        return torch.cat([_exact_slice(s["a"], s["w"], e, a, b) for e, a, b in parts])
    xq, h, y = _exact_rows(s["x_sorted"]), [], []
    for e, a, b in parts:
        g = _exact_slice(xq, s["W1"], e, a, b)
        if case["act"] == "swiglu":
            g = g * torch.sigmoid(g) * _exact_slice(xq, s["W3"], e, a, b)
        else:
            g = g + s["b1"][e].double()
            g = g * torch.special.ndtr(g)
        h.append(g)
    hq = _exact_rows(torch.cat(h))
    for e, a, b in parts:
        part = _exact_slice(hq, s["W2"], e, a, b)
        y.append(part if s["b2"] is None else part + s["b2"][e].double())
    return torch.cat(y)
