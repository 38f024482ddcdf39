"""What is measured of the 8-bit expert products and the router's training operators.

A case is one pass through one operator: the plan that sorts (token, choice) pairs by expert, the
balance loss with its gradient, the quantiser to E4M3 codes with a scale per block of 128, and the
product of two such operands, plain or per expert.  Sizes are those of the routed layer (hidden 2048,
inter 512, 512 experts, 10 choices a token), of its small test layer (64 experts, 8 choices) and
generic ones.

  run(), own = False   the operators in elementary torch operations, in 32 bits
  run(), own = True    the framework's calls
  exact()              the definitions in 64 bits
"""
import math

import torch

own = False

BLOCK = 128          # columns that share a scale (weights: 128 x 128)
E4M3_MAX = 448.0
AMAX_FLOOR = E4M3_MAX * 2.0 ** -126  # blocks below it share the scale 2^-126
WORKSPACE = 4 << 20  # a user's program keeps one scratch buffer for the balance loss


def listed():
    return [
        # a speculative-verify batch: the plan's latency
        {"name": "plan_verify", "op": "plan", "tokens": 8, "experts": 512, "top_k": 10, "skew": 0.3, "padded": 0},
        # a prefill chunk's plan, some of its tokens padding
        {"name": "plan_prefill", "op": "plan", "tokens": 8192, "experts": 512, "top_k": 10, "skew": 0.3, "padded": 77},
        # a small layer's micro-batch in training, fp32 logits
        {"name": "balance_small", "op": "balance", "tokens": 64, "experts": 64, "top_k": 8, "skew": 0.3, "padded": 3,
         "dtype": "f32"},
        # a training micro-batch over every expert, bf16 logits
        {"name": "balance_train", "op": "balance", "tokens": 8192, "experts": 512, "top_k": 10, "skew": 0.3,
         "padded": 500, "dtype": "bf16"},
        # one token's activations, gathered for its experts
        {"name": "quantize_token", "op": "quantize", "tokens": 1, "rows": 10, "cols": 2048, "swiglu": False,
         "dtype": "bf16"},
        # a prefill chunk between gate/up and down: SwiGLU and quantisation in one pass
        {"name": "quantize_swiglu", "op": "quantize", "tokens": 0, "rows": 81920, "cols": 512, "swiglu": True,
         "dtype": "bf16"},
        # one token through the always-on expert's gate/up product
        {"name": "product_token", "op": "product", "rows": 1, "n": 1024, "k": 2048, "out": "bf16"},
        # odd sizes in every direction, fp32 results
        {"name": "product_odd", "op": "product", "rows": 333, "n": 1000, "k": 1111, "out": "f32"},
        # a prefill chunk through a dense projection: arithmetic bound
        {"name": "product_prefill", "op": "product", "rows": 8192, "n": 4096, "k": 4096, "out": "bf16"},
        # one token's gate/up over its ten experts
        {"name": "experts_token", "op": "experts", "tokens": 1, "experts": 512, "top_k": 10, "n": 1024, "k": 2048,
         "skew": 0.3, "padded": 0, "out": "bf16"},
        # a decode batch: most experts read for one or two rows each
        {"name": "experts_batch", "op": "experts", "tokens": 64, "experts": 512, "top_k": 10, "n": 1024, "k": 2048,
         "skew": 0.3, "padded": 5, "out": "f32"},
        # a prefill chunk: ragged groups of about 160 rows
        {"name": "experts_prefill", "op": "experts", "tokens": 8192, "experts": 512, "top_k": 10, "n": 1024,
         "k": 2048, "skew": 0.3, "padded": 100, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "balance", "quantize", "product", "product", "experts", "experts"])
    if op in ("plan", "balance"):
        tokens, experts = _log(rng, 1, 8192), _log(rng, 4, 512)
        c = {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(10, experts)),
             "skew": rng.choice([0.0, 0.3, 0.6]), "padded": rng.randint(0, tokens // 4)}
        if op == "balance":
            c["dtype"] = rng.choice(["f32", "bf16"])
        return c
    if op == "quantize":
        swiglu = rng.random() < 0.5
        rows = _log(rng, 1, 81920)
        cols = _log(rng, 64, min(4096, 81920 * 512 // rows))
        return {"op": op, "tokens": 0 if swiglu else _log(rng, 1, 8192), "rows": rows, "cols": cols, "swiglu": swiglu,
                "dtype": rng.choice(["f32", "bf16"])}
    if op == "product":
        return {"op": op, "rows": _log(rng, 1, 8192), "n": _log(rng, 64, 4096), "k": _log(rng, 64, 4096),
                "out": rng.choice(["f32", "bf16"])}
    tokens, experts = _log(rng, 1, 8192), _log(rng, 8, 512)
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(10, experts)),
            "n": _log(rng, 64, 1024), "k": _log(rng, 64, 2048), "skew": rng.choice([0.0, 0.3, 0.6]),
            "padded": rng.randint(0, tokens // 4), "out": rng.choice(["f32", "bf16"])}


# ---- inputs --------------------------------------------------------------------

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _routing(case, g):
    """Router logits, the chosen experts of each token (-1 for padding) and which tokens are real."""
    T, E = case["tokens"], case["experts"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += case["skew"] * torch.randn(E, generator=g, device="cuda")
    idx = logits.topk(case["top_k"], dim=1).indices.to(torch.int32)
    valid = torch.ones(T, dtype=torch.bool, device="cuda")
    if case["padded"]:
        valid[torch.randperm(T, generator=g, device="cuda")[:case["padded"]]] = False
    return logits, torch.where(valid[:, None], idx, -1).contiguous(), valid


def _codes_buffer(lead, cols):
    """Code rows start on 16-byte boundaries: [..., cols] in rows of the next multiple of 16 bytes."""
    width = -(-cols // 16) * 16
    return torch.zeros(*lead, width, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[..., :cols]


def _quantized_rows(rows, cols, g):
    """Activations as the quantiser leaves them: codes [rows, cols], scales [blocks, rows]."""
    nb = -(-cols // BLOCK)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    amax = x.abs().amax(2).clamp_min(AMAX_FLOOR)
    codes = _codes_buffer((rows,), cols)
    codes.copy_((x * (E4M3_MAX / amax)[..., None]).view(rows, -1)[:, :cols])
    return codes, (amax / E4M3_MAX).t().contiguous()


def _quantized_weights(groups, n, k, g):
    """Weights N(0, 0.02^2) as E4M3 codes [groups, n, k] with a scale per 128 x 128 block."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    codes = _codes_buffer((groups, n), k)
    scales = torch.empty(groups, nb, kb, device="cuda")
    step = max(1, (1 << 26) // (n * k))
    for a in range(0, groups, step):
        b = min(groups, a + step)
        w = 0.02 * torch.randn(b - a, n, k, generator=g, device="cuda")
        w = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
        w = w.view(b - a, nb, BLOCK, kb, BLOCK)
        amax = w.abs().amax((2, 4)).clamp_min(AMAX_FLOOR)
        w = (w * (E4M3_MAX / amax)[:, :, None, :, None]).view(b - a, nb * BLOCK, kb * BLOCK)
        codes[a:b].copy_(w[:, :n, :k])
        scales[a:b] = amax / E4M3_MAX
    return codes, scales


def _sorted_groups(idx, experts):
    """Row offsets [experts + 1] of the pairs sorted by expert."""
    flat = idx.view(-1).long()
    counts = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    counts.scatter_add_(0, torch.where(flat < 0, experts, flat), torch.ones_like(flat))
    offsets = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    offsets[1:] = counts[:experts].cumsum(0)
    return offsets


def prepare(case, seed):
    g = _generator(seed)
    op, s = case["op"], dict(case)
    if op in ("plan", "balance"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        logits, s["idx"], s["valid"] = _routing(case, g)
        s["counts"] = torch.empty(E if op == "plan" else E + 1, dtype=torch.int32, device="cuda")
        if op == "plan":
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            s["rows"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
            s["slots"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        else:
            s["logits"] = logits.to(_dtype(case["dtype"]))
            s["dlogits"] = torch.empty_like(s["logits"])
            s["prob_mean"] = torch.empty(E, device="cuda")
            s["loss"] = torch.empty(1, device="cuda")
            s["dloss"] = torch.rand(1, generator=g, device="cuda") * 0.01 + 1e-3  # the loss's weight in training
            s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    elif op == "quantize":
        R, C = case["rows"], case["cols"]
        if case["swiglu"]:
            s["x"] = torch.randn(R, 2 * C, generator=g, device="cuda").to(_dtype(case["dtype"]))
            s["index"] = None
        else:
            s["x"] = torch.randn(case["tokens"], C, generator=g, device="cuda").to(_dtype(case["dtype"]))
            s["index"] = torch.randint(0, case["tokens"], (R,), generator=g, device="cuda", dtype=torch.int32)
        s["codes"] = _codes_buffer((R,), C)
        s["scales"] = torch.empty(-(-C // BLOCK), R, device="cuda")
    elif op == "product":
        s["a"], s["a_scale"] = _quantized_rows(case["rows"], case["k"], g)
        b, b_scale = _quantized_weights(1, case["n"], case["k"], g)
        s["b"], s["b_scale"] = b[0], b_scale[0]
        s["y"] = torch.zeros(case["rows"], case["n"], dtype=_dtype(case["out"]), device="cuda")
    else:
        E, R = case["experts"], case["tokens"] * case["top_k"]
        _, idx, _ = _routing(case, g)
        offsets = _sorted_groups(idx, E)
        s["offsets"] = offsets.to(torch.int32)
        s["a"], s["a_scale"] = _quantized_rows(R, case["k"], g)
        s["b"], s["b_scale"] = _quantized_weights(E, case["n"], case["k"], g)
        s["y"] = torch.zeros(R, case["n"], dtype=_dtype(case["out"]), device="cuda")
        # the plain form's plan: the experts that have rows, and the largest group
        counts = offsets[1:] - offsets[:-1]
        s["active"] = counts.nonzero().view(-1)
        s["largest"] = int(counts.max())
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    return {"plan": _plan, "balance": _balance, "quantize": _quantize, "product": _product,
            "experts": _experts}[state["op"]](state)


def _plan(s):
    if own:
        import block_quantized_expert_moe_b200 as bq
        bq.moe_expert_plan(s["idx"], s["experts"], s["counts"], s["offsets"], s["rows"], s["slots"])
        return {"counts": s["counts"], "offsets": s["offsets"], "rows": s["rows"], "slots": s["slots"]}
    E, k = s["experts"], s["top_k"]
    flat = s["idx"].view(-1).long()
    used = (flat >= 0) & (flat < E)
    key = torch.where(used, flat, E)
    sorted_key, order = torch.sort(key, stable=True)  # slot -> pair
    counts = torch.zeros(E + 1, dtype=torch.long, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = counts[:E].cumsum(0)
    rows = torch.where(sorted_key < E, order // k, -1)
    slots = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=flat.device))
    slots = torch.where(used, slots, -1).view(-1, k)
    return {"counts": counts[:E].int(), "offsets": offsets, "rows": rows.int(), "slots": slots.int()}


def _balance(s):
    if own:
        import block_quantized_expert_moe_b200 as bq
        bq.moe_balance_loss(s["logits"], s["idx"], s["counts"], s["prob_mean"], s["loss"], s["workspace"],
                            valid=s["valid"])
        bq.moe_balance_loss_backward(s["logits"], s["counts"], s["top_k"], s["dloss"], s["dlogits"],
                                     valid=s["valid"])
        return {"loss": s["loss"], "counts": s["counts"], "prob_mean": s["prob_mean"], "dlogits": s["dlogits"]}
    T, E, k = s["tokens"], s["experts"], s["top_k"]
    valid = s["valid"][:, None]
    logits = s["logits"].float()
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    p = torch.where(valid, e / e.sum(1, keepdim=True), 0.0)
    flat = torch.where(valid & (s["idx"] >= 0) & (s["idx"] < E), s["idx"], E).view(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.long, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    counts[E] = s["valid"].sum()
    n = counts[E].clamp_min(1).float()
    share = counts[:E].float() * (E / (k * n))
    prob_mean = p.sum(0) / n
    loss = (share * prob_mean).sum().view(1)
    dlogits = (s["dloss"] / n) * p * (share - (p * share).sum(1, keepdim=True))
    return {"loss": loss, "counts": counts.int(), "prob_mean": prob_mean, "dlogits": dlogits.to(s["logits"].dtype)}


def _quantize(s):
    if own:
        import block_quantized_expert_moe_b200 as bq
        bq.moe_fp8_quantize(s["x"], s["codes"], s["scales"], rows=s["index"], swiglu=s["swiglu"])
        return {"codes": s["codes"], "scales": s["scales"]}
    R, C = s["rows"], s["cols"]
    nb = -(-C // BLOCK)
    x = s["x"].float()
    if s["swiglu"]:
        gate, up = x[:, :C], x[:, C:]
        x = gate / (1 + torch.exp(-gate)) * up
    else:
        x = x[s["index"].long()]
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - C)).view(R, nb, BLOCK)
    amax = x.abs().amax(2).clamp_min(AMAX_FLOOR)
    codes = (x * (E4M3_MAX / amax)[..., None]).view(R, -1)[:, :C].to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": (amax / E4M3_MAX).t().contiguous()}


def _values(codes, row_scale):
    """codes [..., rows, k] times a scale per row and 128 columns, row_scale [..., rows, blocks]."""
    k = codes.shape[-1]
    return codes.float() * row_scale.repeat_interleave(BLOCK, -1)[..., :k]


def _weights(codes, scale):
    return _values(codes, scale.repeat_interleave(BLOCK, -2)[..., :codes.shape[-2], :])


def _product(s):
    if own:
        import block_quantized_expert_moe_b200 as bq
        bq.moe_fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["y"])
        return s["y"]
    a, b = _values(s["a"], s["a_scale"].t()), _weights(s["b"], s["b_scale"])
    return torch.matmul(a, b.t()).to(s["y"].dtype)


def _experts(s):
    if own:
        import block_quantized_expert_moe_b200 as bq
        bq.moe_fp8_grouped_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], s["offsets"], s["y"])
        return s["y"]
    # every group with rows padded to the largest one: one batched product; rows behind the last
    # group keep what the buffer held
    offsets, active = s["offsets"].long(), s["active"]
    R = s["a"].shape[0]
    a = _values(s["a"], s["a_scale"].t())
    b = _weights(s["b"].view(torch.uint8)[active].view(torch.float8_e4m3fn), s["b_scale"][active])
    at = offsets[active][:, None] + torch.arange(s["largest"], device=a.device)
    y = torch.bmm(a[at.clamp_max(R - 1)], b.transpose(1, 2))
    row = torch.arange(R, device=a.device)
    expert = (torch.searchsorted(offsets, row, right=True) - 1).clamp_max(s["experts"] - 1)
    place = torch.searchsorted(active, expert).clamp_max(active.numel() - 1)
    y = y[place, (row - offsets[expert]).clamp(0, s["largest"] - 1)].to(s["y"].dtype)
    return torch.where((row < offsets[-1])[:, None], y, s["y"])


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    if op == "plan":
        pairs = case["tokens"] * case["top_k"]
        return {"bytes": 12 * pairs + 8 * case["experts"], "flops": 0}
    if op == "balance":
        n = case["tokens"] * case["experts"]
        size = 2 if case["dtype"] == "bf16" else 4
        # forward and backward are calls of their own with training's work between them: logits are read by each
        return {"bytes": 3 * n * size + 4 * case["tokens"] * case["top_k"] + 2 * case["tokens"] + 16 * case["experts"],
                "flops": 14 * n}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        read = 2 * R * C * size if case["swiglu"] else min(R, case["tokens"]) * C * size + 4 * R
        return {"bytes": read + R * C + 4 * R * -(-C // BLOCK), "flops": R * C * (8 if case["swiglu"] else 2)}
    n, k = case["n"], case["k"]
    size = 2 if case["out"] == "bf16" else 4
    blocks = -(-k // BLOCK)
    if op == "product":
        R, matrices = case["rows"], 1
    else:
        T, E, chosen = case["tokens"] - case["padded"], case["experts"], case["top_k"]
        R, matrices = T * chosen, E * (1 - (1 - chosen / E) ** T)  # experts with at least one row, on average
    return {"bytes": int(matrices * (n * k + 4 * blocks * -(-n // BLOCK)) + R * (k + 4 * blocks + n * size)),
            "flops": 2 * R * n * k}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "balance":
        E, k = case["experts"], case["top_k"]
        keep = s["valid"].nonzero().view(-1)
        n = max(1, keep.numel())
        p = torch.softmax(s["logits"][keep].double(), 1)
        chosen = s["idx"][keep].view(-1).long()
        share = torch.bincount(chosen[chosen >= 0], minlength=E).double() * E / (k * n)
        mean = p.sum(0) / n
        d = torch.zeros(case["tokens"], E, dtype=torch.float64, device="cuda")
        d[keep] = s["dloss"].double() / n * (p * share - p * (p @ share)[:, None])
        return {"loss": (share @ mean).view(1), "counts": None, "prob_mean": mean, "dlogits": d}
    if op == "quantize":
        C = case["cols"]
        x = s["x"].double()
        x = x[:, :C] * torch.sigmoid(x[:, :C]) * x[:, C:] if case["swiglu"] else x[s["index"].long()]
        codes, scales = torch.empty_like(x), torch.empty(-(-C // BLOCK), x.shape[0], dtype=torch.float64, device="cuda")
        for b in range(scales.shape[0]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            scales[b] = part.abs().max(1).values.clamp_min(AMAX_FLOOR) / E4M3_MAX
            v = part / scales[b][:, None]
            # nearest E4M3 value: 3 mantissa bits, exponents from -6 (below it, steps of 2^-9)
            e = torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent.double() - 1
            step = torch.exp2(e - 3)
            codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(v / step) * step
        return {"codes": codes, "scales": scales}

    def product(a, a_scale, b, b_scale):
        """Block by block of 128 columns: sum of scale times scale times the codes' product."""
        y = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
        for i in range(b_scale.shape[1]):
            at = slice(i * BLOCK, (i + 1) * BLOCK)
            part = a[:, at].to(torch.float64) @ b[:, at].to(torch.float64).t()
            per_column = b_scale[:, i].double().repeat_interleave(BLOCK)[:b.shape[0]]
            y += part * a_scale[i].double()[:, None] * per_column[None]
        return y

    if op == "product":
        return product(s["a"], s["a_scale"], s["b"], s["b_scale"])
    y = s["y"].double()
    bounds = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            y[lo:hi] = product(s["a"][lo:hi], s["a_scale"][:, lo:hi], s["b"][e], s["b_scale"][e])
    return y
