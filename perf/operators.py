"""Cases that time the layer's 8-bit operators and their plain forms.

Four paths, each as a program that serves a mixture-of-experts model calls it:

* ``route``: ``coli_moe_route_scored``.  Router logits to experts and weights: softmax or sigmoid
  scores, a selection bias, expert groups, top-k, renormalised weights.
* ``linear``: ``coli_quant_act_token`` and ``coli_gemm_q8``.  A dense projection in 8-bit integers
  with a scale for each token and one for each output channel.
* ``experts_in``: ``coli_quant_act_token`` and ``coli_gemm_q8_grouped``.  The routed experts' first
  product (gate and up stacked over the output rows) on the tokens routed to them.
* ``experts_out``: ``coli_swiglu_quant_token``, ``coli_gemm_q8_grouped`` and ``coli_moe_combine``.
  SwiGLU, the routed experts' second product and the weighted sum over each token's experts.

Where ``own`` is false, ``run`` computes the same in elementary torch operations.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoded token of a 256-expert layer: the smallest call, latency alone
        dict(name="route 1x256 sigmoid", op="route", tokens=1, experts=256, top_k=8, groups=8,
             topk_groups=4, score="sigmoid", group_score="top2", renorm=True, scale=2.5,
             dtype="f32", bias=True, off=0),
        # a long prefill chunk through a softmax router without groups, some experts switched off
        dict(name="route 16384x256 softmax", op="route", tokens=16384, experts=256, top_k=8,
             groups=1, topk_groups=1, score="softmax", group_score="max", renorm=True, scale=1.0,
             dtype="bf16", bias=False, off=5),
        # an odd batch through a grouped softmax router of few experts
        dict(name="route 1021x160 groups", op="route", tokens=1021, experts=160, top_k=6, groups=8,
             topk_groups=3, score="softmax", group_score="max", renorm=False, scale=16.0,
             dtype="f32", bias=False, off=0),
        # one decoded token through a projection of the layer's hidden size
        dict(name="linear 1x6144x2048", op="linear", tokens=1, cols=6144, rows=2048, dtype="bf16",
             bias=False, pad=0),
        # a batch of decoding sequences, with a bias and rows of a wider buffer
        dict(name="linear 61x6144x6144", op="linear", tokens=61, cols=6144, rows=6144,
             dtype="bf16", bias=True, pad=256),
        # a short prompt, an odd number of channels
        dict(name="linear 509x2048x6145", op="linear", tokens=509, cols=2048, rows=6145,
             dtype="f16", bias=False, pad=0),
        # a prefill chunk
        dict(name="linear 8192x6144x6144", op="linear", tokens=8192, cols=6144, rows=6144,
             dtype="bf16", bias=False, pad=0),
        # three tokens of a speculative verification through 256 experts
        dict(name="experts_in 3 tokens", op="experts_in", tokens=3, experts=256, top_k=8,
             cols=6144, rows=4096, dtype="bf16", dropped=0.0),
        # a prefill chunk through 256 experts
        dict(name="experts_in 4096 tokens", op="experts_in", tokens=4096, experts=256, top_k=8,
             cols=6144, rows=4096, dtype="bf16", dropped=0.0),
        # one token, float32 in and out
        dict(name="experts_out 1 token", op="experts_out", tokens=1, experts=256, top_k=8,
             cols=2048, rows=6144, dtype="f32", dropped=0.0),
        # an odd batch, the slots of the smallest weights dropped by an expert top-p
        dict(name="experts_out 333 tokens", op="experts_out", tokens=333, experts=64, top_k=8,
             cols=2048, rows=6144, dtype="bf16", dropped=0.3),
        # a prefill chunk through 256 experts
        dict(name="experts_out 4096 tokens", op="experts_out", tokens=4096, experts=256, top_k=8,
             cols=2048, rows=6144, dtype="bf16", dropped=0.0),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "linear", "linear", "experts_in", "experts_out"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _between(rng, 4, 512 // groups)
        experts = groups * per
        kept = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, kept * per))
        tokens = _between(rng, 1, min(16384, 16384 * 256 // experts))
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k,
                    groups=groups, topk_groups=kept, score=rng.choice(["sigmoid", "softmax"]),
                    group_score=rng.choice(["top2", "max"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5, 16.0]), dtype=dtype, bias=rng.random() < 0.5,
                    off=rng.choice([0, 0, 1, experts // 4]))
    while True:
        tokens = _between(rng, 1, 8192 if op == "linear" else 4096)
        cols = 32 * _between(rng, 4, 256)
        rows = _between(rng, 100, 8192)
        if op == "linear":
            case = dict(op=op, tokens=tokens, cols=cols, rows=rows, dtype=dtype,
                        bias=rng.random() < 0.5, pad=rng.choice([0, 0, 64, 1000]))
            if tokens * cols * rows <= 8192 * 6144 * 6144:
                return case
        else:
            experts = _between(rng, 8, 256)
            top_k = rng.randint(1, min(8, experts))
            case = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, cols=cols, rows=rows,
                        dtype=dtype, dropped=rng.choice([0.0, 0.0, 0.3]))
            if op == "experts_out":
                big = 32768 * 2048 * 6144, 256 * 2048 * 6144
            else:
                big = 32768 * 6144 * 4096, 256 * 6144 * 4096
            if tokens * top_k * cols * rows <= big[0] and experts * cols * rows <= big[1]:
                return case


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _codes(shape, g):
    """Int8 weight codes in [-127, 127], most of them small, as quantised normal weights are."""
    a = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-63, 65, generator=g)
    b = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-63, 64, generator=g)
    return a.add_(b).view(torch.uint8)


def _acts(rows, cols, dtype, g, pad=0):
    """Activations with a spread of their own for each channel, as rows of a wider buffer where
    ``pad`` is not zero."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols + pad, generator=g, device="cuda"))
    return x.to(dtype)[:, :cols]


def _scales(shape, g):
    return 0.02 / 32 * (0.5 + torch.rand(shape, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = dict(case=case)
    T = case["tokens"]
    if case["op"] == "route":
        E, k = case["experts"], case["top_k"]
        logits = 1.57 * torch.randn(T, E, generator=g, device="cuda")
        if case["off"]:  # experts that are switched off for the whole batch
            dead = torch.randperm(E, generator=g, device="cuda")[:case["off"]]
            logits[:, dead] = -math.inf
        s["logits"] = logits.to(dt)
        s["bias"] = 0.01 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, device="cuda")
        if own:
            import quantized_moe_coli_amd as C
            s["C"] = C
            s["cfg"] = C.score_cfg(
                E, k, case["groups"], case["topk_groups"],
                score=C.SCORE_SOFTMAX if case["score"] == "softmax" else C.SCORE_SIGMOID,
                group_score=C.GROUP_TOP2 if case["group_score"] == "top2" else C.GROUP_MAX,
                norm_topk_prob=int(case["renorm"]), routed_scaling_factor=case["scale"])
        return s

    K, N = case["cols"], case["rows"]
    if own:
        import quantized_moe_coli_amd as C
        s["C"] = C
        if case["op"] == "experts_out":  # the products as they are computed: only their sum is rounded
            s["o32"] = torch.empty(T * case["top_k"], N, device="cuda")
    if case["op"] == "linear":
        s["x"] = _acts(T, K, dt, g, case["pad"])
        s["w"], s["ws"] = _codes((N, K), g), _scales(N, g)
        s["bias"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["q"] = torch.empty(T, K, dtype=torch.int8, device="cuda")
        s["qs"] = torch.empty(T, device="cuda")
        s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
        return s

    # the routing's tables, which one dispatch makes for both of a layer's products
    E, k = case["experts"], case["top_k"]
    P = T * k
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    if case["dropped"]:
        off = torch.rand(T, k, generator=g, device="cuda") < case["dropped"]
        off[:, 0] = False
        idx, w = idx.masked_fill(off, -1), w.masked_fill(off, 0.0)
    s["idx"], s["wt"] = idx.contiguous(), w / w.sum(1, keepdim=True)
    key = torch.where(idx < 0, E, idx).reshape(-1).long()
    s["perm"] = torch.argsort(key, stable=True).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    s["offs"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())
    s["w"], s["ws"] = _codes((E, N, K), g), _scales((E, N), g)
    if case["op"] == "experts_in":
        s["x"] = _acts(T, K, dt, g)
        s["q"] = torch.empty(T, K, dtype=torch.int8, device="cuda")
        s["qs"] = torch.empty(T, device="cuda")
        s["y"] = torch.zeros(P, N, dtype=dt, device="cuda")  # rows of dropped slots stay zero
    else:
        gu = _acts(P, 2 * K, dt, g)
        s["g"], s["u"] = gu[:, :K], gu[:, K:]
        s["q"] = torch.empty(P, K, dtype=torch.int8, device="cuda")
        s["qs"] = torch.empty(P, device="cuda")
        s["o"] = torch.empty(P, N, dtype=dt, device="cuda")
        s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    C, op = s["C"], s["case"]["op"]
    if op == "route":
        C.coli_moe_route_scored(s["cfg"], s["logits"], s["bias"], s["idx"], s["w"])
        return s["idx"], s["w"]
    if op == "linear":
        C.coli_quant_act_token(s["x"], s["q"], s["qs"])
        C.coli_gemm_q8(s["q"], s["qs"], s["w"], s["ws"], s["y"], bias=s["bias"])
        return s["y"]
    if op == "experts_in":
        C.coli_quant_act_token(s["x"], s["q"], s["qs"])
        C.coli_gemm_q8_grouped(s["q"], s["qs"], s["w"], s["ws"], s["offs"], s["perm"], s["y"],
                               fan=s["case"]["top_k"])
        return s["y"]
    C.coli_swiglu_quant_token(s["g"], s["u"], s["q"], s["qs"])
    C.coli_gemm_q8_grouped(s["q"], s["qs"], s["w"], s["ws"], s["offs"], s["perm"], s["o32"])
    C.coli_moe_combine(s["o32"], s["idx"], s["wt"], s["y"])
    return s["y"]


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _route_plain(s):
    c = s["case"]
    T, E, k, G = c["tokens"], c["experts"], c["top_k"], c["groups"]
    per = E // G
    lg = s["logits"].double()
    on = lg > -math.inf  # an expert whose logit is -inf (or NaN) is off
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-lg))
    else:
        top = torch.where(on, lg, -math.inf).amax(1, keepdim=True)
        e = torch.where(on, torch.exp(lg - top), 0.0)
        p = e / e.sum(1, keepdim=True)
    p = torch.where(on, p, 0.0).float()
    sel = p if s["bias"] is None else p + s["bias"]
    sel = torch.where(on, sel, -math.inf)
    if c["topk_groups"] < G:
        top = sel.view(T, G, per).sort(dim=2, descending=True, stable=True).values
        score = top[:, :, 0]
        if c["group_score"] == "top2" and per > 1:
            score = score + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], 0.0)
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=lg.device).scatter_(1, kept, True)
        sel = torch.where(mask[:, :, None].expand(T, G, per).reshape(T, E), sel, -math.inf)
    got = sel.sort(dim=1, descending=True, stable=True)
    idx = got.indices[:, :k]
    alive = got.values[:, :k] > -math.inf
    w = torch.where(alive, p.gather(1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(alive, idx, -1).to(torch.int32), w * c["scale"]


def _quant_plain(x):
    """A token's codes as float32 whole numbers, and its scale."""
    x = x.float()
    scale = x.abs().amax(1) / 127
    q = torch.round(x / scale[:, None]).clamp(-127, 127)
    return torch.where(scale[:, None] > 0, q, 0.0), scale


def _grouped_plain(s, q, qs, fan):
    """y[p] = codes of row p / fan times the weights of p's expert, scaled; [P, N] in float32, and
    which rows belong to an expert."""
    E = s["case"]["experts"]
    offs, perm = s["offs"].long(), s["perm"].long()
    P, cap = perm.numel(), s["most"]
    at = torch.arange(P, device=q.device)
    expert = torch.searchsorted(offs[1:], at, right=True)
    live = at < offs[-1]
    expert = torch.where(live, expert, E - 1)
    place = torch.where(live, at - offs[expert], cap)
    row = torch.div(perm, fan, rounding_mode="floor")
    if P <= E:  # few pairs: only the weights of their experts are taken
        y = torch.bmm(s["w"].view(torch.int8)[expert].float(), q[row][:, :, None])[:, :, 0]
    else:
        y = _padded_products(s, q, expert, place, row)
    y = y * qs[row][:, None] * s["ws"][expert]
    out = torch.zeros_like(y)
    out[perm] = y
    alive = torch.zeros(P, dtype=torch.bool, device=q.device)
    alive[perm] = live
    return out, alive


def _padded_products(s, q, expert, place, row):
    """The products of every pair with its expert's weights, each expert's rows padded to the
    longest."""
    E, cap = s["case"]["experts"], s["most"]
    slots = q.new_zeros(E, cap + 1, q.shape[1])
    slots[expert, place] = q[row]
    slots = slots[:, :cap].transpose(1, 2).contiguous()
    acc = torch.bmm(s["w"].view(torch.int8).float(), slots)  # [E, N, cap]
    return acc.transpose(1, 2)[expert, place.clamp(max=cap - 1)]


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op == "route":
        return _route_plain(s)
    if op == "linear":
        q, qs = _quant_plain(s["x"])
        y = (q @ s["w"].view(torch.int8).float().t()) * qs[:, None] * s["ws"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(dt)
    if op == "experts_in":
        q, qs = _quant_plain(s["x"])
        y, alive = _grouped_plain(s, q, qs, c["top_k"])
        return torch.where(alive[:, None], y, 0.0).to(dt)
    g = s["g"].double()
    h = (g / (1 + torch.exp(-g)) * s["u"].double()).float()  # codes next to a border: in 64 bits
    q, qs = _quant_plain(h)
    o, alive = _grouped_plain(s, q, qs, 1)
    o = torch.where(alive[:, None], o, 0.0).view(c["tokens"], c["top_k"], c["rows"])
    return (o * s["wt"][:, :, None]).sum(1).to(dt)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    T = case["tokens"]
    if case["op"] == "route":
        E, k = case["experts"], case["top_k"]
        return dict(bytes=T * E * b + T * k * 8 + (4 * E if case["bias"] else 0), flops=4 * T * E)
    K, N = case["cols"], case["rows"]
    if case["op"] == "linear":
        return dict(bytes=T * K * b + N * K + 4 * N * (2 if case["bias"] else 1) + T * N * b,
                    flops=2 * T * N * K)
    E, k = case["experts"], case["top_k"]
    pairs = T * (1 + (k - 1) * (1 - case["dropped"]))
    read = E * (1 - (1 - 1 / E) ** pairs)  # experts that some token is routed to
    weights = read * N * (K + 4)
    if case["op"] == "experts_in":
        return dict(bytes=int(T * K * b + weights + pairs * (4 + N * b)),
                    flops=int(2 * pairs * N * K))
    return dict(bytes=int(2 * pairs * K * b + weights + 12 * pairs + T * N * b),
                flops=int(2 * pairs * N * K))


def _exact_codes(x64):
    """Codes and scale of the definition: the scale and each quotient rounded once to 32 bits."""
    peak = x64.abs().max(dim=1).values
    scale = (peak / 127.0).to(torch.float32).double()
    quot = torch.where(scale[:, None] == 0, torch.zeros_like(x64), x64 / scale[:, None])
    return quot.to(torch.float32).double().round().clamp(-127.0, 127.0), scale


def _exact_product(s, codes, scale, fan):
    """The experts' products one expert at a time, in 64 bits; rows of no expert are zero."""
    c = s["case"]
    y = torch.zeros(c["tokens"] * c["top_k"], c["rows"], dtype=torch.float64, device="cuda")
    flat = s["idx"].reshape(-1).long()
    for e in range(c["experts"]):
        pair = (flat == e).nonzero().reshape(-1)
        if pair.numel():
            a = codes[pair // fan]
            m = a @ s["w"][e].view(torch.int8).to(torch.float64).T.contiguous()
            y[pair] = m * scale[pair // fan].unsqueeze(1) * s["ws"][e].double().unsqueeze(0)
    return y


def _exact_route(s):
    c = s["case"]
    G, per = c["groups"], c["experts"] // c["groups"]
    logits = s["logits"].to(torch.float64)
    off = logits.isneginf() | logits.isnan()
    if c["score"] == "softmax":
        prob = torch.softmax(logits.masked_fill(off, -math.inf), dim=1)
    else:
        prob = torch.sigmoid(logits)
    prob = prob.masked_fill(off, 0.0)
    pick = prob.float()  # the selection goes by scores rounded once to 32 bits
    if s["bias"] is not None:
        pick = pick + s["bias"]
    pick = pick.masked_fill(off, -math.inf)

    def first(v, n):
        """The n largest of each row, the lowest index first among equals."""
        v, got = v.clone(), []
        for _ in range(n):
            big = v.amax(1, keepdim=True)
            at = (v == big).int().argmax(1, keepdim=True)
            got.append(torch.where(big.isneginf(), -1, at))
            v.scatter_(1, at, -math.inf)
        return torch.cat(got, 1)

    if c["topk_groups"] < G:
        by = pick.view(-1, G, per)
        best = by.amax(2)
        if c["group_score"] == "top2" and per > 1:
            at = by.argmax(2, keepdim=True)
            second = by.scatter(2, at, -math.inf).amax(2)
            best = torch.where(second.isneginf(), best, best + second)
        chosen = first(best, c["topk_groups"])
        keep = (chosen[:, :, None] == torch.arange(G, device="cuda")).any(1)
        pick = pick.masked_fill(~keep.repeat_interleave(per, 1), -math.inf)
    idx = first(pick, c["top_k"])
    w = prob.gather(1, idx.clamp(min=0)).masked_fill(idx < 0, 0.0)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    return idx.to(torch.int32), w * c["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "linear":
        codes, scale = _exact_codes(s["x"].to(torch.float64))
        y = codes @ s["w"].view(torch.int8).to(torch.float64).T.contiguous()
        y = y * scale.unsqueeze(1) * s["ws"].to(torch.float64).unsqueeze(0)
        return y if s["bias"] is None else y + s["bias"].to(torch.float64)
    if case["op"] == "experts_in":
        codes, scale = _exact_codes(s["x"].to(torch.float64))
        return _exact_product(s, codes, scale, case["top_k"])
    gate, up = s["g"].to(torch.float64), s["u"].to(torch.float64)
    h = (gate * torch.sigmoid(gate) * up).to(torch.float32).to(torch.float64)
    codes, scale = _exact_codes(h)
    o = _exact_product(s, codes, scale, 1).view(case["tokens"], case["top_k"], case["rows"])
    return torch.matmul(s["wt"].to(torch.float64).unsqueeze(1), o).squeeze(1)
