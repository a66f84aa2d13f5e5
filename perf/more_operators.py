"""Cases that time the residual's normalisation and the 8-bit projection with low-rank adapters, and
their plain forms.

Two operators, each as a program that serves a model calls it:

* ``norm``: ``coli_rmsnorm_quant_token``.  The residual's addition, the root-mean-square norm of the
  sum, and the norm in 8 bits with a scale for each token (the products' operand), in the
  activations' type, or both.
* ``lora``: ``coli_gemm_q8_lora``.  A projection in 8 bits that all tokens share, and beside it the
  low-rank adapters of the requests that the tokens belong to, many adapters in one call.

Where ``own`` is false, ``run`` computes the same in elementary torch operations.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # one decoded token in front of a projection: the smallest call, latency alone
        dict(name="norm 1x6144 codes", op="norm", tokens=1, cols=6144, dtype="bf16", res=True,
             gain=True, out="codes", pad=0),
        # three tokens of a speculative verification, in front of a layer that takes fp32 rows
        dict(name="norm 3x6144 f32", op="norm", tokens=3, cols=6144, dtype="f32", res=True,
             gain=False, out="rows", pad=0),
        # every head of a prefill chunk's keys: many short rows
        dict(name="norm 65536x128 rows", op="norm", tokens=65536, cols=128, dtype="f16", res=False,
             gain=True, out="rows", pad=0),
        # an odd batch with an odd row length, rows of a wider buffer
        dict(name="norm 1021x1001 rows", op="norm", tokens=1021, cols=1001, dtype="bf16", res=True,
             gain=True, out="rows", pad=23),
        # a prefill chunk: the codes for the projections, and the rows for a router and adapters
        dict(name="norm 8192x6144 both", op="norm", tokens=8192, cols=6144, dtype="bf16", res=True,
             gain=True, out="both", pad=0),
        # one decoded token of one request
        dict(name="lora 1x6144x2048 r16", op="lora", tokens=1, cols=6144, rows=2048, rank=16,
             adapters=8, used=1, order="mixed", bare=0.0, dtype="bf16", bias=False, pad=0),
        # a batch of decoding requests, nearly each with an adapter of its own
        dict(name="lora 61x6144x6144 r16", op="lora", tokens=61, cols=6144, rows=6144, rank=16,
             adapters=64, used=64, order="mixed", bare=0.1, dtype="bf16", bias=True, pad=0),
        # float32 activations, few adapters, some requests without one
        dict(name="lora 200x6144x4096 r8", op="lora", tokens=200, cols=6144, rows=4096, rank=8,
             adapters=16, used=5, order="mixed", bare=0.3, dtype="f32", bias=False, pad=0),
        # short prompts of seven requests, an odd number of channels, rows of a wider buffer
        dict(name="lora 509x2048x6145 r32", op="lora", tokens=509, cols=2048, rows=6145, rank=32,
             adapters=32, used=7, order="requests", bare=0.0, dtype="f16", bias=False, pad=256),
        # a scheduler's mixed batch whose tokens do not lie together by request
        dict(name="lora 2047x2048x6144 r24", op="lora", tokens=2047, cols=2048, rows=6144, rank=24,
             adapters=48, used=48, order="mixed", bare=0.1, dtype="bf16", bias=False, pad=0),
        # a prefill chunk of eight requests with large adapters
        dict(name="lora 8192x6144x6144 r64", op="lora", tokens=8192, cols=6144, rows=6144, rank=64,
             adapters=16, used=8, order="requests", bare=0.0, dtype="bf16", bias=False, pad=0),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if rng.random() < 0.4:
        out = rng.choice(["codes", "both", "rows"])
        while True:
            cols = _between(rng, 64, 16384) if out == "rows" else 32 * _between(rng, 2, 512)
            tokens = _between(rng, 1, 65536)
            if tokens * cols * (2 if dtype == "f32" else 1) <= 8192 * 6144:
                return dict(op="norm", tokens=tokens, cols=cols, dtype=dtype,
                            res=rng.random() < 0.7, gain=rng.random() < 0.8, out=out,
                            pad=rng.choice([0, 0, 64, 7]))
    while True:
        tokens = _between(rng, 1, 8192)
        cols = 32 * _between(rng, 4, 256)
        rows = _between(rng, 100, 8192)
        rank = 8 * _between(rng, 1, 16)
        adapters = _between(rng, 1, 256)
        used = min(_between(rng, 1, adapters), tokens)
        if (tokens * cols * rows * (2 if dtype == "f32" else 1) <= 8192 * 6144 * 6144
                and adapters * rank <= 2048 and tokens * rank <= 8192 * 64):
            return dict(op="lora", tokens=tokens, cols=cols, rows=rows, rank=rank,
                        adapters=adapters, used=used, order=rng.choice(["requests", "mixed"]),
                        bare=rng.choice([0.0, 0.1, 0.3]), dtype=dtype, bias=rng.random() < 0.5,
                        pad=rng.choice([0, 0, 64, 1000]))


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _acts(rows, cols, dtype, g, pad=0):
    """Activations with a spread of their own for each channel, as rows of a wider buffer where
    ``pad`` is not zero."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(cols + pad, generator=g, device="cuda"))
    return x.to(dtype)[:, :cols]


def _codes(shape, g):
    """Int8 weight codes in [-127, 127], most of them small, as quantised normal weights are."""
    a = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-63, 65, generator=g)
    b = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-63, 64, generator=g)
    return a.add_(b).view(torch.uint8)


def _adapter_ids(case, g):
    """Each token's adapter, or -1: requests one after another, or tokens in any order."""
    T, used = case["tokens"], case["used"]
    mine = torch.randperm(case["adapters"], generator=g, device="cuda")[:used]
    pick = torch.randint(0, used, (T,), generator=g, device="cuda")
    if case["order"] == "requests":
        pick = pick.sort().values
    ids = mine[pick]
    bare = torch.rand(T, generator=g, device="cuda") < case["bare"]
    return ids.masked_fill(bare, -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    T, K = case["tokens"], case["cols"]
    s = dict(case=case)
    if own:
        import quantized_moe_coli_amd as C
        s["C"] = C
    if case["op"] == "norm":
        s["x"] = _acts(T, K, dt, g, case["pad"])
        s["res"] = 4 * _acts(T, K, dt, g, case["pad"]) if case["res"] else None
        s["gain"] = 1 + 0.2 * torch.randn(K, generator=g, device="cuda") if case["gain"] else None
        s["h"] = torch.empty(T, K, dtype=dt, device="cuda") if case["res"] else None
        s["y"] = torch.empty(T, K, dtype=dt, device="cuda") if case["out"] != "codes" else None
        codes = case["out"] != "rows"
        s["q"] = torch.empty(T, K, dtype=torch.int8, device="cuda") if codes else None
        s["s"] = torch.empty(T, device="cuda") if codes else None
        return s

    N, R, L = case["rows"], case["rank"], case["adapters"]
    s["x"] = _acts(T, K, dt, g, case["pad"])
    x32 = s["x"].float()  # the codes that the layer's quantiser has made of x
    s["s"] = x32.abs().amax(1) * torch.tensor(1 / 127, device="cuda")
    s["q"] = torch.round(x32 / s["s"][:, None]).clamp_(-127, 127).to(torch.int8)
    del x32
    s["w"] = _codes((N, K), g)
    s["ws"] = 0.02 / 32 * (0.5 + torch.rand(N, generator=g, device="cuda"))
    s["bias"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
    s["a"] = (torch.randn(L, R, K, generator=g, device="cuda") / math.sqrt(K)).to(dt)
    s["b"] = (torch.randn(L, N, R, generator=g, device="cuda") / math.sqrt(R)).to(dt)
    s["scale"] = 0.25 + torch.rand(L, generator=g, device="cuda")
    # the batch's table of tokens by adapter, which one dispatch makes for all projections
    s["ids"] = _adapter_ids(case, g)
    key = torch.where(s["ids"] < 0, L, s["ids"]).long()
    s["perm"] = torch.argsort(key, stable=True).to(torch.int32)
    counts = torch.bincount(key, minlength=L + 1)[:L]
    s["offs"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["spans"] = [0] + counts.cumsum(0).tolist()
    s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
    if own:
        s["lora"] = C.Lora(s["a"], s["b"], s["scale"])
        s["ws_lora"] = C.lora_workspace(T, R)
    return s


# ---------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    C = s["C"]
    if s["case"]["op"] == "norm":
        C.coli_rmsnorm_quant_token(s["x"], s["gain"], EPS, q=s["q"], s=s["s"], y=s["y"],
                                   res=s["res"], h=s["h"])
        out = [t for t in (s["h"], s["y"], s["s"]) if t is not None]
        return out if s["q"] is None else out + [s["q"] * s["s"][:, None]]
    C.coli_gemm_q8_lora(s["q"], s["s"], s["w"], s["ws"], s["lora"], s["x"], s["ids"], s["offs"],
                        s["perm"], s["y"], s["ws_lora"], bias=s["bias"])
    return s["y"]


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _norm_plain(s):
    dt = TYPES[s["case"]["dtype"]]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    h64 = h.double()  # codes next to a border: in 64 bits
    y = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + EPS)
    if s["gain"] is not None:
        y = y * s["gain"]
    y = y.float()
    out = [] if s["res"] is None else [h.to(dt)]
    if s["y"] is not None:
        out.append(y.to(dt))
    if s["q"] is None:
        return out
    scale = y.abs().amax(1) / 127
    q = torch.round(y / scale[:, None]).clamp(-127, 127)
    q = torch.where(scale[:, None] > 0, q, 0.0)
    return out + [scale, q * scale[:, None]]


def _adapters_plain(s):
    """scale_a * B_a (A_a x) of every token's adapter a; [T, N] in float32."""
    c = s["case"]
    x, ids = s["x"].float(), s["ids"]
    if c["tokens"] * c["rank"] * (c["cols"] + c["rows"]) <= 1 << 28:  # few tokens: their own copies
        at = ids.clamp(min=0).long()
        u = torch.bmm(s["a"][at].float(), x[:, :, None])
        d = torch.bmm(s["b"][at].float(), u)[:, :, 0] * s["scale"][at][:, None]
        return torch.where(ids[:, None] >= 0, d, 0.0)
    out = torch.zeros(c["tokens"], c["rows"], device=x.device)
    for a, (lo, hi) in enumerate(zip(s["spans"], s["spans"][1:])):
        if hi > lo:
            at = s["perm"][lo:hi].long()
            u = x[at] @ s["a"][a].float().t()
            out[at] = (u @ s["b"][a].float().t()) * s["scale"][a]
    return out


def _run_plain(s):
    if s["case"]["op"] == "norm":
        return _norm_plain(s)
    y = (s["q"].float() @ s["w"].view(torch.int8).float().t()) * s["s"][:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return (y + _adapters_plain(s)).to(TYPES[s["case"]["dtype"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    T, K = case["tokens"], case["cols"]
    if case["op"] == "norm":
        rows = 1 + 2 * case["res"] + (case["out"] != "codes")
        size = T * K * b * rows + 4 * K * case["gain"]
        if case["out"] != "rows":
            size += T * K + 4 * T
        return dict(bytes=size, flops=6 * T * K)
    N, R = case["rows"], case["rank"]
    pairs = T * (1 - case["bare"])
    read = case["used"] * (1 - (1 - 1 / case["used"]) ** pairs)  # adapters that some token has
    size = (T * K + N * K + 4 * N * (2 if case["bias"] else 1) + T * N * b  # the projection
            + pairs * K * b + read * R * (K + N) * b + 8 * T)  # x for the adapters, and they
    return dict(bytes=int(size), flops=int(2 * T * N * K + 2 * pairs * R * (K + N)))


def _exact_norm(s):
    res, gain = s["res"], s["gain"]
    # the sum and the norm are each rounded to 32 bits, and the scale is one product in 32 bits
    h = s["x"].to(torch.float64)
    if res is not None:
        h = (h + res.to(torch.float64)).to(torch.float32).to(torch.float64)
    rms = (h.square().sum(dim=1) / h.shape[1] + EPS).rsqrt()
    y = torch.einsum("tn,t->tn", h, rms)
    if gain is not None:
        y = y * gain.to(torch.float64).unsqueeze(0)
    out = [] if res is None else [h]
    if s["y"] is not None:
        out.append(y)
    if s["q"] is not None:
        y32 = y.to(torch.float32)
        unit = y32.abs().max(dim=1).values * torch.tensor(1.0 / 127.0, dtype=torch.float32)
        quot = (y32.double() / unit.double().unsqueeze(1)).float()
        code = torch.nan_to_num(quot.double().round(), nan=0.0).clamp(-127.0, 127.0)
        out += [unit.double(), code * unit.double().unsqueeze(1)]
    return out


def _exact_lora(s):
    c = s["case"]
    weight = s["w"].view(torch.int8).to(torch.float64) * s["ws"].to(torch.float64).unsqueeze(1)
    y = (s["q"].to(torch.float64) * s["s"].to(torch.float64).unsqueeze(1)) @ weight.T.contiguous()
    if s["bias"] is not None:
        y += s["bias"].to(torch.float64)
    for a in range(c["adapters"]):
        mine = (s["ids"] == a).nonzero().reshape(-1)
        if mine.numel():
            low = s["x"][mine].to(torch.float64) @ s["a"][a].to(torch.float64).T.contiguous()
            add = low @ s["b"][a].to(torch.float64).T.contiguous()
            y.index_add_(0, mine, add * s["scale"][a].to(torch.float64))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_lora(s)
