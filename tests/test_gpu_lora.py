"""The 8-bit product with low-rank adapters (coli_gemm_q8_lora) against the
definition in 64 bits, through the C ABI, alone and behind the norm.

Tolerances.  The projection's part is test_gpu_q8's: exact sums, three roundings
of binary32, one for the bias.  u = a x is a binary32 sum of K products (exact
ones of 16-bit operands): on any path at most K / 4 roundings of four products
each (K of one each in fp32), and 48 to join waves and parts of K, relative to
sum |a x|.  The adapters' sum takes u in pieces that hold it to 2^-18 (2^-25 in
fp32, of two operands each), counted as 2^-17 (2^-24), and rounds at most once
for each of 6 R products and joins.  What is added is rounded once with the rest to
binary32 and once to y's type.  That last rounding comes on top of what its operand
is off: half a step relative to it, and below fp16's smallest normal value, 2^-14,
where steps are 2^-24 whatever the value, 2^-25.
"""
import numpy as np
import pytest
import torch

from quantized_moe_coli_amd import binding as B
from test_gpu_q8 import DT, acts, codes, gen, half_step, scales

pytestmark = pytest.mark.gpu


def tables(ids, L):
    """coli_moe_dispatch's tables of the tokens by adapter."""
    T = ids.numel()
    t = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offs, perm, uniq, n = t(L), t(L + 1), t(T), t(L), t(1)
    B.coli_moe_dispatch(ids.view(T, 1), L, counts, offs, perm, uniq, n)
    return offs, perm


def some_ids(T, L, used, order, bare, seed=0):
    g = gen(T, L, seed)
    mine = torch.randperm(L, generator=g)[:used]
    pick = torch.randint(0, used, (T,), generator=g)
    if order == "requests":
        pick = pick.sort().values
    ids = mine[pick]
    return ids.masked_fill(torch.rand(T, generator=g) < bare, -1).to(torch.int32).cuda()


def last_rounding(dt, size):
    step = half_step(dt) * size
    return step.clamp(min=2.0 ** -25) if dt is torch.float16 else step


class Case:
    def __init__(self, dt, T, N, K, R, L, used=None, order="mixed", bare=0.0, pad=0, bias=False, scale=True,
                 seed=0):
        self.dt, self.T, self.N, self.K, self.R, self.L = DT[dt], T, N, K, R, L
        d = self.dt
        self.x = acts(T, K, d, seed + 1, pad, pad // 2)
        self.q, self.s = codes(T, K, seed=seed), scales(T)
        self.w, self.ws = codes(N, K, seed=seed + 3), scales(N)
        self.bias = torch.randn(N, generator=gen(N, seed)).cuda() if bias else None
        self.a = (torch.randn(L, R, K, generator=gen(L, R, K, seed)) / K ** 0.5).to(d).cuda()
        self.b = torch.randn(L, N, R, generator=gen(L, N, R, seed)).to(d).cuda()
        self.scale = (torch.rand(L, generator=gen(L, seed)) + 0.25).cuda() if scale else None
        self.ids = some_ids(T, L, used or L, order, bare, seed)
        self.work = B.lora_workspace(T, R)
        self.work.fill_(0xFF)  # NaN, whatever is read of it
        self.out = torch.full((T, N + 16), 55.0, dtype=d, device="cuda")
        self.y = self.out[:, :N]

    def run(self, y=None, stream=None, work=None):
        self.lora = B.Lora(self.a, self.b, self.scale)
        self.offs, self.perm = tables(self.ids, self.L)
        y = self.y if y is None else y
        B.coli_gemm_q8_lora(self.q, self.s, self.w.view(torch.uint8), self.ws, self.lora, self.x, self.ids,
                            self.offs, self.perm, y, self.work if work is None else work, bias=self.bias,
                            stream=stream)
        return y

    def reference(self):
        """The result and its tolerance before the last rounding, in float64."""
        acc = self.q.double() @ self.w.double().t().contiguous()
        y = acc * self.s.double()[:, None] * self.ws.double()
        tol = 4 * 2.0 ** -24 * y.abs()
        if self.bias is not None:
            y = y + self.bias.double()
            tol += 2.0 ** -24 * self.bias.double().abs()
        f32 = self.dt is torch.float32
        deep = (self.K if f32 else self.K / 4) + 48
        for e in range(self.L):
            m = (self.ids == e).nonzero()[:, 0]
            if m.numel() == 0:
                continue
            x, a, b = self.x[m].double(), self.a[e].double(), self.b[e].double()
            c = 1.0 if self.scale is None else float(self.scale[e])
            at, bt = a.t().contiguous(), b.t().contiguous()
            u, du = x @ at, deep * 2.0 ** -24 * (x.abs() @ at.abs())
            y[m] += c * (u @ bt)
            size = c * (u.abs() @ bt.abs())
            tol[m] += c * (du @ bt.abs()) + (6 * self.R * 2.0 ** -24 + (2.0 ** -24 if f32 else 2.0 ** -17)) * size
        return y, tol + 2.0 ** -24 * y.abs()

    def check(self, y, rows=None):
        ref, tol = self.reference()
        tol = tol + last_rounding(self.dt, ref.abs() + tol)
        bad = (y.double() - ref).abs() > tol
        bad |= torch.isnan(y)
        if rows is not None:
            bad = bad[rows]
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                               float(((y.double() - ref).abs() / tol).max()))
        assert (self.out[:, self.N:] == 55.0).all()


# sizes that each of the product's kernels takes, with few adapters and many
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,N,K,R,L,used,order,bare,pad", [
    (1, 33, 32, 8, 1, 1, "mixed", 0.0, 0), (1, 2048, 6144, 16, 4, 1, "mixed", 0.0, 0),
    (2, 100, 64, 128, 3, 2, "mixed", 0.0, 0), (5, 6145, 160, 16, 7, 5, "mixed", 0.2, 0),
    (16, 100, 2048, 24, 40, 16, "mixed", 0.0, 8), (17, 515, 1056, 40, 3, 3, "requests", 0.3, 0),
    (20, 9000, 96, 8, 20, 20, "mixed", 0.1, 0), (40, 6145, 288, 64, 64, 30, "mixed", 0.0, 3),
    (61, 1001, 1504, 56, 61, 61, "mixed", 0.1, 0), (64, 66000, 64, 16, 9, 9, "mixed", 0.1, 0),
    (65, 333, 512, 72, 2, 2, "mixed", 0.5, 0), (130, 1029, 96, 16, 300, 100, "mixed", 0.1, 0),
    (200, 4096, 64, 8, 1, 1, "mixed", 0.3, 0), (200, 6145, 128, 32, 5, 5, "requests", 0.0, 7),
    (509, 6145, 96, 16, 9, 7, "requests", 0.0, 0), (700, 6145, 64, 48, 20, 20, "mixed", 0.1, 0),
    (700, 1000, 800, 128, 3, 3, "requests", 0.1, 1), (1100, 4097, 64, 16, 1024, 500, "mixed", 0.1, 0),
    (1500, 6144, 64, 24, 4, 3, "requests", 0.1, 8), (2047, 6144, 32, 8, 48, 48, "mixed", 0.1, 0),
    (2100, 517, 128, 64, 6, 6, "requests", 0.0, 0), (9001, 130, 64, 16, 3, 3, "mixed", 0.1, 0)])
def test_lora(dt, T, N, K, R, L, used, order, bare, pad):
    c = Case(dt, T, N, K, R, L, used, order, bare, pad, bias=N % 2 == 0, scale=N % 3 != 0)
    c.check(c.run())


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,N,K", [(1, 64, 64), (40, 1024, 160), (300, 4000, 64), (600, 6145, 64), (1500, 6144, 64)])
@pytest.mark.parametrize("ids", ["some", "none"])
def test_tokens_without_an_adapter_are_the_plain_products(dt, T, N, K, ids):
    """Ids below zero and past the last adapter; their rows equal coli_gemm_q8's."""
    c = Case(dt, T, N, K, 16, 5, bare=0.5, bias=True)
    out = torch.tensor([-1, -7, 5, 6, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    other = out[torch.arange(T, device="cuda") % 6]
    c.ids = torch.where(c.ids < 0, other, c.ids) if ids == "some" else other
    y = c.run()
    plain = torch.empty(T, N, dtype=c.dt, device="cuda")
    B.coli_gemm_q8(c.q, c.s, c.w.view(torch.uint8), c.ws, plain, bias=c.bias)
    bare = (c.ids < 0) | (c.ids >= 5)
    assert bare.any() and torch.equal(y[bare], plain[bare])
    c.check(y)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,N,K,R", [(3, 64, 64, 8), (61, 1024, 160, 16), (64, 66000, 32, 16), (600, 6145, 64, 40),
                                     (1500, 6144, 64, 16)])
def test_broken_adapters_and_rows_stay_with_their_tokens(dt, T, N, K, R):
    """NaN and infinities in adapters that others of the same tile use, in slots
    that nobody uses, and in one token's activations."""
    c = Case(dt, T, N, K, R, 6, used=4, bare=0.2)
    used = [int(v) for v in c.ids.unique() if v >= 0]
    spare = [v for v in range(6) if v not in used]
    c.a[spare], c.b[spare] = float("nan"), float("inf")
    broken = used[0]
    c.a[broken, 0] = float("inf")
    c.b[broken, ::2] = float("nan")
    if len(used) > 1:
        c.b[used[1], 3] = float("inf")
    lost = T // 2
    c.x[lost, K // 2] = float("nan")
    y = c.run()
    bad = (c.ids == broken) | (torch.arange(T, device="cuda") == lost) & (c.ids >= 0)
    assert torch.isnan(y[c.ids == broken][:, ::2]).all()
    if (bad & (c.ids != broken)).any():
        assert torch.isnan(y[lost]).all()
    part = ~bad
    if len(used) > 1:
        mine = c.ids == used[1]
        assert not torch.isfinite(y[mine & part][:, 3]).any()
        y[mine, 3] = 0
    keep = torch.ones_like(y, dtype=torch.bool)
    if len(used) > 1:
        keep[mine, 3] = False
    for t in (c.a, c.b, c.x):
        t.masked_fill_(~torch.isfinite(t), 0)
    ref, tol = c.reference()
    tol = tol + last_rounding(c.dt, ref.abs() + tol)
    ok = ((y.double() - ref).abs() <= tol) | ~keep
    assert ok[part].all()


@pytest.mark.parametrize("dt,T,N,K,R", [("bf16", 7, 300, 160, 16), ("f16", 300, 4000, 96, 24),
                                        ("f32", 1500, 6144, 64, 8), ("bf16", 1500, 6144, 64, 64)])
def test_same_bits_again_and_the_workspace_keeps_nothing(dt, T, N, K, R):
    c = Case(dt, T, N, K, R, 8, bare=0.1)
    first = c.run().clone()
    c.work.fill_(0xFF)
    assert torch.equal(c.run(), first)
    wide = torch.full((c.work.numel() * 2,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(work=wide), first)
    assert (wide[c.work.numel():] == 0xFF).all()
    with pytest.raises(B.ColiError, match="orkspace"):
        c.run(work=c.work[:-256])


def test_large_ranges_of_16_bit_operands():
    """fp16 activations and adapters whose products pass fp16's range, and tiny
    ones below its normal values."""
    for T, N in ((3, 200), (300, 4000), (1500, 6144)):
        for big, small in ((200.0, 2.0 ** -9), (2.0 ** -13, 30.0)):
            c = Case("f16", T, N, 64, 16, 4, bare=0.1)
            c.x.mul_(big)
            c.a.mul_(big)
            c.b.mul_(small / 16)
            c.check(c.run())


def test_adapters_past_32_bit_offsets():
    L, R, K, N, T = 1024, 128, 32768, 32768, 5
    a = torch.empty(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(L, N, R, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    ids = torch.tensor([1023, 3, 1000, -1, 1023], dtype=torch.int32, device="cuda")
    for e in (3, 1000, 1023):
        a[e] = torch.randn(R, K, generator=g, device="cuda") / K ** 0.5
        b[e] = torch.randn(N, R, generator=g, device="cuda")
    c = Case("bf16", T, 8, 32, 8, 1)
    c.N, c.K, c.R, c.L, c.a, c.b, c.ids, c.scale = N, K, R, L, a, b, ids, None
    c.x, c.q = acts(T, K, torch.bfloat16), codes(T, K)
    c.w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    c.ws, c.work = scales(N), B.lora_workspace(T, R)
    c.out = torch.full((T, N + 16), 55.0, dtype=torch.bfloat16, device="cuda")
    c.y = c.out[:, :N]
    y = c.run()
    for t in range(T):  # (a row at a time: the weights in 64 bits are 8.6 GB)
        one = c.q[t].double() @ c.w.double().t()
        ref = one * float(c.s[t]) * c.ws.double()
        tol = 4 * 2.0 ** -24 * ref.abs()
        e = int(ids[t])
        if e >= 0:
            x, a64, b64 = c.x[t].double(), a[e].double(), b[e].double()
            u = a64 @ x
            ref += b64 @ u
            tol += b64.abs() @ ((K / 4 + 48) * 2.0 ** -24 * (a64.abs() @ x.abs()))
            tol += (6 * R * 2.0 ** -24 + 2.0 ** -17) * (b64.abs() @ u.abs())
        tol = tol + (half_step(torch.bfloat16) + 2.0 ** -24) * (ref.abs() + tol)
        assert ((y[t].double() - ref).abs() <= tol).all(), t


def test_empty_batch():
    c = Case("bf16", 1, 64, 64, 16, 2)
    z = lambda *s, d=torch.int32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    B.coli_gemm_q8_lora(z(0, 64, d=torch.int8), z(0, d=torch.float32), c.w.view(torch.uint8), c.ws,
                        B.Lora(c.a, c.b), z(0, 64, d=c.dt), z(0), torch.zeros(3, dtype=torch.int32, device="cuda"),
                        z(0), z(0, 64, d=c.dt), c.work)


def test_binding_refuses():
    c = Case("bf16", 4, 64, 64, 16, 2)
    c.run()
    call = lambda **k: B.coli_gemm_q8_lora(*[k.get(n, v) for n, v in dict(  # noqa: E731
        q=c.q, s=c.s, w=c.w.view(torch.uint8), ws=c.ws, lora=c.lora, x=c.x, ids=c.ids, offs=c.offs, perm=c.perm,
        y=c.y, workspace=c.work).items()])
    call()
    with pytest.raises(ValueError, match="adapters must be of 64 columns"):
        call(lora=B.Lora(c.a.float(), c.b.float()))
    with pytest.raises(ValueError, match="adapters must be of 64 columns"):
        call(lora=B.Lora(c.a[:, :, :32].contiguous(), c.b))
    with pytest.raises(ValueError, match="x must be"):
        call(x=c.x.float())
    with pytest.raises(ValueError, match="w must hold"):
        call(w=c.w[:32].view(torch.uint8))
    with pytest.raises(ValueError, match="ids must be torch.int32"):
        call(ids=c.ids.long())
    with pytest.raises(ValueError, match="offs must hold 3"):
        call(offs=c.offs[:2])
    with pytest.raises(ValueError, match="workspace must be a device tensor"):
        call(workspace=c.work.cpu())
    with pytest.raises(ValueError, match="b must be"):
        B.Lora(c.a, c.b[:1])
    with pytest.raises(ValueError, match="b must be contiguous"):
        B.Lora(c.a, torch.empty(2, 16, 64, dtype=c.dt, device="cuda").transpose(1, 2))


# --- as a model's layers use them --------------------------------------------------------------
class FFN:
    """A dense feed-forward block in 8 bits with adapters on both projections:
    norm, gate and up, SwiGLU, down, and the next block's norm."""

    def __init__(self, T, H, I, R, L, dt):
        g = gen(T, H, I, R)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.I, self.dt = T, H, I, dt
        self.w1, self.s1 = codes(2 * I, H, seed=1), scales(2 * I)
        self.w2, self.s2 = codes(H, I, seed=2), scales(H)
        self.l1 = B.Lora((r(L, R, H) / H ** 0.5).to(dt).cuda(), (0.3 * r(L, 2 * I, R)).to(dt).cuda(),
                         (torch.rand(L, generator=g) + 0.5).cuda())
        self.l2 = B.Lora((r(L, R, I) / I ** 0.5).to(dt).cuda(), (0.3 * r(L, H, R)).to(dt).cuda())
        self.gain = (1 + 0.1 * r(H)).cuda()
        e = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        self.h, self.y, self.gu, self.hid, self.d = e(T, H), e(T, H), e(T, 2 * I), e(T, I), e(T, H)
        self.h2, self.y2 = e(T, H), e(T, H)
        self.q, self.s = e(T, H, d=torch.int8), e(T, d=torch.float32)
        self.hq, self.hs = e(T, I, d=torch.int8), e(T, d=torch.float32)
        self.q2, self.sc2 = e(T, H, d=torch.int8), e(T, d=torch.float32)
        self.work = B.lora_workspace(T, R)

    def run(self, x, res, ids, offs, perm):
        I = self.I
        B.coli_rmsnorm_quant_token(x, self.gain, 1e-6, q=self.q, s=self.s, y=self.y, res=res, h=self.h)
        B.coli_gemm_q8_lora(self.q, self.s, self.w1.view(torch.uint8), self.s1, self.l1, self.y, ids, offs, perm,
                            self.gu, self.work)
        gate, up = self.gu[:, :I], self.gu[:, I:]
        B.coli_swiglu_quant_token(gate, up, self.hq, self.hs)
        # the down projection's adapters read the codes' values
        self.hid.copy_(self.hq * self.hs[:, None])
        B.coli_gemm_q8_lora(self.hq, self.hs, self.w2.view(torch.uint8), self.s2, self.l2, self.hid, ids, offs,
                            perm, self.d, self.work)
        B.coli_rmsnorm_quant_token(self.d, self.gain, 1e-6, q=self.q2, s=self.sc2, y=self.y2, res=self.h, h=self.h2)
        return [t.clone() for t in (self.h, self.y, self.q, self.gu, self.hq, self.d, self.h2, self.y2, self.q2,
                                    self.sc2)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", [(1, 1024, 768), (19, 512, 1056), (300, 2048, 1536)])
def test_norm_projection_and_adapters_together(dt, T, H, I):
    """The chain's result against the same chain in 64 bits from the codes that it
    made: the norm's rows and codes are its own test's, so each product is
    checked on the operands it had, and the last norm on the chain's end."""
    R, L = 16, 5
    f = FFN(T, H, I, R, L, DT[dt])
    ids = some_ids(T, L, L, "mixed", 0.2)
    offs, perm = tables(ids, L)
    x, res = acts(T, H, DT[dt], 5), acts(T, H, DT[dt], 6)
    got = f.run(x, res, ids, offs, perm)
    for q, s, w, ws, lora, xin, out in ((f.q, f.s, f.w1, f.s1, f.l1, f.y, f.gu),
                                        (f.hq, f.hs, f.w2, f.s2, f.l2, f.hid, f.d)):
        c = Case.__new__(Case)
        c.dt, c.q, c.s, c.w, c.ws, c.bias, c.x, c.ids = DT[dt], q, s, w, ws, None, xin, ids
        c.a, c.b, c.scale, c.L, c.R, c.K, c.N = lora.a, lora.b, lora.scale, L, R, q.shape[1], w.shape[0]
        c.out = torch.full((1, c.N + 16), 55.0, device="cuda")
        c.check(out)
    h = f.h.double() + f.d.double()
    ref = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * f.gain.double()
    assert ((f.y2.double() - ref).abs() <= (half_step(DT[dt]) + 2.0 ** -21) * ref.abs() + 1e-30).all()

    # captured and replayed, with other tokens of other adapters each time
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            outs = f.run(x, res, ids, offs, perm)
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(acts(T, H, DT[dt], 20 + i))
        ids.copy_(some_ids(T, L, L, "mixed", 0.3, seed=i))
        o, p = tables(ids, L)
        offs.copy_(o)
        perm.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        replay = [t.clone() for t in outs]
        for r, e in zip(replay, f.run(x, res, ids, offs, perm)):
            assert torch.equal(r, e), i
    assert len(got) == len(outs)


def test_two_streams_with_a_workspace_each():
    a, b = Case("bf16", 61, 1024, 2048, 16, 9, seed=1), Case("bf16", 700, 1000, 512, 32, 4, seed=2)
    want = a.run().clone(), b.run().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st in ((a, s1), (b, s2)):
            with torch.cuda.stream(st):
                B.coli_gemm_q8_lora(c.q, c.s, c.w.view(torch.uint8), c.ws, c.lora, c.x, c.ids, c.offs, c.perm, c.y,
                                    c.work, bias=c.bias)
    torch.cuda.synchronize()
    assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])
    st = torch.cuda.Stream()
    a.y.fill_(0)
    torch.cuda.synchronize()
    B.coli_gemm_q8_lora(a.q, a.s, a.w.view(torch.uint8), a.ws, a.lora, a.x, a.ids, a.offs, a.perm, a.y, a.work,
                        stream=st)
    st.synchronize()
    assert torch.equal(a.y, want[0])
