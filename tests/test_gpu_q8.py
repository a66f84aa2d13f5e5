"""The 8-bit products with token and channel scales, the experts' form, the
token quantisers and the combine, against 64-bit forms, through the C ABI.

Tolerances.  Codes are compared exactly: every rounding of their definition is
fixed (the scale and the quotient in binary32; SwiGLU's result once from
binary64).  A product y = fl(fl(fl(acc) * fl(st * ws)) + b) has an exact acc,
so its relative error before the last rounding is at most three half-steps of
binary32 (the conversion, the scales' product, the product; 2^-24 each), plus
one for the bias's addition relative to |y| + |b|; the last rounding adds half a
step of y's type.  For fp16 results below the smallest normal value half a
step is absolute (2^-25).
"""
import numpy as np
import pytest
import torch

import q8_ref as R
from quantized_moe_coli_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def gen(*seed):
    return torch.Generator().manual_seed(hash(seed) & 0x7FFFFFFF)


def acts(T, n, dt, seed=0, pad=0, shift=0):
    """[T, n] rows of a wider buffer (pad more columns, starting at shift)."""
    x = torch.randn(T, n + pad, generator=gen(T, n, seed)).to(dt).cuda()
    return x[:, shift:shift + n]


def codes(*shape, seed=0):
    return torch.randint(-127, 128, shape, generator=gen(*shape, seed), dtype=torch.int8).cuda()


def scales(*shape, seed=0):
    return (torch.rand(*shape, generator=gen(*shape, seed, 7)) * 1e-3 + 1e-4).cuda()


def assert_product(y, ref, dt, bias=0.0):
    got = f64(y)
    err = np.abs(got - ref)
    tol = 3 * 2.0 ** -24 * (np.abs(ref) + np.abs(bias)) + 2.0 ** -24 * (np.abs(ref) + 2 * np.abs(bias))
    tol = tol + half_step(dt) * (np.abs(ref) + tol)
    if dt is torch.float16:
        tol = np.maximum(tol, 2.0 ** -25 + 2.0 ** -22 * np.abs(ref))
    bad = err > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((err / tol).max()))


# --- quantisers --------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,n,pad,shift", [
    (1, 32, 0, 0), (5, 64, 0, 0), (3, 2048, 0, 0), (7, 2080, 32, 0), (2, 6144, 0, 0),
    (3, 8192, 8, 0), (2, 8224, 0, 0), (2, 32768, 0, 0), (1, 33024, 0, 0), (2, 131040, 0, 0),
    (4, 96, 5, 3), (2, 6176, 1, 1), (1021, 160, 0, 0)])
def test_quant_act_token(dt, T, n, pad, shift):
    x = acts(T, n, DT[dt], 1, pad, shift)
    q = torch.full((T, n), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(T, device="cuda")
    B.coli_quant_act_token(x, q, s)
    rq, rs = R.quant(f64(x))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_quant_codes_next_to_borders():
    """Every quotient within a few units of the last place of a half."""
    s = np.float32(0.0123)
    k = np.arange(-126, 126, dtype=np.float32) + np.float32(0.5)
    base = (k * s).astype(np.float32)
    rows = [base]
    up = dn = base
    for _ in range(3):
        up = np.nextafter(up, np.float32(np.inf))
        dn = np.nextafter(dn, np.float32(-np.inf))
        rows += [up, dn]
    x = np.zeros((len(rows), 256), dtype=np.float32)
    for i, r in enumerate(rows):
        x[i, :252] = r
        x[i, 252] = np.float32(127) * s
    xt = torch.from_numpy(x).cuda()
    q, sc = torch.empty(len(rows), 256, dtype=torch.int8, device="cuda"), torch.empty(len(rows), device="cuda")
    B.coli_quant_act_token(xt, q, sc)
    rq, rs = R.quant(x)
    np.testing.assert_array_equal(sc.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_quant_extremes():
    """Zero rows, subnormal rows (a scale that is subnormal or rounds to zero),
    the largest values, and rows with an infinity or a NaN."""
    x = torch.zeros(9, 64)
    x[1, 3] = 1e-45
    x[2] = torch.linspace(-1e-43, 1e-43, 64)
    x[3] = torch.linspace(-3e-38, 3e-38, 64)
    x[4] = torch.linspace(-3.4e38, 3.4e38, 64)
    x[5] = torch.randn(64, generator=gen(5))
    x[5, 63] = float("inf")
    x[6, 0] = float("nan")
    x[7] = torch.linspace(-1e-30, 1e-30, 64)
    x[8] = -0.0
    xd = x.cuda()
    q, s = torch.full((9, 64), 5, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    B.coli_quant_act_token(xd, q, s)
    rq, rs = R.quant(x.numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,n,wide", [(1, 32, True), (3, 2048, True), (5, 2048, False), (2, 8224, True),
                                      (257, 96, False), (2, 33056, False)])
def test_swiglu_quant_token(dt, T, n, wide):
    """h is rounded once from binary64, so a code can differ from the 64-bit
    form's only where that rounding itself is undecided in binary64."""
    gu = (torch.randn(T, 2 * n, generator=gen(T, n, 3)) * 2).to(DT[dt]).cuda()
    g, u = (gu[:, :n], gu[:, n:]) if wide else (gu[:, :n].contiguous(), gu[:, n:].contiguous())
    q, s = torch.empty(T, n, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    B.coli_swiglu_quant_token(g, u, q, s)
    rq, rs = R.quant(R.swiglu(f64(g), f64(u)))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_swiglu_far_values():
    """Gates so negative that the exponential overflows, so large that silu is
    the gate, zeros, and infinities (which poison the row)."""
    g = torch.tensor([[-1e4, -800.0, -709.0, -100.0, -50.0, 0.0, 50.0, 1e4] * 4,
                      [float("-inf")] + [1.0] * 31, [float("inf")] + [1.0] * 31])
    u = torch.randn(3, 32, generator=gen(11))
    q, s = torch.empty(3, 32, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    B.coli_swiglu_quant_token(g.cuda(), u.cuda(), q, s)
    rq, rs = R.quant(R.swiglu(g.numpy(), u.numpy()))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


def test_quant_more_rows_than_one_grid_axis():
    """Over 2^22 rows of 32: workgroups along both axes.  Every row's codes
    against the definition in torch, each quotient rounded once from float64."""
    T, n = (1 << 22) + 5, 32
    x = torch.randn(T, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    q, s = torch.empty(T, n, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    B.coli_swiglu_quant_token(torch.full_like(x, 1e4), x, q, s)  # silu(1e4) = 1e4
    h = (x.double() * 1e4).float()
    rs = h.abs().amax(1) * float(np.float32(1) / np.float32(127))
    assert torch.equal(s, rs)
    assert torch.equal(q, torch.round((h.double() / rs[:, None].double()).float()).to(torch.int8))


def test_calls_on_a_given_stream():
    """Every call enqueues on the stream it is given, not on the current one."""
    st = torch.cuda.Stream()
    T, k, E, H = 4, 2, 4, 64
    x, q, s = acts(T, H, torch.bfloat16, 1), torch.zeros(T, H, dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
    w, ws, y = codes(40, H, seed=3), scales(40), torch.zeros(T, 40, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)  # what follows on this stream waits
    B.coli_quant_act_token(x, q, s, stream=st)
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y, stream=st)
    idx, wt = torch.full((T, k), -5, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    lg = torch.randn(T, E, generator=gen(3)).cuda()
    early = y.clone()  # on the current stream, which does not wait
    B.coli_moe_route_scored(B.score_cfg(E, k), lg, None, idx, wt, stream=st.cuda_stream)
    st.synchronize()
    assert (early == 0).all()
    rq, rs = R.quant(f64(x))
    assert_product(y, R.product(rq, rs, w.cpu().numpy(), ws.cpu().numpy()), torch.float32)
    assert (idx >= 0).all()


# --- dense product -----------------------------------------------------------------------------
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 32), (1, 17, 96), (2, 16, 128), (5, 100, 160), (12, 33, 1024), (13, 64, 6144),
    (16, 31, 2080), (28, 48, 224), (29, 70, 352), (64, 96, 544), (65, 130, 160), (127, 257, 96),
    (128, 128, 128), (129, 127, 2048), (300, 200, 32), (515, 259, 288), (1024, 256, 64),
    (1500, 515, 416), (1, 2048, 6144), (3, 300, 8192), (1, 5, 131040), (70, 40, 16416),
    # sizes from which other variants are taken: blocks of 32 and 64 channels,
    # the sweep (whole and part chunks, few and many), 64 x 64, the tiles
    (3, 4100, 288), (16, 4097, 2592), (20, 8200, 96), (31, 8193, 1568), (61, 8200, 544),
    (61, 65601, 32), (33, 65536, 896), (64, 65550, 1120), (200, 6145, 800), (512, 6144, 160),
    (509, 6147, 544), (1024, 6145, 96), (1021, 6144, 416), (2048, 6150, 160), (2047, 6144, 608),
    (2048, 6144, 32), (2100, 6145, 1056)])
@pytest.mark.parametrize("dt,bias", [("f32", False), ("bf16", True), ("f16", False)])
def test_gemm_q8(T, N, K, dt, bias):
    q, w = codes(T, K, seed=1), codes(N, K, seed=2)
    s, ws = scales(T), scales(N, seed=3)
    b = torch.randn(N, generator=gen(N)).cuda() if bias else None
    wide = torch.full((T, N + 3), 77.0, dtype=DT[dt], device="cuda")
    y = wide[:, :N]
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y, bias=b)
    bn = b.cpu().numpy() if bias else None
    ref = R.product(q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy(), bn)
    assert_product(y, ref, DT[dt], 0.0 if bn is None else bn[None, :])
    assert (f64(wide[:, N:]) == 77.0).all()


def test_gemm_q8_largest_sums():
    """All codes at -128: the largest sum an int32 accumulator has to hold."""
    K = 131040
    q = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((70, K), -128, dtype=torch.int8, device="cuda")
    y = torch.empty(3, 70, device="cuda")
    B.coli_gemm_q8(q, torch.ones(3, device="cuda"), w.view(torch.uint8), torch.ones(70, device="cuda"), y)
    assert (f64(y) == float(np.float32(128 * 128 * K))).all()
    q = q[:1].expand(70, K).contiguous()
    y = torch.empty(70, 70, device="cuda")
    B.coli_gemm_q8(q, torch.ones(70, device="cuda"), w.view(torch.uint8), torch.ones(70, device="cuda"), y)
    assert (f64(y) == float(np.float32(128 * 128 * K))).all()


@pytest.mark.parametrize("T,N", [(3, 40), (70, 40), (512, 6144)])
def test_gemm_q8_small_scales(T, N):
    """Scales whose product is subnormal where the result is not."""
    K = 96
    q, w = codes(T, K, seed=1), codes(N, K, seed=2)
    s, ws = scales(T) * 1e-34, scales(N, seed=3) * 1e-3
    y = torch.empty(T, N, device="cuda")
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y)
    ref = R.product(q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())
    ok = np.abs(f64(y) - ref) <= 3 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -149  # and one subnormal step
    assert ok.all()


def test_gemm_q8_nan_scale_stays_in_its_row():
    q, w = codes(40, 256, seed=1), codes(50, 256, seed=2)
    s, ws = scales(40), scales(50)
    s[7] = float("nan")
    y = torch.empty(40, 50, dtype=torch.bfloat16, device="cuda")
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y)
    nan = torch.isnan(y).cpu()
    assert nan[7].all() and nan.sum() == 50


def test_gemm_q8_rows_past_32_bit_offsets():
    """An output whose last rows lie more than 2^32 elements from its start."""
    T, N, K, ld = 130, 40, 64, 34_000_000
    need = T * ld * 2 + (1 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs %d bytes of device memory" % need)
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    y = buf.as_strided((T, N), (ld, 1))
    q, w, s, ws = codes(T, K, seed=1), codes(N, K, seed=2), scales(T), scales(N)
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y)
    ref = R.product(q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())
    assert_product(y, ref, torch.bfloat16)


# --- experts' products -------------------------------------------------------------------------
def routing(T, k, E, seed, drop=0.0, few=None):
    g = gen(T, k, E, seed)
    idx = torch.stack([torch.randperm(few or E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if drop:
        idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx


@pytest.mark.parametrize("T,k,E,N,K,drop,few", [
    (1, 1, 1, 5, 32, 0, None), (1, 8, 256, 48, 96, 0, None), (3, 8, 256, 33, 544, 0.3, None),
    (40, 2, 5, 70, 160, 0.5, None), (7, 3, 100, 16, 128, 0, 3), (200, 4, 9, 40, 224, 0.2, None),
    (600, 2, 8, 140, 96, 0.1, None), (300, 2, 2, 130, 64, 0, None), (1500, 2, 3, 260, 160, 0.2, None),
    (65, 1, 1024, 20, 64, 0, None), (33, 2, 1000, 30, 32, 0, 2), (5, 2, 7, 30, 64, 1.0, None),
    # the sweeps (up to 32 and 64 tokens a tile; whole and part chunks, few and
    # many), experts with more tokens than a tile, one expert with all of them
    (40, 8, 64, 1100, 96, 0.1, None), (33, 8, 64, 1089, 1216, 0, None), (64, 8, 300, 260, 1184, 0, None),
    (160, 8, 64, 1100, 64, 0.1, None), (161, 8, 64, 1101, 1024, 0.1, None), (330, 8, 64, 1090, 1248, 0, None),
    (300, 4, 40, 1700, 928, 0, 4), (24, 4, 40, 1700, 608, 0, 4), (700, 1, 9, 600, 96, 0, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fan", [True, False])
def test_gemm_q8_grouped(T, k, E, N, K, drop, few, dt, fan):
    idx = routing(T, k, E, 1, drop, few)
    P = T * k
    offs, perm = R.tables(idx.numpy(), E)
    rows = T if fan else P
    q, s = codes(rows, K, seed=1), scales(rows)
    w, ws = codes(E, N, K, seed=2), scales(E, N)
    y = torch.full((P, N), 55.0, dtype=DT[dt], device="cuda")
    d = {n: torch.zeros(m, dtype=torch.int32, device="cuda") for n, m in
         (("counts", E), ("offs", E + 1), ("perm", P), ("uniq", E), ("n", 1))}
    B.coli_moe_dispatch(idx.cuda(), E, d["counts"], d["offs"], d["perm"], d["uniq"], d["n"])
    B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, d["offs"], d["perm"], y, fan=k if fan else 1)
    np.testing.assert_array_equal(d["offs"].cpu().numpy(), offs)
    flat = idx.numpy().ravel()
    qn, sn, wn, wsn = q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy()
    got = f64(y)
    for e in np.unique(flat):
        pairs = np.flatnonzero(flat == e)
        if e < 0:
            assert (got[pairs] == 55.0).all()
            continue
        r = pairs // k if fan else pairs
        assert_product(y[torch.from_numpy(pairs).cuda()], R.product(qn[r], sn[r], wn[e], wsn[e]), DT[dt])


@pytest.mark.parametrize("P,E", [(24, 6), (600, 3)])
def test_gemm_q8_grouped_skips_what_lies_outside(P, E):
    """Tables that name pairs and rows outside the buffers, or whose offsets
    are no running sum: nothing outside is touched, the rest is computed."""
    N, K = 40, 64
    q, s = codes(P, K, seed=1), scales(P)
    w, ws = codes(E, N, K, seed=2), scales(E, N)
    per = P // E
    offs = torch.arange(E + 1, dtype=torch.int32) * per
    perm = torch.arange(P, dtype=torch.int32)
    perm[3], perm[5] = -7, P + 100
    big = torch.full((P + 200, N), 9.0, device="cuda")
    B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, offs.cuda(), perm.cuda(), big[:P])
    got = f64(big)
    ref = np.full((P + 200, N), 9.0)
    for i in range(P):
        if 0 <= perm[i] < P:
            ref[i] = R.product(*(t[i:i + 1].cpu().numpy() for t in (q, s)), w[i // per].cpu().numpy(),
                               ws[i // per].cpu().numpy())[0]
    same = np.abs(got - ref) <= 5 * 2.0 ** -24 * np.abs(ref)
    assert same.all(), np.argwhere(~same)[:5]
    # rows of q past the end
    big.fill_(9.0)
    B.coli_gemm_q8_grouped(q[:P // 2], s[:P // 2], w.view(torch.uint8), ws, offs.cuda(),
                           torch.arange(P, dtype=torch.int32).cuda(), big[:P])
    assert (f64(big)[P // 2:] == 9.0).all() and (f64(big)[:P // 2] != 9.0).any()
    # offsets that are no running sum: no result is promised, only that rows outside stay
    big.fill_(9.0)
    bad = torch.randint(-1000, 1000, (E + 1,), generator=gen(3), dtype=torch.int32)
    B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, bad.cuda(),
                           torch.arange(P, dtype=torch.int32).cuda(), big[:P])
    assert (f64(big)[P:] == 9.0).all()


# --- combine -----------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,k,H,pad,add", [(1, 1, 1, 0, False), (3, 8, 6144, 0, False), (5, 2, 100, 4, True),
                                           (2, 32, 515, 0, True), (700, 3, 64, 0, True), (2, 4, 33, 1, False)])
def test_moe_combine(dt, T, k, H, pad, add):
    o = acts(T * k, H, DT[dt], 4, pad)
    w = torch.randn(T, k, generator=gen(T, k)).cuda()
    idx = torch.randint(-1, 3, (T, k), generator=gen(T, k, 2), dtype=torch.int32)
    on = (idx >= 0).numpy()
    o2 = o.clone() if pad else o
    o2[torch.from_numpy(~on.ravel()).cuda()] = float("nan")  # rows that are not read
    a = acts(T, H, DT[dt], 6) if add else None
    y = torch.empty(T, H, dtype=DT[dt], device="cuda")
    B.coli_moe_combine(o2, idx.cuda(), w, y, add=a)
    terms = f64(o).reshape(T, k, H) * f64(w)[:, :, None]
    terms = np.where(on[:, :, None], terms, 0.0)
    ref = terms.sum(1) + (f64(a) if add else 0.0)
    size = np.abs(terms).sum(1) + (np.abs(f64(a)) if add else 0.0)
    # at most k roundings of partial sums, each no larger than `size`
    tol = k * 2.0 ** -24 * size * 1.01
    tol = tol + half_step(DT[dt]) * (np.abs(ref) + tol) + (2.0 ** -25 if dt == "f16" else 0.0)
    assert (np.abs(f64(y) - ref) <= tol).all()
    if add:  # in place
        B.coli_moe_combine(o2, idx.cuda(), w, a, add=a)
        assert torch.equal(a, y)


def test_moe_combine_without_idx_and_all_dropped():
    o = acts(6, 64, torch.float32, 1)
    w = torch.rand(3, 2, generator=gen(1)).cuda()
    y, z = torch.empty(3, 64, device="cuda"), torch.empty(3, 64, device="cuda")
    B.coli_moe_combine(o, None, w, y)
    B.coli_moe_combine(o, torch.zeros(3, 2, dtype=torch.int32, device="cuda"), w, z)
    assert torch.equal(y, z)
    B.coli_moe_combine(o, torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), w, z)
    assert (z == 0).all()


# --- scored router -----------------------------------------------------------------------------
def check_route(logits, bias, cfg, dt="f32"):
    E, k, G, TG, score, gs, norm, rsf = cfg
    lg = logits.to(DT[dt]).cuda() if not logits.is_cuda else logits
    T = lg.shape[0]
    idx = torch.full((T, k), 12345, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 9.0, device="cuda")
    c = B.score_cfg(E, k, G, TG, score=B.SCORE_SOFTMAX if score == "softmax" else B.SCORE_SIGMOID,
                    group_score=B.GROUP_TOP2 if gs == "top2" else B.GROUP_MAX,
                    norm_topk_prob=int(norm), routed_scaling_factor=rsf)
    B.coli_moe_route_scored(c, lg, bias.cuda() if bias is not None else None, idx, w)
    ri, rw = R.route(f32(lg), None if bias is None else bias.numpy(), k, G, TG, score, gs, norm, rsf)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    # p, its sum over k terms, the quotient and the product by rsf: (k + 3) half-steps
    tol = (k + 3) * 2.0 ** -24 * np.abs(rw) + 2.0 ** -149
    assert (np.abs(f64(w) - rw) <= tol).all()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("score,gs,norm", [("softmax", "max", True), ("softmax", "top2", False),
                                           ("sigmoid", "top2", True), ("sigmoid", "max", False)])
@pytest.mark.parametrize("T,E,k,G,TG", [
    (1, 1, 1, 1, 1), (4, 7, 3, 1, 1), (9, 64, 8, 8, 3), (33, 256, 8, 8, 4), (5, 256, 8, 1, 1),
    (3, 160, 6, 8, 3), (2, 1024, 32, 1, 1), (3, 1023, 17, 33, 5), (2, 1024, 32, 64, 9), (5, 30, 2, 3, 1),
    (3, 34, 2, 17, 4), (2, 512, 16, 5 - 1, 2), (4, 5, 5, 5, 5), (3, 65, 4, 1, 1)])
def test_route_scored(dt, score, gs, norm, T, E, k, G, TG):
    g = gen(T, E, k)
    logits = torch.randn(T, E, generator=g) * 2
    bias = torch.randn(E, generator=g) * 0.02 if E % 2 else None
    check_route(logits, bias, (E, k, G, TG, score, gs, norm, 2.5), dt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gs", ["top2", "max"])
def test_route_scored_ties_masks_and_infinities(score, gs):
    E, k, G, TG = 48, 6, 6, 2
    rows = []
    rows.append(torch.zeros(E))                                   # every score equal
    rows.append(torch.full((E,), torch.finfo(torch.float32).min))  # the type's lowest value is a value
    rows.append(torch.full((E,), -float("inf")))                  # nothing can be chosen
    r = torch.full((E,), -float("inf")); r[[5, 40]] = 1.0; rows.append(r)  # fewer than k
    r = torch.randn(E, generator=gen(1)); r[::2] = float("nan"); rows.append(r)
    r = torch.randn(E, generator=gen(2)); r[[3, 30]] = float("inf"); rows.append(r)
    r = torch.full((E,), -300.0); r[7] = -299.0; rows.append(r)   # sigmoid scores of zero
    r = torch.randint(0, 3, (E,), generator=gen(3)).float(); rows.append(r)  # many ties
    r = torch.randn(E, generator=gen(4)); r[:40] = -float("inf"); rows.append(r)  # one live group
    r = torch.zeros(E); r[1] = 1e-9; r[2] = 2e-9; rows.append(r)  # logits that give equal scores
    r = torch.full((E,), torch.finfo(torch.float32).min); r[9] = 0.0; rows.append(r)
    logits = torch.stack(rows)
    for norm in (True, False):
        check_route(logits, None, (E, k, G, TG, score, gs, norm, 1.0))
        check_route(logits, None, (E, k, 1, 1, score, gs, norm, 1.0))
    bias = torch.zeros(E)
    bias[0], bias[1], bias[2] = float("-inf"), float("nan"), float("inf")
    check_route(torch.randn(4, E, generator=gen(5)), bias, (E, k, G, TG, score, gs, True, 1.0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("score,gs", [("softmax", "max"), ("sigmoid", "top2")])
@pytest.mark.parametrize("T,E,k,G,TG", [(1024, 256, 8, 1, 1), (1029, 256, 8, 8, 4), (1500, 60, 6, 4, 2),
                                        (1025, 16, 9, 16, 9), (1031, 7, 3, 1, 1), (1030, 128, 4, 2, 1),
                                        (1027, 256, 17, 1, 1), (1026, 45, 5, 9, 3), (1033, 512, 8, 8, 3)])
def test_route_scored_batches(dt, score, gs, T, E, k, G, TG):
    """Batches that take the four-tokens-a-wave kernel, and neighbours of its
    limits; with ties, dead experts and rows without any."""
    g = gen(T, E, k)
    logits = (torch.randn(T, E, generator=g) * 2)
    logits[::3] = torch.randint(-3, 4, (len(range(0, T, 3)), E), generator=g).float()
    logits[torch.rand(T, E, generator=g) < 0.1] = float("-inf")
    logits[5] = float("-inf")
    logits[7] = float("nan")
    logits[9, : E // 2] = float("inf")
    logits[11] = torch.finfo(torch.bfloat16).min
    bias = torch.randn(E, generator=g) * 0.02 if E % 2 else None
    check_route(logits, bias, (E, k, G, TG, score, gs, T % 2 == 0, 2.5), dt)


def test_route_scored_strided_rows_and_matches_sigmoid_router():
    """Rows of a wider buffer; and with sigmoid scores, groups by their two
    best and normalised weights it is coli_moe_route, bit for bit."""
    T, E, k = 37, 256, 8
    wide = torch.randn(T, E + 9, generator=gen(8)).cuda()
    lg = wide[:, 5:5 + E]
    check_route(lg, None, (E, k, 8, 4, "softmax", "max", True, 1.0))
    bias = (torch.randn(E, generator=gen(9)) * 0.01).cuda()
    out = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
           for _ in range(2)]
    B.coli_moe_route(B.router_cfg(E, k, 8, 4, 1, 2.5), lg.contiguous(), bias, *out[0])
    B.coli_moe_route_scored(B.score_cfg(E, k, 8, 4, B.SCORE_SIGMOID, B.GROUP_TOP2, 1, 2.5), lg, bias, *out[1])
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


# --- together ----------------------------------------------------------------------------------
class Layer8:
    """A routed layer in 8 bits, from logits to y, as a program calls it."""

    def __init__(self, T, E, k, H, I, dt, seed=0):
        self.T, self.E, self.k, self.H, self.I, self.dt = T, E, k, H, I, dt
        self.w1, self.s1 = codes(E, 2 * I, H, seed=seed), scales(E, 2 * I, seed=seed)
        self.w2, self.s2 = codes(E, H, I, seed=seed + 1), scales(E, H, seed=seed + 1)
        z = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        i32, P = torch.int32, T * k
        self.cfg = B.score_cfg(E, k, score=B.SCORE_SOFTMAX)
        self.x, self.logits = z(T, H), z(T, E)
        self.idx, self.w = z(T, k, d=i32), z(T, k, d=torch.float32)
        self.tab = [z(E, d=i32), z(E + 1, d=i32), z(P, d=i32), z(E, d=i32), z(1, d=i32)]
        self.q, self.qs = z(T, H, d=torch.int8), z(T, d=torch.float32)
        self.gu, self.hq, self.hs = z(P, 2 * I), z(P, I, d=torch.int8), z(P, d=torch.float32)
        self.o, self.y = z(P, H), z(T, H)

    def fill(self, seed):
        self.x.copy_(torch.randn(self.T, self.H, generator=gen(seed)))
        self.logits.copy_(torch.randn(self.T, self.E, generator=gen(seed, 1)))

    def run(self):
        B.coli_moe_route_scored(self.cfg, self.logits, None, self.idx, self.w)
        B.coli_moe_dispatch(self.idx, self.E, *self.tab)
        B.coli_quant_act_token(self.x, self.q, self.qs)
        B.coli_gemm_q8_grouped(self.q, self.qs, self.w1.view(torch.uint8), self.s1, self.tab[1],
                               self.tab[2], self.gu, fan=self.k)
        B.coli_swiglu_quant_token(self.gu[:, :self.I], self.gu[:, self.I:], self.hq, self.hs)
        B.coli_gemm_q8_grouped(self.hq, self.hs, self.w2.view(torch.uint8), self.s2, self.tab[1],
                               self.tab[2], self.o)
        B.coli_moe_combine(self.o, self.idx, self.w, self.y)

    def reference(self):
        """The layer in 64 bits, rounding only where a buffer's type rounds."""
        idx, w = R.route(f32(self.logits), None, self.k, score="softmax")
        q, s = R.quant(f64(self.x))
        y = np.zeros((self.T, self.H))
        for e in range(self.E):
            for t, j in np.argwhere(idx == e):
                gu = R.product(q[t:t + 1], s[t:t + 1], self.w1[e].cpu().numpy(), self.s1[e].cpu().numpy())
                gu = torch.from_numpy(gu).to(self.dt).double().numpy()
                hq, hs = R.quant(R.swiglu(gu[:, :self.I], gu[:, self.I:]))
                y[t] += w[t, j] * R.product(hq, hs, self.w2[e].cpu().numpy(), self.s2[e].cpu().numpy())[0]
        return idx, y


@pytest.mark.parametrize("T,dt", [(1, "f32"), (3, "bf16"), (50, "f32")])
def test_layer_of_8_bit_operators(T, dt):
    """Gate/up results that round the other way move h by one step of their
    type (relative 2 * half_step, twice), a code of h by one at most (1/127 of
    its row's largest value over I terms of random sign); the bound is that
    per-term error times sqrt(I), far below any wrong index or scale."""
    L = Layer8(T, 12, 3, 128, 96, DT[dt])
    L.fill(3)
    L.run()
    idx, y = L.reference()
    np.testing.assert_array_equal(L.idx.cpu().numpy(), idx)
    err = np.abs(f64(L.y) - y).max(axis=1) / np.abs(y).max(axis=1)
    assert (err <= 4 * half_step(DT[dt]) + 1e-3).all(), err


def test_layer_replayed_from_a_graph_on_another_stream():
    """Captured once, replayed on new inputs with eager work between: every
    replay equals the eager result, bit for bit; and two layers on two streams
    do not disturb one another."""
    A, C = Layer8(5, 16, 2, 256, 128, torch.bfloat16), Layer8(70, 16, 2, 256, 128, torch.bfloat16, 5)
    for L in (A, C):
        L.fill(1)
        L.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        A.run()
    for r in range(4):
        A.fill(10 + r)
        C.fill(20 + r)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(st):
            C.run()
        torch.cuda.synchronize()
        ga, gc = A.y.clone(), C.y.clone()
        A.run()
        C.run()
        torch.cuda.synchronize()
        assert torch.equal(ga, A.y) and torch.equal(gc, C.y)


def test_empty_batches():
    e = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    q, s, w, ws = e(0, 64, d=torch.int8), e(0), codes(40, 64), scales(40)
    B.coli_quant_act_token(e(0, 64), q, s)
    B.coli_swiglu_quant_token(e(0, 64), e(0, 64), q, s)
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, e(0, 40))
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    B.coli_gemm_q8_grouped(q, s, codes(2, 40, 64).view(torch.uint8), scales(2, 40), offs,
                           e(0, d=torch.int32), e(0, 40))
    B.coli_moe_combine(e(0, 8), None, e(0, 2), e(0, 8))
    B.coli_moe_route_scored(B.score_cfg(8, 2), e(0, 8), None, e(0, 2, d=torch.int32), e(0, 2))
