"""The 8-bit operators on the paths that a model's layers take: results of the
types and strides that are stored in 16-byte words, rings that come round
several times, tokens in batches of any size.  Against 64-bit forms, with the
tolerances that test_gpu_q8.py derives.
"""
import numpy as np
import pytest
import torch

import q8_ref as R
from quantized_moe_coli_amd import binding as B
from test_gpu_q8 import (DT, acts, assert_product, check_route, codes, f64, gen, half_step, routing,
                         scales)

pytestmark = pytest.mark.gpu


# --- combine of float32 rows -------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,H,pad,add", [(1, 1, 1, 0, False), (3, 8, 6144, 0, False), (5, 2, 100, 4, True),
                                           (2, 32, 515, 0, True), (700, 3, 64, 0, True), (4, 2, 2064, 4, True),
                                           (2, 4, 33, 1, False), (3, 2, 512, 2, False)])
def test_combine_of_float32_rows(dt, T, k, H, pad, add):
    """At most k roundings of partial sums in binary32, each no larger than the
    sum of the terms' sizes, and the result's rounding to its type: the rows
    themselves are not rounded."""
    o = acts(T * k, H, torch.float32, 4, pad)
    w = torch.randn(T, k, generator=gen(T, k)).cuda()
    idx = torch.randint(-1, 3, (T, k), generator=gen(T, k, 2), dtype=torch.int32)
    on = (idx >= 0).numpy()
    o[torch.from_numpy(~on.ravel()).cuda()] = float("nan")  # rows that are not read
    a = acts(T, H, DT[dt], 6) if add else None
    y = torch.empty(T, H, dtype=DT[dt], device="cuda")
    B.coli_moe_combine(o, idx.cuda(), w, y, add=a)
    terms = np.where(on[:, :, None], f64(o).reshape(T, k, H) * f64(w)[:, :, None], 0.0)
    ref = terms.sum(1) + (f64(a) if add else 0.0)
    size = np.abs(terms).sum(1) + (np.abs(f64(a)) if add else 0.0)
    tol = k * 2.0 ** -24 * size * 1.01
    tol = tol + half_step(DT[dt]) * (np.abs(ref) + tol) + (2.0 ** -25 if dt == "f16" else 0.0)
    assert (np.abs(f64(y) - ref) <= tol).all()
    if add:  # in place
        B.coli_moe_combine(o, idx.cuda(), w, a, add=a)
        assert torch.equal(a, y)


@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 16, 264, 96), (45, 4, 8, 512, 160), (300, 2, 3, 260, 64)])
def test_experts_product_in_float32_and_its_sum_in_bf16(T, k, E, N, K):
    """The experts' second product with float32 results and their sum in bf16:
    one rounding to bf16 from the 64-bit definition, beside what binary32 adds
    (a product's three roundings and the k of the sum, relative to the terms)."""
    idx = routing(T, k, E, 5, 0.2)
    offs, perm = (torch.from_numpy(v).cuda() for v in R.tables(idx.numpy(), E))
    P = T * k
    q, s, w, ws = codes(P, K, seed=1), scales(P), codes(E, N, K, seed=2), scales(E, N)
    wt = torch.rand(T, k, generator=gen(T, k)).cuda()
    o, y = torch.full((P, N), float("nan"), device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, offs, perm, o)
    B.coli_moe_combine(o, idx.cuda(), wt, y)
    flat, terms = idx.numpy().ravel(), np.zeros((P, N))
    for e in range(E):
        r = np.flatnonzero(flat == e)
        terms[r] = R.product(q.cpu().numpy()[r], s.cpu().numpy()[r], w[e].cpu().numpy(), ws[e].cpu().numpy())
    terms = terms.reshape(T, k, N) * f64(wt)[:, :, None]
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    tol = (k + 3) * 2.0 ** -24 * 1.01 * size
    tol = tol + half_step(torch.bfloat16) * (np.abs(ref) + tol)
    assert (np.abs(f64(y) - ref) <= tol).all()


def test_combine_refuses_rows_of_another_16_bit_type():
    w, y = torch.rand(2, 2).cuda(), torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="o must be torch.bfloat16"):
        B.coli_moe_combine(acts(4, 8, torch.float16), None, w, y)
    with pytest.raises(ValueError, match="add must be torch.bfloat16"):
        B.coli_moe_combine(acts(4, 8, torch.float32), None, w, y, add=acts(2, 8, torch.float32))


# --- one definition in every kernel ------------------------------------------------------------
def fused(x, s, b):
    """x * s + b of float32 arrays in binary64, the product exact and the sum
    rounded to odd (where it is inexact, to the neighbour with an odd last
    place), so that a rounding to fewer bits is that of the exact value."""
    p, b = x.astype(np.float64) * s.astype(np.float64), b.astype(np.float64)
    v = p + b
    t = v - p
    err = (p - (v - t)) + (b - t)
    even = (v.view(np.int64) & 1) == 0
    v = np.where((err != 0) & even, np.nextafter(v, np.where(err > 0, np.inf, -np.inf)), v)
    return v


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bias", [False, True])
def test_a_tokens_result_is_the_same_in_every_batch(dt, bias):
    """Batches and numbers of channels that take each kernel of the dense
    product: a token's channels have the same bits in all of them, and those of
    the definition: sum, conversion, channel's scale, and the token's scale and
    the bias in one step to float32 and from there to bf16, or to fp16."""
    K, N = 416, 65536
    q, s = codes(1500, K, seed=1), scales(1500)
    w, ws = codes(N, K, seed=2), scales(N, seed=3)
    b = torch.randn(N, generator=gen(N)).cuda() if bias else None
    y = {}
    for T, n in ((1, 2064), (1, 6144), (45, 6144), (130, 6144), (200, 6144), (512, 6144), (1021, 6144),
                 (1500, 6144), (45, N)):
        r = torch.empty(T, n, dtype=DT[dt], device="cuda")
        B.coli_gemm_q8(q[:T], s[:T], w[:n].view(torch.uint8), ws[:n], r, bias=b[:n] if bias else None)
        y[T, n] = r
    most = y[1500, 6144]
    for (T, n), r in y.items():
        m = min(n, 6144)
        assert torch.equal(r[:, :m], most[:T, :m]), (T, n)
    t, n = 160, 400
    acc = (f64(q[:t]) @ f64(w[:n]).T).astype(np.float32)
    sn, st = ws[:n].cpu().numpy()[None], s[:t].cpu().numpy()[:, None]
    bn = b[:n].cpu().numpy()[None] if bias else np.zeros((1, 1), np.float32)
    ref = fused((acc * sn).astype(np.float32), st, bn)
    ref = torch.from_numpy(ref.astype(np.float16 if dt == "f16" else np.float32)).to(DT[dt])
    assert torch.equal(most[:t, :n].cpu(), ref)


@pytest.mark.parametrize("dt", DT)
def test_a_pairs_result_is_the_same_in_every_batch(dt):
    """The same over experts: each kernel gives a pair the bits that the dense
    product gives its token."""
    K, N = 416, 2048
    w, ws = codes(40, N, K, seed=2), scales(40, N, seed=3)
    q, s = codes(2400, K, seed=1), scales(2400)
    for E, per in ((40, 2), (2, 3), (40, 40), (2, 40), (4, 60), (3, 700)):
        P = E * per
        offs = (torch.arange(E + 1) * per).to(torch.int32).cuda()
        y = torch.empty(P, N, dtype=DT[dt], device="cuda")
        B.coli_gemm_q8_grouped(q[:P], s[:P], w[:E].view(torch.uint8), ws[:E], offs,
                               torch.arange(P, dtype=torch.int32).cuda(), y)
        for e in range(E):
            r = torch.empty(per, N, dtype=DT[dt], device="cuda")
            B.coli_gemm_q8(q[e * per:(e + 1) * per], s[e * per:(e + 1) * per], w[e].view(torch.uint8), ws[e], r)
            assert torch.equal(y[e * per:(e + 1) * per], r), (E, per, e)


# --- the token's scale -------------------------------------------------------------------------
@pytest.mark.parametrize("dt", DT)
def test_token_scale_against_the_quotient(dt):
    """s = fl(a c) with c = fl(1 / 127) and 127 c = 1 - 2^-28: off a / 127 by at
    most 2^-24 + 2^-28 of it.  With both roundings of a code's quotient, the
    value q s is off x by at most half a scale and 127 * 2^-24 of it (the
    quotient's rounding; at the row's largest, a / s <= 127 (1 + 2^-23))."""
    c = float(np.float32(1) / np.float32(127))
    assert 127 * c == 1 - 2.0 ** -28
    T, n = 2000, 256
    x = acts(T, n, DT[dt], 12)
    q, s = torch.empty(T, n, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    B.coli_quant_act_token(x, q, s)
    x, s = f64(x), f64(s)
    a = np.abs(x).max(1)
    assert (np.abs(s - a / 127) <= (2.0 ** -24 + 2.0 ** -28) * (1 + 2.0 ** -24) * a / 127).all()
    off = np.abs(x - f64(q) * s[:, None])
    assert (off <= s[:, None] * (0.5 + 127 * 2.0 ** -23)).all()


# --- results stored in 16-byte words -----------------------------------------------------------
def padded(rows, cols, pad, dt):
    """[rows, cols] of a wider buffer whose other columns hold 77, and these."""
    wide = torch.full((rows, cols + pad), 77.0, dtype=dt, device="cuda")
    return wide[:, :cols], wide[:, cols:]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,K,pad", [
    # rows of whole words, and rows that end inside one (their stride is of whole
    # words): 16 x 16, 16 x 32, 32 x 64, 64 x 32, 64 x 64, the tiles, the sweep
    (1, 2048, 416, 0), (13, 2049, 96, 7), (3, 6144, 160, 8), (3, 6145, 160, 7), (130, 6152, 160, 0),
    (130, 6147, 96, 5), (61, 6144, 544, 0), (61, 6145, 352, 7), (200, 6144, 96, 0), (200, 6145, 160, 7),
    (509, 6144, 288, 0), (512, 6145, 160, 7), (700, 6144, 416, 0), (1021, 6145, 96, 7), (1500, 6145, 160, 7),
    (2047, 6144, 96, 0), (64, 65536, 160, 0), (45, 65545, 96, 7)])
def test_dense_results_in_whole_words(dt, T, N, K, pad):
    q, w, s, ws = codes(T, K, seed=1), codes(N, K, seed=2), scales(T), scales(N, seed=3)
    y, rest = padded(T, N, pad, DT[dt])
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y)
    assert_product(y, R.product(q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy()), DT[dt])
    assert (rest == 77.0).all()


def check_experts(counts, N, K, dt, pad, fan=1, seed=1):
    """The experts' product with counts[e] pairs of expert e in any order, and
    five of no expert, into rows of a wider buffer."""
    E, P = len(counts), sum(counts) + 5
    e_of = np.concatenate([np.repeat(np.arange(E), counts), np.full(5, -1)])
    e_of = e_of[torch.randperm(P, generator=gen(P, seed)).numpy()]
    offs, perm = (torch.from_numpy(v).cuda() for v in R.tables(e_of[:, None], E))
    rows = (P + fan - 1) // fan
    q, s, w, ws = codes(rows, K, seed=1), scales(rows), codes(E, N, K, seed=2), scales(E, N)
    y, rest = padded(P, N, pad, DT[dt])
    B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, offs, perm, y, fan=fan)
    qn, sn = q.cpu().numpy(), s.cpu().numpy()
    for e in range(E):
        p = np.flatnonzero(e_of == e)
        if len(p):
            ref = R.product(qn[p // fan], sn[p // fan], w[e].cpu().numpy(), ws[e].cpu().numpy())
            assert_product(y[torch.from_numpy(p).cuda()], ref, DT[dt])
    assert (y[torch.from_numpy(np.flatnonzero(e_of < 0)).cuda()] == 77.0).all() and (rest == 77.0).all()


def spread(E, per):
    """E counts around ``per``, one of them zero and one of them one."""
    c = [max(2, per * (3 + e % 7) // 6) for e in range(E)]
    c[E // 2], c[E // 3] = 0, 1
    return c


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,per,N,K,pad", [
    # 16 x 32, 64 x 32, the sweeps of 32 and 64 tokens, the tile: rows of whole
    # words, rows that end inside one, rows of no alignment
    (9, 4, 264, 96, 0), (9, 4, 257, 160, 7), (9, 4, 260, 96, 1), (9, 40, 264, 160, 0), (9, 40, 257, 96, 7),
    (9, 40, 260, 96, 1), (65, 5, 1104, 96, 0), (65, 5, 1097, 160, 7), (65, 5, 1104, 96, 3),
    (66, 25, 1104, 160, 0), (66, 25, 1097, 96, 7), (66, 25, 1104, 96, 3), (4, 150, 264, 96, 0),
    (4, 150, 257, 160, 7), (4, 150, 260, 96, 1)])
def test_experts_results_in_whole_words(dt, E, per, N, K, pad):
    check_experts(spread(E, per), N, K, dt, pad, fan=1 + per % 2)


# --- rings that come round several times --------------------------------------------------------
@pytest.mark.parametrize("T,N,K", [
    # many stages of each dense kernel, with a part stage at the end and without:
    # 16 x 16 (8 stages of 256), 16 x 32 (6), 32 x 64 and 64 x 32 (3), 64 x 64
    # (2), the tiles (2 or 3 of 128, 4 with one workgroup a CU), the sweep (4 chunks)
    (3, 70, 6176), (13, 4096, 6144), (16, 6145, 4128), (130, 6147, 2080), (61, 8200, 2080), (64, 6144, 2048),
    (200, 6145, 1568), (512, 6145, 2080), (509, 6144, 2048), (700, 6145, 2080), (1500, 6145, 2080),
    (1505, 6144, 1024), (45, 65536, 2080), (33, 65537, 2048)])
def test_dense_rings_come_round(T, N, K):
    q, w, s, ws = codes(T, K, seed=1), codes(N, K, seed=2), scales(T), scales(N, seed=3)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    B.coli_gemm_q8(q, s, w.view(torch.uint8), ws, y)
    at = torch.randperm(N, generator=gen(N))[:2500]  # every channel block is compared in some row
    ref = R.product(q.cpu().numpy(), s.cpu().numpy(), w.cpu()[at].numpy(), ws.cpu()[at].numpy())
    assert_product(y[:, at.cuda()], ref, torch.bfloat16)


@pytest.mark.parametrize("fan", [1, 2])
@pytest.mark.parametrize("counts,N,K", [
    # the tile with 1 to 8 groups of 32 tokens for a wave, and two tiles of an
    # expert: 2 to 4 stages of 128 bytes
    ([20, 40, 70, 100, 140, 170, 200, 256, 290], 260, 2080), ([31, 64, 90, 127, 150, 191, 220, 230, 513], 300, 2048),
    ([20, 40, 70, 100, 140, 170, 200, 256, 290], 60, 1056),
    # the rings of 16 and 64 tokens (3 stages of 256 bytes)
    ([1, 0, 16, 5, 17, 3], 70, 2080), ([2, 9, 0, 30], 45, 6144), ([33, 64, 20, 70, 1], 70, 2080),
    ([50, 12, 65], 40, 4096),
    # the sweeps of 32 and 64 tokens (chunks of 128 bytes, 4 and 3 ahead)
    (spread(65, 5), 1100, 2432), (spread(64, 11), 1024, 2400), (spread(66, 25), 1030, 2432),
    (spread(64, 45), 1024, 2048)])
def test_experts_rings_come_round(counts, N, K, fan):
    check_experts(counts, N, K, "bf16", 0, fan=fan)


# --- routing of large fp16 batches ---------------------------------------------------------------
@pytest.mark.parametrize("score,gs", [("softmax", "max"), ("softmax", "top2"), ("sigmoid", "top2"),
                                      ("sigmoid", "max")])
@pytest.mark.parametrize("T,E,k,G,TG", [(1024, 256, 8, 1, 1), (1029, 256, 8, 8, 4), (2050, 60, 6, 4, 2),
                                        (1025, 16, 9, 16, 9), (4097, 45, 5, 9, 3), (1027, 257, 16, 1, 1)])
def test_route_scored_fp16_batches(score, gs, T, E, k, G, TG):
    """fp16 logits (many of them equal), dead experts, rows without any, rows of
    the type's lowest value, rows of a wider buffer."""
    g = gen(T, E, k)
    wide = (torch.randn(T, E + 3, generator=g) * 2).to(torch.float16)
    wide[::3] = torch.randint(-3, 4, (len(range(0, T, 3)), E + 3), generator=g).to(torch.float16)
    wide[torch.rand(T, E + 3, generator=g) < 0.1] = float("-inf")
    wide[5], wide[7], wide[11] = float("-inf"), float("nan"), torch.finfo(torch.float16).min
    wide[9, : E // 2] = float("inf")
    bias = torch.randn(E, generator=g) * 0.02 if E % 2 else None
    check_route(wide.cuda()[:, 2:2 + E], bias, (E, k, G, TG, score, gs, T % 2 == 0, 2.5))


# --- streams -------------------------------------------------------------------------------------
@pytest.mark.parametrize("as_handle", [False, True])
def test_experts_calls_on_a_given_stream(as_handle):
    """SwiGLU's codes, the experts' product and the combine enqueue on the
    stream they are given: behind a wait there, nothing is written yet when the
    current stream looks, and all of it is afterwards."""
    T, k, E, H, I = 6, 2, 4, 72, 64
    P = T * k
    g, u = acts(P, I, torch.bfloat16, 1), acts(P, I, torch.bfloat16, 2)
    idx = routing(T, k, E, 3)
    offs, perm = (torch.from_numpy(v).cuda() for v in R.tables(idx.numpy(), E))
    w, ws = codes(E, H, I, seed=3), scales(E, H)
    wt, idx = torch.rand(T, k, generator=gen(4)).cuda(), idx.cuda()
    q, s = torch.full((P, I), 99, dtype=torch.int8, device="cuda"), torch.full((P,), -1.0, device="cuda")
    o, y = torch.full((P, H), 5.0, device="cuda"), torch.full((T, H), 7.0, device="cuda")
    st = torch.cuda.Stream()
    at = st.cuda_stream if as_handle else st

    def run():
        B.coli_swiglu_quant_token(g, u, q, s, stream=at)
        B.coli_gemm_q8_grouped(q, s, w.view(torch.uint8), ws, offs, perm, o, stream=at)
        B.coli_moe_combine(o, idx, wt, y, stream=at)
        return [t.clone() for t in (q, s, o, y)]  # on the current stream, which does not wait

    run()  # loads the kernels, which takes longer than the wait below
    torch.cuda.synchronize()
    for t, v in ((q, 99), (s, -1.0), (o, 5.0), (y, 7.0)):
        t.fill_(v)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(200_000_000)  # what follows on this stream waits
    early = run()
    torch.cuda.current_stream().synchronize()
    assert not st.query()  # it waits still
    st.synchronize()
    assert [t.unique().tolist() for t in early] == [[99], [-1.0], [5.0], [7.0]]
    rq, rs = R.quant(R.swiglu(f64(g), f64(u)))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    flat, ref = idx.cpu().numpy().ravel(), np.zeros((P, H))
    for e in range(E):
        p = np.flatnonzero(flat == e)
        ref[p] = R.product(rq[p], rs[p], w[e].cpu().numpy(), ws[e].cpu().numpy())
    assert_product(o, ref, torch.float32)
    terms = f64(o).reshape(T, k, H) * f64(wt)[:, :, None]
    assert (np.abs(f64(y) - terms.sum(1)) <= (k + 1) * 2.0 ** -24 * 1.01 * np.abs(terms).sum(1)).all()


# --- four tokens a wave --------------------------------------------------------------------------
@pytest.mark.parametrize("dt,score,gs", [("f32", "softmax", "max"), ("bf16", "sigmoid", "top2"),
                                         ("f16", "softmax", "top2")])
@pytest.mark.parametrize("T,E,k,G,TG", [(8192, 256, 8, 1, 1), (8195, 256, 16, 8, 4), (4096, 60, 6, 4, 2),
                                        (4099, 16, 9, 16, 9), (8193, 45, 5, 9, 3), (4101, 7, 3, 1, 1),
                                        (8194, 128, 4, 2, 1), (8191, 256, 8, 1, 1), (4095, 64, 8, 1, 1),
                                        (8200, 256, 17, 1, 1), (8197, 512, 8, 8, 3)])
def test_route_scored_four_tokens_a_wave(dt, score, gs, T, E, k, G, TG):
    """Batches from which four tokens share a wave, and neighbours of that
    limit.  Some rows of each kind against the definition; every row against
    the same rows in small batches, which a wave each routes: equal indices,
    and weights whose scores may round differently (by one step, where the two
    orders of a binary64 sum lie on both sides of a border: two half-steps for
    the score and for the sum's, and the quotient's half-step on each side)."""
    g = gen(T, E, k)
    logits = torch.randn(T, E, generator=g) * 2
    logits[::3] = torch.randint(-3, 4, (len(range(0, T, 3)), E), generator=g).float()
    logits[torch.rand(T, E, generator=g) < 0.1] = float("-inf")
    logits[5], logits[7], logits[11] = float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min
    logits[9, : E // 2] = float("inf")
    bias = (torch.randn(E, generator=g) * 0.02).cuda() if E % 2 else None
    lg = logits.to(DT[dt]).cuda()
    norm = T % 2 == 0
    cfg = B.score_cfg(E, k, G, TG, score=B.SCORE_SOFTMAX if score == "softmax" else B.SCORE_SIGMOID,
                      group_score=B.GROUP_TOP2 if gs == "top2" else B.GROUP_MAX, norm_topk_prob=int(norm),
                      routed_scaling_factor=2.5)
    idx, w = torch.full((T, k), 12345, dtype=torch.int32, device="cuda"), torch.full((T, k), 9.0, device="cuda")
    B.coli_moe_route_scored(cfg, lg, bias, idx, w)
    si, sw = torch.empty_like(idx), torch.empty_like(w)
    for a in range(0, T, 1000):
        B.coli_moe_route_scored(cfg, lg[a:a + 1000], bias, si[a:a + 1000], sw[a:a + 1000])
    assert torch.equal(idx, si)
    assert ((w - sw).abs().double() <= 6 * 2.0 ** -24 * sw.abs().double()).all()
    some = torch.cat([torch.arange(40), torch.randint(0, T, (150,), generator=g), torch.arange(T - 20, T)]).cuda()
    ri, rw = R.route(lg[some].float().cpu().numpy(), None if bias is None else bias.cpu().numpy(), k, G, TG, score,
                     gs, norm, 2.5)
    np.testing.assert_array_equal(idx[some].cpu().numpy(), ri)
    assert (np.abs(f64(w[some]) - rw) <= (k + 3) * 2.0 ** -24 * np.abs(rw) + 2.0 ** -149).all()
