"""The residual's norm with 8-bit codes (coli_rmsnorm_quant_token) against the
definition in 64 bits, through the C ABI.

Tolerances.  h is one binary32 sum and one rounding: equal bit for bit.  The
binary64 evaluation of y is off by less than (n + 8) 2^-53 of it, below 2^-35 for
every n here, before y is rounded to binary32 (half a step, 2^-24) and to its
type (half a step more, relative to the rounded value; for fp16 results below
the smallest normal value half a step is 2^-25).  Codes belong to the binary32 y:
the reference makes them from its own, which is the same but where a value lies
within 2^-35 of a rounding's border.  Then a row's scale may be its neighbour,
and only then may the row's codes differ, by one.
"""
import numpy as np
import pytest
import torch

import q8_ref as R
from quantized_moe_coli_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def gen(*seed):
    return torch.Generator().manual_seed(sum((i + 1) * int(v) for i, v in enumerate(seed)) + 17)


def rows(T, n, dt, seed=0, pad=0, shift=0, scale=1.0):
    x = (scale * torch.randn(T, n + pad, generator=gen(T, n, seed))).to(dt).cuda()
    return x[:, shift:shift + n]


def reference(x, res, gain, eps=EPS):
    """h (binary32) and y (binary64) of the definition, on the host."""
    h = x.float().cpu()
    if res is not None:
        h = h + res.float().cpu()
    h64 = h.double().numpy()
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((h64 * h64).sum(axis=1, keepdims=True) / h64.shape[1] + np.float64(np.float32(eps)))
        y = h64 * r
    if gain is not None:
        y = y * gain.double().cpu().numpy()
    return h, y


def check(x, res, gain, h=None, y=None, q=None, s=None, ref=None, eps=EPS):
    hr, yr = ref or reference(x, res, gain, eps)
    if h is not None:
        assert torch.equal(h.cpu(), hr.to(h.dtype)) or np.array_equal(
            h.float().cpu().numpy(), hr.to(h.dtype).float().numpy(), equal_nan=True)
    if y is not None:
        got = y.double().cpu().numpy()
        fin = np.isfinite(yr)
        assert np.isnan(got[~fin]).all()
        half = torch.finfo(y.dtype).eps / 2
        tol = np.abs(yr) * (half * (1 + 2.0 ** -24) + 2.0 ** -24 + 2.0 ** -34)
        if y.dtype is torch.float16:
            tol = np.maximum(tol, 2.0 ** -25 * (1 + 2.0 ** -10))
        tol = np.maximum(tol, 2.0 ** -149)
        assert (np.abs(got - yr) <= tol)[fin].all()
    if q is not None:
        with np.errstate(over="ignore"):
            rq, rs = R.quant(yr.astype(np.float32))
        gs, gq = s.cpu().numpy(), q.cpu().numpy()
        same = (gs == rs) | (np.isnan(gs) & np.isnan(rs))
        near = np.abs(gs - rs) <= np.abs(rs) * 2.0 ** -23
        assert (same | near).all() and same.mean() >= 0.99 - 1.0 / len(same)
        np.testing.assert_array_equal(gq[same], rq[same])
        assert (np.abs(gq.astype(int) - rq)[~same] <= 1).all()


def call(x, res=None, gain=None, codes=True, y=True, h=True, stream=None, eps=EPS):
    """The call with outputs of its own; rows of h and y lie in wider buffers,
    whose other elements have to stay."""
    T, n = x.shape
    hb = torch.full((T, n + 8), 77.0, dtype=x.dtype, device="cuda") if h else None
    yb = torch.full((T, n + 8), 77.0, dtype=x.dtype, device="cuda") if y else None
    q = torch.full((T, n), 99, dtype=torch.int8, device="cuda") if codes else None
    s = torch.full((T,), -1.0, device="cuda") if codes else None
    B.coli_rmsnorm_quant_token(x, gain, eps, q=q, s=s, y=None if yb is None else yb[:, :n],
                               res=res, h=None if hb is None else hb[:, :n], stream=stream)
    for b in (hb, yb):
        if b is not None:
            assert (b[:, n:] == 77.0).all()
    return dict(h=None if hb is None else hb[:, :n], y=None if yb is None else yb[:, :n], q=q, s=s)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,n,pad,shift", [
    (1, 32, 0, 0), (5, 64, 0, 0), (3, 128, 8, 0), (7, 160, 0, 0), (2, 512, 0, 0), (3, 544, 32, 0),
    (2, 2048, 0, 0), (2, 2080, 0, 0), (1, 6144, 0, 0), (3, 8192, 8, 0), (2, 8224, 0, 0), (2, 32768, 0, 0),
    (1, 33024, 0, 0), (1, 131040, 0, 0), (4, 96, 5, 3), (2, 6176, 1, 1), (1, 40032, 3, 2),
    (513, 64, 0, 0), (514, 160, 0, 0), (600, 2048, 8, 0), (515, 2080, 0, 0), (520, 8224, 0, 0),
    (513, 96, 5, 3), (2049, 64, 0, 0), (2053, 160, 0, 0), (2100, 2048, 8, 0), (2049, 512, 0, 0),
    (2049, 96, 5, 3), (385, 2080, 0, 0),
    (2061, 224, 0, 0), (2049, 384, 8, 0), (2052, 288, 7, 1), (386, 9952, 7, 0), (385, 9952, 0, 0)])
def test_norm_codes(dt, T, n, pad, shift):
    x, res = rows(T, n, DT[dt], 1, pad, shift), rows(T, n, DT[dt], 2, pad, shift, 3.0)
    gain = (1 + 0.3 * torch.randn(n, generator=gen(n))).cuda()
    check(x, res, gain, **call(x, res, gain))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,n", [(1, 1), (3, 2), (70, 7), (5, 9), (4, 127), (1021, 129), (9, 513), (700, 1001),
                                 (2, 8191), (1, 8193), (2, 32773), (1, 131071), (1, 131072), (530, 33),
                                 (2051, 33), (2049, 1001), (2200, 513)])
def test_norm_rows_of_any_length(dt, T, n):
    x, res = rows(T, n, DT[dt], 3), rows(T, n, DT[dt], 4, scale=2.0)
    gain = (1 + 0.3 * torch.randn(n, generator=gen(n, 1))).cuda()
    check(x, res, gain, **call(x, res, gain, codes=False))


@pytest.mark.parametrize("has_res", [0, 1])
@pytest.mark.parametrize("has_gain", [0, 1])
@pytest.mark.parametrize("outs", ["codes", "y", "codes y", "codes h", "y h"])
@pytest.mark.parametrize("T,n", [(3, 2048), (600, 96), (2, 40000)])
def test_norm_each_operand_and_output_may_be_left_out(has_res, has_gain, outs, T, n):
    x = rows(T, n, torch.bfloat16, 5)
    res = rows(T, n, torch.bfloat16, 6) if has_res else None
    gain = torch.randn(n, generator=gen(n, 2)).cuda() if has_gain else None
    check(x, res, gain, **call(x, res, gain, codes="codes" in outs, y="y" in outs, h="h" in outs))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("T,n", [(2, 6144), (600, 160), (1, 40000), (3, 1001)])
@pytest.mark.parametrize("where", ["h=res", "h=x", "h=res y=x", "h=x y=res", "y=x"])
def test_norm_in_place(dt, T, n, where):
    x, res = rows(T, n, DT[dt], 7), rows(T, n, DT[dt], 8)
    ref = reference(x, res, None)
    bufs = dict(x=x, res=res)
    out = {k: bufs[v] for k, v in (p.split("=") for p in where.split())}
    codes = n % 32 == 0
    q = torch.empty(T, n, dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(T, device="cuda") if codes else None
    if not codes and "y" not in out:
        out["y"] = torch.empty_like(x)
    B.coli_rmsnorm_quant_token(x, None, EPS, q=q, s=s, res=res, **out)
    check(None, None, None, ref=ref, q=q, s=s, **out)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n", [96, 2048, 40000])
def test_norm_extremes(dt, n):
    """Zero rows, tiny and huge ones, and rows with a NaN or infinities, each beside
    others that stay as they are."""
    t = DT[dt]
    big = torch.finfo(t).max
    x = torch.randn(9, n, generator=gen(n, 3))
    x[1] = 0
    x[2] *= 1e-6 if t is torch.float16 else 1e-30
    x[3] = big / 2 * torch.sign(x[3])
    x[4, 5] = float("nan")
    x[5, n - 1] = float("inf")
    x[6, 0], x[6, 1] = float("inf"), -float("inf")
    x[7] = 0
    x[7, 3] = torch.finfo(t).tiny
    x = x.to(t).cuda()
    for res in (None, x.clone()):
        out = call(x, res)
        check(x, res, None, **out)
        s = out["s"].cpu()
        assert s[1] == 0 and torch.isnan(s[[4, 5, 6]]).all() and torch.isfinite(s[[0, 2, 3, 7, 8]]).all()
        assert (out["q"][[1, 4, 5, 6]] == 0).all() and (out["y"][1] == 0).all()
        assert torch.isnan(out["y"][4]).all() and torch.isnan(out["y"][5, n - 1])


def test_norm_eps_counts():
    x = rows(4, 256, torch.float32, 9, scale=1e-3)
    for eps in (1e-12, 1e-6, 0.1, 7.0):
        check(x, None, None, eps=eps, **call(x, eps=eps))


def test_norm_many_short_rows():
    """More rows than a grid's first axis holds workgroups of."""
    T, n = (1 << 22) + 37, 8
    x = torch.randn(T, n, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    y = torch.full((T, n), float("nan"), device="cuda")
    B.coli_rmsnorm_quant_token(x, None, EPS, y=y)
    ref = x.double() * (x.double().square().mean(1, keepdim=True) + np.float64(np.float32(EPS))).rsqrt()
    assert ((y - ref).abs() <= ref.abs() * (2.0 ** -24 + 2.0 ** -34)).all()


def test_norm_rows_far_apart():
    """Offsets of elements that pass 32 bits."""
    ld = (1 << 31) // 2 + 64
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 96), (ld, 1))
    x.copy_(rows(3, 96, torch.bfloat16, 10))
    y = buf.as_strided((3, 96), (ld, 1), 128)
    q, s = torch.empty(3, 96, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    B.coli_rmsnorm_quant_token(x, None, EPS, q=q, s=s, y=y)
    check(x, None, None, y=y, q=q, s=s)


def test_norm_empty_batch_writes_nothing():
    x = torch.empty(0, 64, device="cuda")
    B.coli_rmsnorm_quant_token(x, None, EPS, y=torch.empty(0, 64, device="cuda"))


def test_norm_on_a_given_stream_and_in_a_graph():
    x, res = rows(5, 2048, torch.bfloat16, 11), rows(5, 2048, torch.bfloat16, 12)
    first = call(x, res)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    again = call(x, res, stream=st)
    st.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    q, s = torch.empty_like(first["q"]), torch.empty_like(first["s"])
    y = torch.empty(5, 2048, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.coli_rmsnorm_quant_token(x, None, EPS, q=q, s=s, y=y, res=res)
    for i in range(4):
        x.copy_(rows(5, 2048, torch.bfloat16, 20 + i))
        g.replay()
        torch.cuda.synchronize()
        check(x, res, None, y=y, q=q, s=s)


def test_norm_results_do_not_depend_on_the_batch():
    """The same rows in batches that other kernels take."""
    for n in (128, 2048, 6144):
        x = rows(1200, n, torch.bfloat16, 13)
        whole = call(x)
        part = call(x[300:340])
        for k in whole:
            assert torch.equal(whole[k][300:340], part[k]), (n, k)
