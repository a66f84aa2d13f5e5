"""How far the adapters' sums of coli_gemm_q8_lora are off, on operands chosen so
that what a kernel leaves out of them shows in the result.

Each row of a has one element, so that u is one exact product, and the codes'
product is a whole number below 2^24 with scales of one, so that it is exact too.
Sizes are those that the ring, the ring by the tokens' order, and the tiles of
128 and 256 rows take.
"""
import pytest
import torch

from quantized_moe_coli_amd import binding as B
from test_gpu_lora import DT, some_ids, tables

pytestmark = pytest.mark.gpu
SIZES = [(3, 64), (61, 1024), (200, 4096), (64, 66000), (300, 4000), (600, 6145), (1500, 6144)]


def run(dt, q, w, x, a, b, ids, scale=None):
    """y of a call with scales of one and a workspace that holds NaN."""
    T, N, L = q.shape[0], w.shape[0], a.shape[0]
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    offs, perm = tables(ids, L)
    work = B.lora_workspace(T, a.shape[1])
    work.fill_(0xFF)
    y = torch.empty(T, N, dtype=dt, device="cuda")
    B.coli_gemm_q8_lora(q, one(T), w.view(torch.uint8), one(N), B.Lora(a, b, scale), x, ids, offs, perm, y, work)
    return y


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("R,r0,r1", [(8, 0, 1), (40, 7, 34), (72, 70, 3)])
def test_low_parts_of_u_and_b_meet(dt, T, N, R, r0, r1):
    """(1 + 2^-8) (1 + 2^-8) - (1 + 3 2^-8) (1 + 2^-8) = -2^-7 - 2^-15: each factor is
    8 bits and a rest of 2^-8, and the two products of the rests are 2^-16 each,
    with one sign, where everything else cancels to 2^-7.  The result has few enough
    bits for each type here, and so has every sum on the way, so it is exact: 2^-15 is
    four times what two pieces of u may lose of these products, 2^-17 of 2.03."""
    t, K, L = DT[dt], 96, 5
    ids = some_ids(T, L, min(T, L), "mixed", 0.1)
    x = torch.zeros(T, K, dtype=t, device="cuda")
    x[:, r0] = x[:, r1] = 2.0 ** (torch.arange(T, device="cuda") % 3 - 1).to(t)
    a = torch.zeros(L, R, K, dtype=t, device="cuda")
    a[:, r0, r0], a[:, r1, r1] = 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8
    sign = 1 - 2 * (torch.arange(N, device="cuda") % 2).to(t)
    b = torch.zeros(L, N, R, dtype=t, device="cuda")
    b[:, :, r0], b[:, :, r1] = (1 + 2.0 ** -8) * sign, -(1 + 2.0 ** -8) * sign
    zero = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    y = run(t, zero(T, K), zero(N, K), x, a, b, ids)
    ref = x[:, r0, None].double() * sign.double() * -(2.0 ** -7 + 2.0 ** -15) * (ids >= 0)[:, None]
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("R", [16, 64, 128])
def test_small_adapters_beside_a_large_product(T, N, R):
    """Every product 127 * 127 * 64 = 1032256 has steps of 2^-4 in binary32, and the
    adapters add R / 16 parts of 0.03, each below half a step.  Their sum is one of 16
    ranks or more: what is added in binary32 is at most R / 32 parts (one, of 16), each
    rounded by half a step, and the sum's own roundings are 2^-24 of 0.24 each."""
    K, L = 64, 3
    ids = some_ids(T, L, min(T, L), "mixed", 0.1)
    full = lambda *s: torch.full(s, 127, dtype=torch.int8, device="cuda")  # noqa: E731
    x = torch.zeros(T, K, device="cuda")
    x[:, 5] = 1
    a = torch.zeros(L, R, K, device="cuda")
    a[:, :, 5] = 1
    b = torch.full((L, N, R), 0.03 / 16, device="cuda")
    y = run(torch.float32, full(T, K), full(N, K), x, a, b, ids)
    ref = 1032256 + R * float(b[0, 0, 0].double()) * (ids >= 0).double()[:, None]
    tol = max(1, R // 32) * 2.0 ** -5 + 6 * R * 2.0 ** -24 * 0.24
    assert ((y.double() - ref).abs() <= tol).all(), float((y.double() - ref).abs().max())
