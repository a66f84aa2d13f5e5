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
from test_gpu_lora import some_ids, tables

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
