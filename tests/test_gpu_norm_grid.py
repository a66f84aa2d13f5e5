"""The residual's norm over more workgroups than a grid's first axis holds (2^20):
rows of the second axis and workgroups past the last row, by 16, 64 and 256
threads a row.  Tolerances as in test_gpu_norm.py."""
import numpy as np
import pytest
import torch

from quantized_moe_coli_amd import binding as B

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.mark.parametrize("T,n,dt", [((1 << 24) + 37, 8, torch.float32), ((1 << 22) + 3, 416, torch.bfloat16),
                                    ((1 << 20) + 1, 2080, torch.bfloat16)])
def test_rows_of_the_second_axis(T, n, dt):
    g = torch.Generator("cuda").manual_seed(n)
    x = torch.empty(T, n, dtype=dt, device="cuda").normal_(generator=g)
    buf = torch.full((T + 64, n), float("nan"), dtype=dt, device="cuda")
    codes = n % 32 == 0
    q = torch.empty(T, n, dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(T, device="cuda") if codes else None
    B.coli_rmsnorm_quant_token(x, None, EPS, q=q, s=s, y=buf[:T])
    assert torch.isnan(buf[T:]).all()
    for t in range(0, T, 1 << 18):
        p = slice(t, min(t + (1 << 18), T))
        ref = x[p].double()
        ref = ref * (ref.square().mean(1, keepdim=True) + np.float64(np.float32(EPS))).rsqrt()
        half = 0.0 if dt is torch.float32 else torch.finfo(dt).eps / 2 * (1 + 2.0 ** -24)
        assert ((buf[p].double() - ref).abs() <= ref.abs() * (half + 2.0 ** -24 + 2.0 ** -34)).all(), t
        if codes:
            scale = ref.abs().amax(1) / 127
            # the largest value, 1 / 127 and their product are a rounding each
            assert ((s[p].double() - scale).abs() <= scale * 3.01 * 2.0 ** -24).all(), t
            unit = s[p].double()[:, None]
            # half a code, the values' roundings, and a clamp at 127 codes of a scale that is low
            assert ((q[p].double() * unit - ref).abs() <= (0.5 + 127 * 4 * 2.0 ** -24) * unit).all(), t
