"""Calls of the 8-bit operators whose arguments the host decides on: they are
accepted or refused before a device is touched."""
import pytest
import torch

from quantized_moe_coli_amd import binding as B

P = 1 << 20  # an aligned address, never followed


@pytest.mark.parametrize("dt", [B.COLI_F32, B.COLI_BF16, B.COLI_F16])
def test_combine_takes_float32_rows_with_any_result_type(dt):
    fn = B.lib().coli_moe_combine
    flag = B.COLI_COMBINE_O_F32

    def call(dtype=dt | flag, o=P, ldo=8, T=3):
        return fn(dtype, o, ldo, None, P, T, 2, 8, None, 0, P, 8, None)

    assert call(T=0) == B.COLI_OK
    if not torch.cuda.is_available():
        assert call() == B.COLI_ERR_DEVICE
    for bad in (dict(o=P + 2), dict(ldo=7), dict(o=None), dict(dtype=3 | flag), dict(dtype=dt | 2 * flag),
                dict(dtype=-1), dict(dtype=dt | flag | 1 << 30)):
        assert call(**bad) == B.COLI_ERR_INVALID_ARG, bad


def test_package_follows_a_function_replaced_in_the_binding(monkeypatch):
    """The package's names are the binding's at the time of each access."""
    import quantized_moe_coli_amd as C

    assert C.coli_gemm_q8 is B.coli_gemm_q8 and C.coli_moe_route is B.coli_moe_route  # read once
    for name in ("coli_gemm_q8", "coli_moe_route"):
        monkeypatch.setattr(B, name, len)
        assert getattr(C, name) is len
    assert "coli_gemm_q8" not in vars(C)
