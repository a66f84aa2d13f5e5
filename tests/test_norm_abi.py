"""Refusals of the residual's norm with 8-bit codes, on the host: every bad
argument is refused before a device is touched."""
import pytest
import torch

from quantized_moe_coli_amd import binding as B
from test_q8_abi import P, no_device_or_empty, refuse

NAN, INF = float("nan"), float("inf")


def test_rmsnorm_quant_token():
    good = dict(dt=1, x=P, ldx=64, res=P, ldr=64, gain=P, eps=1e-6, T=2, n=64, h=P, ldh=64, y=2 * P, ldy=64,
                q=P, s=P, st=None)
    refuse("coli_rmsnorm_quant_token", good, [
        dict(dt=3), dict(dt=-1), dict(x=None), dict(x=P + 1), dict(dt=0, x=P + 2), dict(ldx=63),
        dict(res=P + 1), dict(ldr=63), dict(gain=P + 2), dict(eps=0.0), dict(eps=-1e-6), dict(eps=NAN),
        dict(eps=INF), dict(T=-1), dict(T=(1 << 25) + 1), dict(n=0), dict(n=-32), dict(n=48),
        dict(n=131072, ldx=1 << 20, ldr=1 << 20, ldh=1 << 20, ldy=1 << 20),
        dict(n=131073, q=None, s=None, ldx=1 << 20, ldr=1 << 20, ldh=1 << 20, ldy=1 << 20),
        dict(h=P + 1), dict(ldh=63), dict(y=P + 1), dict(ldy=63), dict(y=P), dict(q=P + 8), dict(s=P + 2),
        dict(q=None), dict(s=None), dict(q=None, s=None, y=None)])
    no_device_or_empty("coli_rmsnorm_quant_token", good, dict(T=0, x=None))


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="device tensor"):
        B.coli_rmsnorm_quant_token(torch.zeros(2, 64), None, 1e-6, y=torch.zeros(2, 64))
