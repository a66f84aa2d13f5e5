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


def test_outputs_on_inputs_of_another_row_stride():
    """A row written where another row is read: refused, as long as there is another row."""
    X, R, Y = P, 2 * P, 3 * P
    good = dict(dt=1, x=X, ldx=64, res=R, ldr=96, gain=P, eps=1e-6, T=2, n=64, h=4 * P, ldh=64, y=Y, ldy=64,
                q=5 * P, s=P, st=None)
    refuse("coli_rmsnorm_quant_token", good, [
        dict(h=X, ldh=96), dict(h=R, ldh=64), dict(y=X, ldy=96), dict(y=R, ldy=64), dict(h=X, ldh=65),
        dict(y=X, ldy=96, h=None, ldh=0), dict(h=R, ldh=128, y=None, ldy=0), dict(h=R, ldh=96, y=X, ldy=96),
        dict(res=X, h=X, ldh=64)])
    fn = B.lib().coli_rmsnorm_quant_token
    if not torch.cuda.is_available():
        for change in (dict(h=X), dict(h=R, ldh=96), dict(y=X), dict(y=R, ldy=96), dict(h=R, ldh=96, y=X),
                       dict(T=1, h=X, ldh=96), dict(T=1, y=R, ldy=64), dict(res=None, ldr=0, h=X),
                       dict(res=None, ldr=0, h=None, ldh=0, y=X)):
            assert fn(*dict(good, **change).values()) == B.COLI_ERR_DEVICE, change
