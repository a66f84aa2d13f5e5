"""Refusals of the 8-bit product with low-rank adapters, on the host: every bad
argument is refused before a device is touched."""
import ctypes

import pytest
import torch

from quantized_moe_coli_amd import binding as B
from test_q8_abi import P, UNSUPPORTED, no_device_or_empty, refuse


def adapters(**kw):
    d = dict(n_adapters=4, rank=16, a=P, b=P, scale=P)
    d.update(kw)
    return ctypes.pointer(B.LoraC(*d.values()))


def test_gemm_q8_lora():
    good = dict(q=P, s=P, T=4, w=P, ws=P, N=10, K=64, bias=None, lora=adapters(), x=P, ldx=64, ids=P, offs=P,
                perm=P, dt=1, y=P, ldy=10, ws_=P, wsn=1 << 20, st=None)
    refuse("coli_gemm_q8_lora", good, [
        dict(q=None), dict(q=P + 8), dict(s=None), dict(s=P + 1), dict(T=-1), dict(T=(1 << 20) + 1),
        dict(w=None), dict(w=P + 4), dict(ws=None), dict(ws=P + 2), dict(N=0), dict(N=-3), dict(K=0),
        dict(K=40), dict(K=131072), dict(bias=P + 2), dict(dt=5), dict(y=None), dict(y=P + 1), dict(ldy=9),
        dict(lora=None), dict(lora=adapters(n_adapters=0)), dict(lora=adapters(n_adapters=1025)),
        dict(lora=adapters(rank=0)), dict(lora=adapters(rank=4)), dict(lora=adapters(rank=12)),
        dict(lora=adapters(rank=136)), dict(lora=adapters(rank=-8)), dict(lora=adapters(a=None)),
        dict(lora=adapters(b=None)), dict(lora=adapters(a=P + 8)), dict(lora=adapters(b=P + 2)),
        dict(lora=adapters(scale=P + 2)), dict(x=None), dict(x=P + 1), dict(ldx=63), dict(ids=None),
        dict(ids=P + 2), dict(offs=None), dict(offs=P + 1), dict(perm=None), dict(perm=P + 3)])
    need = B.coli_lora_workspace_bytes(4, 16)
    refuse("coli_gemm_q8_lora", good, [dict(ws_=None), dict(ws_=P + 128), dict(wsn=need - 1), dict(wsn=0)],
           B.COLI_ERR_WORKSPACE)
    refuse("coli_gemm_q8_lora", good, [dict(T=1 << 20, N=1 << 30, ldy=1 << 30, wsn=1 << 40),
                                       dict(T=1 << 16, K=1 << 16, ldx=1 << 16, N=6144, ldy=6144, wsn=1 << 40)], UNSUPPORTED)
    no_device_or_empty("coli_gemm_q8_lora", dict(good, wsn=need), dict(T=0, q=None, s=None, y=None, ws_=None, x=None))


def test_workspace_bytes():
    for bad in ((-1, 16), ((1 << 20) + 1, 16), (4, 0), (4, 12), (4, 136), (4, -8)):
        assert B.coli_lora_workspace_bytes(*bad) == 0
    last = 0
    for t in (0, 1, 2, 16, 61, 1024, 1171, 8192, 8193, 1 << 20):  # a larger batch never needs less
        n = B.coli_lora_workspace_bytes(t, 64)
        assert n % 256 == 0 and n >= max(t, 1) * 64 * 4 and n >= last
        last = n
    with pytest.raises(ValueError, match="no workspace"):
        B.lora_workspace(4, 12, device="cpu")


def test_binding_refuses_host_tensors_and_shapes():
    z = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        B.Lora(z(2, 8, 64), z(2, 10, 8))
    with pytest.raises(ValueError, match=r"must be \[2, N, 8\]"):
        B.Lora(z(2, 8, 64), z(2, 10, 16))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        B.Lora(z(2, 8, 64).double(), z(2, 10, 8).double())
