"""Refusals of the 8-bit operators and the scored router, on the host: every
bad argument is refused before a device is touched."""
import ctypes

import pytest
import torch

from quantized_moe_coli_amd import binding as B

INVALID, UNSUPPORTED = B.COLI_ERR_INVALID_ARG, B.COLI_ERR_UNSUPPORTED
P = 1 << 20  # an aligned address, never followed


def refuse(name, good, bad, code=INVALID):
    """The call with arguments ``good`` changed by each of ``bad``."""
    fn = getattr(B.lib(), name)
    for change in bad:
        args = dict(good)
        args.update(change)
        assert fn(*args.values()) == code, (name, change)


def no_device_or_empty(name, good, empty):
    fn = getattr(B.lib(), name)
    if not torch.cuda.is_available():
        assert fn(*good.values()) == B.COLI_ERR_DEVICE
    args = dict(good)
    args.update(empty)
    assert fn(*args.values()) == B.COLI_OK


def test_quant_act_token():
    good = dict(dt=1, x=P, ld=64, T=2, n=64, q=P, s=P, st=None)
    refuse("coli_quant_act_token", good, [
        dict(dt=3), dict(dt=-1), dict(x=None), dict(x=P + 1), dict(dt=0, x=P + 2), dict(ld=63), dict(ld=-64),
        dict(T=-1), dict(T=(1 << 20) + 1), dict(n=0), dict(n=48), dict(n=-32), dict(n=131072, ld=1 << 20),
        dict(q=None), dict(q=P + 8), dict(s=None), dict(s=P + 2)])
    no_device_or_empty("coli_quant_act_token", good, dict(T=0, x=None, q=None, s=None))


def test_swiglu_quant_token():
    good = dict(dt=1, g=P, ldg=64, u=P, ldu=64, T=2, n=64, q=P, s=P, st=None)
    refuse("coli_swiglu_quant_token", good, [
        dict(dt=3), dict(g=None), dict(u=None), dict(g=P + 1), dict(u=P + 1), dict(ldg=60), dict(ldu=63),
        dict(T=-1), dict(T=(1 << 25) + 1), dict(n=0), dict(n=33), dict(q=None), dict(q=P + 4), dict(s=None)])
    no_device_or_empty("coli_swiglu_quant_token", good, dict(T=0))


def test_gemm_q8():
    good = dict(q=P, s=P, T=4, w=P, ws=P, N=10, K=64, bias=None, dt=1, y=P, ldy=10, st=None)
    refuse("coli_gemm_q8", good, [
        dict(q=None), dict(q=P + 8), dict(s=None), dict(s=P + 1), dict(T=-1), dict(T=(1 << 20) + 1),
        dict(w=None), dict(w=P + 4), dict(ws=None), dict(ws=P + 2), dict(N=0), dict(N=-3), dict(K=0),
        dict(K=40), dict(K=131072), dict(bias=P + 2), dict(dt=5), dict(y=None), dict(y=P + 1), dict(ldy=9)])
    refuse("coli_gemm_q8", good, [dict(T=1 << 20, N=1 << 30, ldy=1 << 30)], UNSUPPORTED)
    no_device_or_empty("coli_gemm_q8", good, dict(T=0, q=None, s=None, y=None))


def test_gemm_q8_grouped():
    good = dict(q=P, s=P, rows=4, w=P, ws=P, E=4, N=10, K=64, offs=P, perm=P, Pn=8, fan=2, dt=1, y=P,
                ldy=10, st=None)
    refuse("coli_gemm_q8_grouped", good, [
        dict(q=None), dict(q=P + 8), dict(s=None), dict(rows=-1), dict(rows=0), dict(w=None), dict(w=P + 1),
        dict(ws=None), dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(K=48), dict(K=131072),
        dict(offs=None), dict(offs=P + 2), dict(perm=None), dict(perm=P + 1), dict(Pn=-1),
        dict(Pn=(1 << 25) + 1), dict(fan=0), dict(fan=-1), dict(dt=7), dict(y=None), dict(ldy=9)])
    refuse("coli_gemm_q8_grouped", good, [dict(Pn=1 << 25, N=1 << 30, ldy=1 << 30),
                                          dict(rows=1 << 16, K=1 << 16)], UNSUPPORTED)
    no_device_or_empty("coli_gemm_q8_grouped", good, dict(Pn=0, rows=0))


def test_moe_combine():
    good = dict(dt=2, o=P, ldo=8, idx=None, w=P, T=3, k=2, H=8, add=None, lda=0, y=P, ldy=8, st=None)
    refuse("coli_moe_combine", good, [
        dict(dt=3), dict(o=None), dict(o=P + 1), dict(ldo=7), dict(idx=P + 2), dict(w=None), dict(w=P + 2),
        dict(T=-1), dict(T=(1 << 20) + 1), dict(k=0), dict(k=33), dict(H=0), dict(H=131073, ldo=1 << 18, ldy=1 << 18),
        dict(add=P, lda=7), dict(add=P + 1, lda=8), dict(y=None), dict(y=P + 1), dict(ldy=7)])
    no_device_or_empty("coli_moe_combine", good, dict(T=0))


def test_moe_route_scored():
    def cfg(**kw):
        c = dict(n_experts=16, top_k=2, n_group=4, topk_group=2)
        c.update(kw)
        return ctypes.pointer(B.score_cfg(**c))

    good = dict(cfg=cfg(), dt=0, lg=P, ld=16, bias=None, T=2, idx=P, w=P, st=None)
    refuse("coli_moe_route_scored", good, [
        dict(cfg=None), dict(cfg=cfg(n_experts=0)), dict(cfg=cfg(n_experts=1028)), dict(cfg=cfg(n_group=3)),
        dict(cfg=cfg(topk_group=5)), dict(cfg=cfg(topk_group=0)), dict(cfg=cfg(top_k=0)),
        dict(cfg=cfg(top_k=9)), dict(cfg=cfg(score=2)), dict(cfg=cfg(score=-1)), dict(cfg=cfg(group_score=2)),
        dict(dt=3), dict(lg=None), dict(lg=P + 2), dict(ld=15), dict(bias=P + 2), dict(T=-1),
        dict(T=(1 << 20) + 1), dict(idx=None), dict(idx=P + 2), dict(w=None), dict(w=P + 1)])
    no_device_or_empty("coli_moe_route_scored", good, dict(T=0, lg=None, idx=None, w=None))


def test_binding_refuses_host_tensors_shapes_and_types():
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d)  # noqa: E731
    q, s = z(2, 64, d=torch.int8), z(2)
    with pytest.raises(ValueError, match="device tensor"):
        B.coli_quant_act_token(z(2, 64), q, s)
    with pytest.raises(ValueError, match="device tensor"):
        B.coli_gemm_q8(q, s, z(4, 64, d=torch.uint8), z(4), z(2, 4))
    with pytest.raises(ValueError, match="device tensor"):
        B.coli_moe_route_scored(B.score_cfg(8, 2), z(2, 8), None, z(2, 2, d=torch.int32), z(2, 2))
    # the helpers that every call uses (host tensors lie on "device" -1)
    with pytest.raises(ValueError, match=r"must be \[2, 8\]"):
        B._rowed(z(2, 9), 2, 8, torch.float32, -1, "x")
    with pytest.raises(ValueError, match="must be torch.float32"):
        B._rowed(z(2, 8, d=torch.bfloat16), 2, 8, torch.float32, -1, "x")
    with pytest.raises(ValueError, match="consecutive"):
        B._rowed(z(8, 2).t(), 2, 8, torch.float32, -1, "x")
    with pytest.raises(ValueError, match="consecutive"):
        B._rowed(z(1, 8).expand(2, 8), 2, 8, torch.float32, -1, "x")
    with pytest.raises(ValueError, match="current device"):
        B._rowed(z(2, 8), 2, 8, torch.float32, 0, "x")
    assert B._rowed(z(2, 12)[:, :8], 2, 8, torch.float32, -1, "x")[1] == 12
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        B._float_type(z(2, d=torch.float64), "x")
