"""Host-side checks of the grouped routing, its gradient, the 8-bit GEMMs and the block norms (no
GPU): every case is refused, or has nothing to do, before any launch; the made-up pointers are
never read."""
import ctypes
import types

import pytest
import torch

P, ODD, NUL = ctypes.c_void_p(4096), ctypes.c_void_p(4100), None
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from routing_dispatch_expert_moe_b200 import build
    build.build()
    from routing_dispatch_expert_moe_b200 import moe
    return moe.lib()


def _call(f, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


def test_route_grouped(L):
    base = dict(l=P, bias=NUL, T=4, E=64, k=8, G=8, kept=4, gs=1, score=1, renorm=1, scale=1.0, idx=P, gate=P, s=NUL)
    f = lambda **kw: _call(L.moe_route_grouped, base, kw)
    for bad in (dict(l=NUL), dict(idx=NUL), dict(gate=NUL), dict(T=-1), dict(k=0), dict(G=0), dict(kept=0),
                dict(kept=9), dict(G=7), dict(k=33, kept=4), dict(gs=2), dict(gs=-1), dict(score=3), dict(renorm=2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(E=0)):
        assert f(**bad) == INVALID, bad
    assert f(E=2048, G=8, kept=8) == UNSUPPORTED
    assert f(E=1024, G=64, kept=64) == UNSUPPORTED                       # more groups than lanes
    assert f(E=1024, G=8, kept=8, k=33) == UNSUPPORTED
    assert f(T=1 << 24) == UNSUPPORTED
    assert f(T=0, l=NUL, idx=NUL, gate=NUL) == 0


def test_route_backward(L):
    base = dict(l=P, idx=P, u=P, T=4, E=64, k=8, score=0, renorm=1, scale=1.0, load=P, aux=0.1, z=0.1, d=P, s=NUL)
    f = lambda **kw: _call(L.moe_route_backward, base, kw)
    for bad in (dict(l=NUL), dict(d=NUL), dict(idx=NUL), dict(u=NUL), dict(load=NUL), dict(T=-1), dict(k=0),
                dict(k=65), dict(score=-1), dict(renorm=5), dict(scale=float("inf")), dict(aux=float("nan")),
                dict(z=float("inf"))):
        assert f(**bad) == INVALID, bad
    assert f(E=1025) == UNSUPPORTED and f(k=33) == UNSUPPORTED
    assert f(T=0, l=NUL, d=NUL) == 0
    assert f(T=0, idx=NUL, u=NUL, k=0) == 0                              # the losses alone: k is ignored


def test_quantize_rows(L):
    base = dict(x=P, dt=0, rows=4, cols=64, row_of=NUL, k=0, rows_max=0, q=P, scale=P, s=NUL)
    f = lambda **kw: _call(L.moe_quantize_rows_i8, base, kw)
    for bad in (dict(x=NUL), dict(q=NUL), dict(scale=NUL), dict(rows=-1), dict(cols=0), dict(dt=2),
                dict(row_of=P, k=0, rows_max=4), dict(row_of=P, k=2, rows_max=-1),
                dict(row_of=P, k=2, rows_max=4, q=NUL)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(cols=24), dict(cols=16400), dict(rows=1 << 31), dict(row_of=P, k=33, rows_max=4), dict(x=ODD),
                dict(q=ODD)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(rows=0, x=NUL, q=NUL, scale=NUL) == 0


def test_expert_gemms_i8(L):
    gu = dict(x=P, xs=P, off=P, E=8, d=128, F=128, rows=16, W=P, ws=P, h=P, s=NUL)
    ga = dict(x=P, xs=P, T=4, tok=P, off=P, E=8, d=128, F=128, rows=16, W=P, ws=P, h=P, s=NUL)
    dn = dict(x=P, xs=P, off=P, E=8, d=128, F=128, rows=16, W=P, ws=P, gate=NUL, dt=0, h=P, s=NUL)
    for f, base in ((L.moe_expert_gate_up_i8, gu), (L.moe_expert_gate_up_gather_i8, ga), (L.moe_expert_down_i8, dn)):
        for bad in (dict(x=NUL), dict(xs=NUL), dict(off=NUL), dict(W=NUL), dict(ws=NUL), dict(h=NUL), dict(E=0),
                    dict(d=0), dict(F=-16), dict(rows=-1)):
            assert _call(f, base, bad) == INVALID, (f, bad)
        for bad in (dict(E=1025), dict(d=136), dict(F=120), dict(d=112), dict(F=112), dict(d=16400), dict(F=16400),
                    dict(rows=1 << 31), dict(x=ODD), dict(W=ODD), dict(ws=ODD), dict(h=ODD)):
            assert _call(f, base, bad) == UNSUPPORTED, (f, bad)
        assert _call(f, base, dict(rows=0, x=NUL, xs=NUL, h=NUL)) == 0
    assert _call(L.moe_expert_gate_up_gather_i8, ga, dict(tok=NUL)) == INVALID
    assert _call(L.moe_expert_gate_up_gather_i8, ga, dict(T=-1)) == INVALID
    assert _call(L.moe_expert_gate_up_gather_i8, ga, dict(T=1 << 24)) == UNSUPPORTED
    assert _call(L.moe_expert_gate_up_gather_i8, ga, dict(T=0, x=NUL, tok=NUL)) == 0
    assert _call(L.moe_expert_down_i8, dn, dict(dt=3)) == INVALID


def test_block_norm(L):
    nm = dict(r=P, rdt=0, y=P, ydt=0, post=P, gate=P, G=2, alpha=1.0, pre=P, eps=1e-6, T=4, d=64, x=P, n=P, ndt=0, s=NUL)
    cb = dict(r=P, rdt=0, y=P, ydt=0, row_of=P, tg=NUL, sh=NUL, k=2, rows_max=8, post=P, gate=P, G=2, alpha=1.0, pre=P,
              eps=1e-6, T=4, d=64, y_out=NUL, x=P, n=P, ndt=0, s=NUL)
    for f, base in ((L.moe_block_norm, nm), (L.moe_combine_norm, cb)):
        for bad in (dict(r=NUL), dict(y=NUL), dict(n=NUL), dict(pre=NUL), dict(x=NUL, n=NUL, pre=NUL), dict(G=0),
                    dict(G=3), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")),
                    dict(T=-1), dict(d=0), dict(rdt=2), dict(ydt=-1), dict(ndt=7)):
            assert _call(f, base, bad) == INVALID, (f, bad)
        for bad in (dict(d=60), dict(d=8200), dict(T=1 << 24), dict(r=ODD), dict(y=ODD), dict(post=ODD), dict(gate=ODD),
                    dict(pre=ODD), dict(x=ODD), dict(n=ODD)):
            assert _call(f, base, bad) == UNSUPPORTED, (f, bad)
        assert _call(f, base, dict(T=0, r=NUL)) == 0
    for bad in (dict(row_of=NUL), dict(k=0), dict(rows_max=-1)):
        assert _call(L.moe_combine_norm, cb, bad) == INVALID, bad
    assert _call(L.moe_combine_norm, cb, dict(k=33)) == UNSUPPORTED
    assert _call(L.moe_combine_norm, cb, dict(sh=ODD)) == UNSUPPORTED


def test_block_norm_backward(L):
    need = L.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need > 0 and L.moe_block_norm_backward_workspace_bytes(0, 64) == 0
    base = dict(dx=P, dn=P, x=P, y=P, rdt=0, ndt=0, ydt=0, post=P, gate=P, G=2, alpha=1.0, pre=P, eps=1e-6, T=4, d=64,
                dr=P, dy=P, dpost=P, dgate=P, dpre=P, ws=P, wsb=need, s=NUL)
    f = lambda **kw: _call(L.moe_block_norm_backward, base, kw)
    for bad in (dict(dr=NUL), dict(dy=NUL), dict(y=NUL), dict(post=NUL), dict(gate=NUL), dict(pre=NUL), dict(dn=NUL),
                dict(x=NUL), dict(dx=NUL, dn=NUL, pre=NUL, dpre=NUL), dict(G=3), dict(eps=0.0), dict(T=-4), dict(rdt=9)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(d=8200), dict(dx=ODD), dict(dn=ODD), dict(x=ODD), dict(dr=ODD), dict(dy=ODD), dict(dgate=ODD),
                dict(ws=ODD)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(ws=NUL) == WORKSPACE and f(wsb=need - 1) == WORKSPACE


@pytest.mark.parametrize("kw,msg", [
    (dict(W_gu_i8=True), "8-bit experts need both"),
    (dict(W_gu_i8=True, W_dn_i8=True, combine="fused"), "8-bit experts need both"),
    (dict(no_weights=True), "W_gu and W_dn are needed"),
    (dict(n_groups=4, routing="uniform"), "groups of experts"),
])
def test_layer_refuses_before_allocating(kw, msg):
    from routing_dispatch_expert_moe_b200.layer import MoELayer, MoEWeights
    w = MoEWeights(Wg=torch.zeros(128, 8), W_gu=torch.zeros(8, 256, 128, dtype=torch.bfloat16),
                   W_dn=torch.zeros(8, 128, 128, dtype=torch.bfloat16))
    if kw.pop("no_weights", False):
        w.W_gu = None
    for name in ("W_gu_i8", "W_dn_i8"):
        if kw.pop(name, False):
            setattr(w, name, (torch.zeros(8, 256, 128, dtype=torch.int8), torch.zeros(8, 256)))
    with pytest.raises(ValueError, match=msg):
        MoELayer(w, 2, 16, **kw)


def test_block_refuses_a_fused_combine():
    from routing_dispatch_expert_moe_b200.layer import MoEBlock
    with pytest.raises(ValueError, match="rows"):
        MoEBlock(types.SimpleNamespace(combine_mode="fused"), torch.ones(8))
    with pytest.raises(ValueError, match="pre_weight"):
        MoEBlock(types.SimpleNamespace(combine_mode="rows"), None)


def test_bindings_refuse_wrong_choices_before_a_launch():
    from routing_dispatch_expert_moe_b200 import moe as M
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.moe_route_grouped(torch.zeros(2, 8), 2, 2, 1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.moe_block_norm(torch.zeros(2, 8), pre_weight=torch.ones(8))
