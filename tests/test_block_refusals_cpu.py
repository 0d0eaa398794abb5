"""A block refuses a call before it launches anything (no GPU: a launch would fail)."""
import types

import pytest
import torch

BF = torch.bfloat16


def _block(gate=None):
    from routing_dispatch_expert_moe_b200.layer import MoEBlock
    layer = types.SimpleNamespace(combine_mode="rows", T_max=12, d=64, device="cpu", dtype=BF, rows_dtype=BF)
    return MoEBlock(layer, torch.ones(64), gate=gate)


@pytest.mark.parametrize("shape,dtype,n,msg", [
    ((13, 64), BF, None, "exceeds"), ((4, 32), BF, None, "residual"), ((4, 64), torch.float32, None, "residual"),
    ((4, 64, 1), BF, None, "residual"), ((4, 64), BF, (3, 64), "n must"), ((4, 64), BF, (4, 32), "n must"),
    ((5, 64), BF, None, "do not divide"), ((1, 64), BF, (1, 64), "do not divide"),
])
def test_forward(shape, dtype, n, msg):
    blk = _block(torch.ones(2, 64))
    with pytest.raises(ValueError, match=msg):
        blk.forward(torch.zeros(shape, dtype=dtype), None if n is None else torch.zeros(n, dtype=BF))


@pytest.mark.parametrize("gate", [(64,), (0, 64), (2, 32)])
def test_gate(gate):
    with pytest.raises(ValueError, match="gate must be"):
        _block(torch.ones(gate))
