"""Size queries of the block norms' gradients (no GPU): every size is answered, the ones that the
call refuses with zero bytes."""
import ctypes

import pytest

P, NUL = ctypes.c_void_p(4096), None
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def L():
    from routing_dispatch_expert_moe_b200 import build
    build.build()
    from routing_dispatch_expert_moe_b200 import moe
    return moe.lib()


@pytest.mark.parametrize("d", [1, 4, 7, 12, 8200])
@pytest.mark.parametrize("T", [1, 4, 5000])
def test_refused_widths_need_no_workspace(L, T, d):
    assert L.moe_block_norm_backward_workspace_bytes(T, d) == 0
    status = L.moe_block_norm_backward(P, P, P, P, 0, 0, 0, P, P, 1, 1.0, P, 1e-6, T, d, P, P, P, P, P, NUL, 0, NUL)
    assert status == UNSUPPORTED


def test_sizes_at_the_limits(L):
    f = L.moe_block_norm_backward_workspace_bytes
    assert f(1 << 24, 64) == 0 and f(-1, 64) == 0 and f(4, -8) == 0 and f(4, 0) == 0
    for T in (1, 7, 5000, (1 << 24) - 1):
        for d in (8, 16, 256, 264, 2048, 8192):
            assert f(T, d) > 0 and f(T, d) % (16 * d) == 0               # four fp32 rows a block


def test_gate_up_i8_orientation_query(L, monkeypatch):
    """Weight-major tiles below 192 rows an expert on average; the override variable wins, as in the
    GEMMs and in the layer's choice of its dispatch."""
    from routing_dispatch_expert_moe_b200 import moe as M
    monkeypatch.delenv("MOE_B200_EXPERT_TILES", raising=False)
    f = M.moe_gate_up_i8_weight_major
    assert f(191, 1) and not f(192, 1) and f(0, 8) and f(192 * 64 - 1, 64) and not f(192 * 64, 64)
    for query in (f, M.moe_gate_up_weight_major):
        for bad in ((-1, 8), (10, 0)):
            with pytest.raises(M.MoEError):
                query(*bad)
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", "tokens")
    assert not f(1, 1)
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", "weights")
    assert f(1 << 20, 1)
