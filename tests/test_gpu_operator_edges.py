"""Calls of the routing gradient, the 8-bit products and the block norms at their edges, against
the float64 reference."""
import numpy as np
import pytest
import torch

from oracle import block_ops as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _M():
    from routing_dispatch_expert_moe_b200 import moe as M
    return M


def _ok():
    torch.cuda.synchronize()
    assert _M().moe_get_device_error() == 0


# ---------------------------------------------------------------- the norms' gradients
@pytest.mark.parametrize("d", [1, 4, 7])
def test_norm_gradients_refuse_narrow_rows(d):
    """Narrower than one vector of eight: refused by the call, after its size query answered."""
    M = _M()
    x = torch.ones((4, d), device="cuda")
    with pytest.raises(M.MoEError):
        M.moe_block_norm_backward(x, None, x)
    with pytest.raises(M.MoEError):
        M.moe_block_norm_backward(x, x, x, pre_weight=torch.ones(d, device="cuda"))
    _ok()


def test_column_sums_of_calls_that_share_a_workspace():
    """Two calls take turns on one workspace, with no wait in between: the second launch of each
    starts while its first one ends, and has to see that one's sums and not the other call's."""
    M = _M()
    T, d = 700, 264
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    calls = []
    for i in range(2):
        calls.append(dict(d_x=rnd(T, d), d_n=rnd(T, d), x_out=rnd(T, d), y=rnd(T, d), post_weight=rnd(d),
                          gate=rnd(1 if i else 70, d), pre_weight=rnd(d)))
    want = [M.moe_block_norm_backward(**c) for c in calls]
    _ok()
    ws = torch.empty(int(M.lib().moe_block_norm_backward_workspace_bytes(T, d)), dtype=torch.uint8, device="cuda")
    got = [M.moe_block_norm_backward(**calls[i % 2], workspace=ws) for i in range(60)]
    _ok()
    for i, v in enumerate(got):
        for key, t in v.items():
            assert torch.equal(t, want[i % 2][key]), (i, key)
