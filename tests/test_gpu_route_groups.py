"""Group-limited routing and the routing's gradient on the GPU against the float64 reference.

Bars.  Indices: equal wherever the reference's deciding distance exceeds 1e-13 of the row's
largest key, score or bias (both sides take keys in fp64: an exponential, a logarithm, a square
root, a quotient and two sums, each a step or two of 2^-52, the softmax's sum of up to 1024 terms
40 more: under 1e-14), and everywhere on logits whose ties are exact.  Gates: taken in fp64 and rounded
once (2^-24), except the full softmax probability, whose sum is fp32: at most 64 + 5 additions,
2 steps an exponential and half a step of each difference (at most 32 here): 120 * 2^-24.
Gradients: M = scale max|u| + aux E / T max f + 2 z / T |lse| bounds every factor that multiplies
a derivative (all at most 1) up to the difference with its mean, hence twice; sums have at most
32 + 5 terms in a row and every product a dozen roundings: 128 * 2^-24 * 2 M.
"""
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


def _M():
    from routing_dispatch_expert_moe_b200 import moe as M
    return M


def _ok():
    torch.cuda.synchronize()
    assert _M().moe_get_device_error() == 0


def _check(l, k, G, kept, gs, score, renorm, scale, bias, everywhere=False):
    M = _M()
    idx, gate = M.moe_route_grouped(torch.from_numpy(l).cuda(), k, G, kept, gs, score, renorm, scale,
                                    None if bias is None else torch.from_numpy(bias).cuda())
    _ok()
    wi, wg, margin = B.route_grouped(l, k, G, kept, gs, score, renorm, scale, bias)
    sure = np.ones(len(l), bool) if everywhere else margin > 1e-13
    assert sure.mean() > 0.9
    idx, gate = idx.cpu().numpy(), gate.cpu().numpy().astype(np.float64)
    assert np.array_equal(idx[sure], wi[sure])
    tol = 120 * U if score == "softmax" and not renorm else 2 * U
    assert (np.abs(gate - wg)[sure] <= tol * np.abs(wg[sure]) + 1e-44).all()


SHAPES = [  # T, E, k, groups, kept
    (1, 1, 1, 1, 1), (1, 2, 2, 2, 2), (3, 8, 3, 1, 1), (5, 64, 8, 8, 4), (33, 256, 8, 8, 4), (7, 37, 5, 1, 1),
    (9, 60, 7, 3, 2), (4, 90, 32, 9, 5), (6, 896, 16, 16, 4), (5, 1008, 16, 28, 6), (3, 1024, 32, 32, 8),
    (2, 1020, 12, 17, 3), (3, 1024, 32, 1, 1), (4, 620, 20, 31, 31), (300, 20, 4, 4, 1), (5, 33, 3, 3, 3),
]


@pytest.mark.parametrize("T,E,k,G,kept", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_selection_and_gates(T, E, k, G, kept, score, with_bias):
    rng = np.random.default_rng([T, E, k, G])
    l = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32) if with_bias else None
    for gs in ("max", "top2"):
        for renorm in (True, False):
            _check(l, k, G, kept, gs, score, renorm, 2.5 if renorm else 1.0, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
def test_exact_ties_take_the_lower_index(score):
    rng = np.random.default_rng(4)
    l = rng.integers(-2, 3, (64, 64)).astype(np.float32)
    _check(l, 8, 8, 3, "max", score, True, 1.0, None, everywhere=True)
    _check(l, 8, 8, 3, "top2", score, True, 1.0, None, everywhere=True)
    _check(l, 8, 8, 3, "top2", score, True, 1.0, np.zeros(64, np.float32), everywhere=True)
    same = np.zeros((3, 896), np.float32)                    # a router at its zero start
    _check(same, 16, 16, 4, "top2", score, True, 1.0, np.zeros(896, np.float32), everywhere=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_experts_and_rows(score, renorm):
    rng = np.random.default_rng(8)
    l = rng.standard_normal((12, 64)).astype(np.float32)
    l[:, 5] = -np.inf
    l[1, 8:16] = -np.inf                                     # a whole group
    l[2] = -np.inf                                           # a whole row
    l[3, 3:] = -np.inf                                       # fewer than k left
    l[4, ::2] = np.nan
    l[5, 7] = np.inf
    l[6] = np.finfo(np.float32).min                          # the type's lowest value is a number
    l[7, :32] = np.finfo(np.float32).min
    bias = np.abs(rng.standard_normal(64).astype(np.float32))
    for b in (None, bias):
        for gs in ("max", "top2"):
            _check(l, 6, 8, 4, gs, score, renorm, 1.0, b, everywhere=b is None)


def test_keys_closer_than_fp32_holds():
    """Scores that fp32 cannot tell apart, decided by fp64."""
    rng = np.random.default_rng(2)
    l = (8.0 + rng.standard_normal((50, 64)) * 1e-3).astype(np.float32)     # sigmoid within 1e-6 of 1
    bias = (rng.standard_normal(64) * 1e-7).astype(np.float32)
    _check(l, 8, 8, 4, "top2", "sigmoid", True, 1.0, bias)
    _check(l, 8, 8, 4, "top2", "sqrt_softplus", True, 1.0, bias)
    _check((l - 8.0) * 1e-3, 8, 8, 4, "top2", "softmax", False, 1.0, bias)
    _check(l - 60.0, 8, 8, 4, "top2", "sigmoid", True, 1.0, (bias * 1e-18).astype(np.float32))


def test_grouped_matches_moe_route_with_one_group():
    M = _M()
    l = torch.randn(64, 128, device="cuda")
    x = torch.eye(128, device="cuda")[:64].contiguous()
    W = torch.zeros(128, 128, device="cuda")
    W[:64] = l
    lg, idx, gate = M.moe_route(x, W, 8, "sigmoid", True, 2.0)
    i2, g2 = M.moe_route_grouped(lg, 8, 1, 1, "max", "sigmoid", True, 2.0)
    _ok()
    assert torch.equal(idx, i2)
    assert torch.allclose(gate, g2, rtol=1e-6, atol=0)


def test_unaligned_rows_and_empty_batch():
    M = _M()
    big = torch.randn(33 * 64 + 1, device="cuda")
    l = big[1:].view(33, 64)                                 # four bytes off a 16-byte boundary
    a = M.moe_route_grouped(l, 4, 4, 2)
    b = M.moe_route_grouped(l.clone(), 4, 4, 2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    i, g = M.moe_route_grouped(torch.empty(0, 64, device="cuda"), 4, 4, 2)
    assert i.shape == (0, 4) and g.shape == (0, 4)
    u = torch.randn(33, 4, device="cuda")
    # rows off the boundary are read one logit at a time, which sums a lane's logits in another
    # order: each side is within the gradient's bar, so they are within twice that
    d0, d1 = (M.moe_route_backward(v, a[0], u, z_coef=0.1) for v in (l, l.clone()))
    off = float((d0 - d1).abs().max())
    assert off <= 2 * 128 * U * 2 * (float(u.abs().max()) + 0.2 / 33 * (float(l.max()) + 8.0))
    _ok()


# ---------------------------------------------------------------- the gradient
def _grad(l, idx, u, score, renorm, scale, load, aux, z):
    M = _M()
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()
    got = M.moe_route_backward(c(l), c(idx), c(u), score, renorm, scale, c(load), aux, z).cpu().numpy().astype(np.float64)
    _ok()
    T, E = l.shape
    want = B.route_backward(l, idx, u, score, renorm, scale, load, aux, z)
    m = np.where(np.isfinite(l), l, -1e30).max(1)
    M_ = 0.0 if u is None else abs(scale) * np.abs(u).max()
    M_ += abs(aux) * E / T * (0.0 if load is None else load.max()) + 2 * abs(z) / T * (np.abs(m).max() + 8.0)
    assert np.isfinite(got).all()
    assert np.abs(got - want).max() <= 128 * U * 2 * M_
    return got, want


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (17, 64, 8), (5, 37, 5), (4, 896, 16), (2, 1024, 32),
                                   (3, 1023, 16), (9, 100, 7), (2, 301, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient(T, E, k, score, renorm):
    rng = np.random.default_rng([T, E, k])
    l = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    idx = np.argsort(-l, 1)[:, :k].astype(np.int32)
    u = rng.standard_normal((T, k)).astype(np.float32)
    load = rng.random(E).astype(np.float32)
    _grad(l, idx, u, score, renorm, 1.5, None, 0.0, 0.0)
    _grad(l, idx, u, score, renorm, 1.5, load, 0.3, 0.2)
    _grad(l, None, None, score, renorm, 1.0, load, 0.3, 0.0)
    _grad(l, None, None, score, renorm, 1.0, None, 0.0, 0.2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_masked_and_repeated(score, renorm):
    rng = np.random.default_rng(6)
    l = rng.standard_normal((8, 32)).astype(np.float32)
    idx = np.stack([rng.permutation(32)[:4] for _ in range(8)]).astype(np.int32)
    l[0, idx[0, 1]] = -np.inf
    l[1] = -np.inf
    l[2, 5] = np.nan
    l[3] -= 150.0                                            # every sigmoid underflows in fp32
    idx[4, 2] = idx[4, 0]                                    # an expert named twice
    u = rng.standard_normal((8, 4)).astype(np.float32)
    if score != "softmax" and renorm:
        l[3] += 100.0                                        # fp32 holds the scores it divides by
    load = rng.random(32).astype(np.float32)
    got, _ = _grad(l, idx, u, score, renorm, 1.0, load if score == "softmax" else None,
                   0.2 if score == "softmax" else 0.0, 0.1)
    assert (got[1] == 0).all() and got[0, idx[0, 1]] == 0 and got[2, 5] == 0


def test_gradient_against_differences_of_the_gates():
    M = _M()
    torch.manual_seed(0)
    l = torch.randn(6, 16, device="cuda")
    idx, _ = M.moe_route_grouped(l, 4, 4, 2, score="sigmoid")
    u = torch.randn(6, 4, device="cuda")
    got = M.moe_route_backward(l, idx, u, "sigmoid").double().cpu().numpy()
    ln, i = l.double().cpu().numpy(), idx.long().cpu().numpy()
    h = 1e-5
    for t, e in [(0, int(i[0, 0])), (1, int(i[1, 2])), (5, int(i[5, 3]))]:
        a, b = ln.copy(), ln.copy()
        a[t, e] += h
        b[t, e] -= h
        args = (i, u.double().cpu().numpy(), "sigmoid", True, 1.0, None, 0.0, 0.0)
        d = (B.routing_loss(a, *args) - B.routing_loss(b, *args)) / (2 * h)
        assert abs(d - got[t, e]) <= 1e-8 + 256 * U * float(u.abs().max())


def test_a_bad_expert_is_recorded_and_left_out():
    M = _M()
    l = torch.randn(4, 16, device="cuda")
    idx = torch.tensor([[0, 1], [2, 99], [-3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    u = torch.ones(4, 2, device="cuda")
    d = M.moe_route_backward(l, idx, u, "sigmoid", False)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 1
    want = torch.sigmoid(l) * torch.sigmoid(-l)
    for t, keep in enumerate([[0, 1], [2], [4], [5, 6]]):
        row = torch.zeros(16, device="cuda")
        row[keep] = want[t, keep]
        assert torch.allclose(d[t], row, rtol=1e-6, atol=1e-9)


def test_other_stream_and_graph_replay():
    M = _M()
    l = torch.randn(65, 64, device="cuda")
    want = M.moe_route_grouped(l, 8, 8, 4)
    u = torch.randn(65, 8, device="cuda")
    wantd = M.moe_route_backward(l, want[0], u, "sigmoid")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = M.moe_route_grouped(l, 8, 8, 4, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st = torch.zeros_like(l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i, gate = M.moe_route_grouped(st, 8, 8, 4)
        d = M.moe_route_backward(st, i, u, "sigmoid")
    st.copy_(l)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(i, want[0]) and torch.equal(gate, want[1]) and torch.equal(d, wantd)
    _ok()


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [32, 30])
def test_a_masked_slots_upstream_gradient_is_not_used(score, renorm, E):
    rng = np.random.default_rng(8)
    l = rng.standard_normal((6, E)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:4] for _ in range(6)]).astype(np.int32)
    u = rng.standard_normal((6, 4)).astype(np.float32)
    l[0, idx[0, 1]] = -np.inf
    l[3, idx[3, 3]] = np.nan
    u[0, 1] = u[3, 3] = 0.0
    _grad(l, idx, u, score, renorm, 1.0, None, 0.0, 0.1)      # against the formula
    M = _M()
    on = lambda a: torch.from_numpy(a).cuda()
    d0 = M.moe_route_backward(on(l), on(idx), on(u), score, renorm, 1.0, None, 0.0, 0.1)
    u[0, 1], u[3, 3] = np.nan, np.inf
    d1 = M.moe_route_backward(on(l), on(idx), on(u), score, renorm, 1.0, None, 0.0, 0.1)
    _ok()
    assert torch.isfinite(d0).all() and torch.equal(d0, d1)


@pytest.mark.parametrize("E", [32, 30])
def test_a_repeated_expert_adds_in_slot_order(E):
    """scores without renormalising: a slot's term is s'(l) u; at l = 0 the sigmoid's s' is exactly 1/4,
    so the sum in slot order is known to the bit: (2^24 + 1) - 2^24 rounds to 0, any order that takes
    2^24 and -2^24 together gives 1."""
    M = _M()
    l = torch.zeros((5, E), device="cuda")
    idx = torch.tensor([[3, 7, 3, 3]], dtype=torch.int32, device="cuda").repeat(5, 1)
    u = 4.0 * torch.tensor([[2.0 ** 24, 5.0, 1.0, -2.0 ** 24]], device="cuda").repeat(5, 1)
    d = M.moe_route_backward(l, idx, u, "sigmoid", False, 1.0)
    _ok()
    want = torch.zeros((5, E))
    want[:, 7] = 5.0
    assert torch.equal(d.cpu(), want)


def test_refused_sizes():
    M = _M()
    l = torch.zeros((4, 32), device="cuda")
    for k in (0, -1):
        with pytest.raises(ValueError):
            M.moe_route_grouped(l, k, 4, 2)
    with pytest.raises(ValueError):
        M.moe_route_backward(l, torch.empty((4, 0), dtype=torch.int32, device="cuda"), torch.empty((4, 0), device="cuda"))


def test_many_tokens_with_a_bias_keep_their_rows():
    """The keys replace a row in shared memory while the next row is fetched into the same place:
    enough tokens a warp that a row is reused many times, bit-equal to one token a call."""
    M = _M()
    torch.manual_seed(1)
    T, E = 9001, 64
    l, b = torch.randn(T, E, device="cuda"), torch.randn(E, device="cuda")
    idx, gate = M.moe_route_grouped(l, 8, 8, 4, "top2", "sigmoid", select_bias=b)
    at = list(range(0, 128)) + list(range(T - 128, T))
    for t in at:
        i1, g1 = M.moe_route_grouped(l[t:t + 1], 8, 8, 4, "top2", "sigmoid", select_bias=b)
        assert torch.equal(i1[0], idx[t]) and torch.equal(g1[0], gate[t])
    _ok()
