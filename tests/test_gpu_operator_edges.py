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


def _norm_bars(v, x, y, post, gate, pre, alpha, eps=1e-6):
    """Sizes of the terms of each gradient, as in the norms' own tests."""
    T, d = x.shape
    u, out = np.abs(v["d_x"]), {}
    if pre is not None:
        rx = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
        g, xh = np.abs(v["d_n"] * pre), np.abs(x * rx)
        out["d_pre_weight"] = (np.abs(v["d_n"]) * xh).sum(0)
        u = u + rx * (g + xh * (g * xh).mean(1, keepdims=True))
    yr = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    b = np.abs(y * yr * post)
    out["d_residual"] = abs(alpha) * u
    out["d_gate"] = (u * b).reshape(gate.shape[0], -1, d).sum(1)
    ug = u * np.repeat(np.abs(gate), T // gate.shape[0], axis=0)
    out["d_post_weight"] = (ug * np.abs(y * yr)).sum(0)
    h, yh = ug * np.abs(post), np.abs(y * yr)
    out["d_y"] = yr * (h + yh * (h * yh).mean(1, keepdims=True))
    return out


@pytest.mark.parametrize("T,d,G", [(450, 8192, 3), (300, 7168, 300), (450, 5736, 1), (1500, 2048, 5), (900, 4096, 2),
                                   (900, 4088, 9), (1800, 1112, 4), (2400, 520, 6)])
@pytest.mark.parametrize("yt,rt,nt", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("with_pre", [True, False])
def test_norm_gradients_of_several_rows_a_block(T, d, G, yt, rt, nt, with_pre):
    """More tokens than blocks: the ring of one to four rows turns over, and gate groups end inside a
    block's run and span several."""
    M = _M()
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    g = torch.Generator(device="cuda").manual_seed(T + d)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    v = dict(d_x=(rnd(T, d) * 0.1).to(dt[rt]), d_n=(rnd(T, d) * 0.1).to(dt[nt]) if with_pre else None,
             x_out=rnd(T, d).to(dt[rt]), y=(rnd(T, d) * 0.3).to(dt[yt]))
    post, pre, gate = rnd(d), rnd(d) if with_pre else None, rnd(G, d)
    got = M.moe_block_norm_backward(**v, post_weight=post, gate=gate, alpha=0.5, pre_weight=pre)
    again = M.moe_block_norm_backward(**v, post_weight=post, gate=gate, alpha=0.5, pre_weight=pre)
    _ok()
    n = {k: None if t is None else t.double().cpu().numpy() for k, t in v.items()}
    p = [None if t is None else t.double().cpu().numpy() for t in (post, gate, pre)]
    want = B.block_norm_backward(n["d_x"], n["d_n"], n["x_out"], n["y"], p[0], p[1], 0.5, p[2])
    half = {"d_residual": 2.0 ** -8 if rt == "bf16" else U, "d_y": 2.0 ** -8 if yt == "bf16" else U}
    for key, size in _norm_bars(n, n["x_out"], n["y"], p[0], p[1], p[2], 0.5).items():
        assert torch.equal(got[key], again[key]), key
        err = np.abs(got[key].double().cpu().numpy() - want[key])
        # rows: 256 roundings; column sums: one more for each token
        terms = 256 + (0 if key in half else T)
        assert (err <= terms * U * size + half.get(key, U) * np.abs(want[key]) + 1e-30).all(), key


# ---------------------------------------------------------------- the routing's gradient
def _score64(l, score):
    """Score and derivative in 64 bits, without a difference of near numbers; 0 where masked."""
    e = np.exp(-np.abs(l))
    sig = np.where(l >= 0, 1.0, e) / (1.0 + e)
    if score == "sigmoid":
        return sig, e / (1.0 + e) ** 2
    root = np.sqrt(np.maximum(l, 0.0) + np.log1p(e))
    return root, sig / (2.0 * np.where(root > 0, root, 1.0))


def _parts(l, idx, u, score, renorm, load, aux):
    """The gradient's balance term and gate term, and the sizes of what each is made of: for every
    expert s' / S (|x| + |mean of x|)."""
    s, ds = _score64(l, score)
    out, size = np.zeros_like(l), np.zeros_like(l)
    if load is not None:
        S, f = s.sum(1, keepdims=True), load.astype(np.float64)
        c = aux * l.shape[1] / l.shape[0]
        mean = (s / S * f).sum(1, keepdims=True)
        out += c * ds / S * (f - mean)
        size += c * ds / S * (f + mean)
    if u is not None:
        si, di = np.take_along_axis(s, idx, 1), np.take_along_axis(ds, idx, 1)
        u = u.astype(np.float64)
        if renorm:
            S = si.sum(1, keepdims=True)
            mean, size_m = (si / S * u).sum(1, keepdims=True), (si / S * np.abs(u)).sum(1, keepdims=True)
            g, w = di / S * (u - mean), di / S * (np.abs(u) + size_m)
        else:
            g, w = di * u, di * np.abs(u)
        for t in range(len(l)):
            out[t, idx[t]] += g[t]
            size[t, idx[t]] += w[t]
    return out, size


def _relative(l, score, renorm=True, k=6, gates=True, balance=True, seed=0, floor=0.0):
    """Every expert's gradient within 128 * 2^-24 of the sizes of its own terms.  The score, its
    derivative and the exponentials they share are within 16 steps, sums over a row within 32 + 5
    roundings, each of the 12 products and sums of a term half a step: under 80.  floor: what fp32's
    smallest normal number costs, relative to the row's largest term."""
    M = _M()
    T, E = l.shape
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if gates else None
    u = rng.standard_normal((T, k)).astype(np.float32) if gates else None
    load = (rng.random(E) * 4 / E).astype(np.float32) if balance else None
    aux = 0.25 if balance else 0.0
    c = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a.astype(t))).cuda()
    got = M.moe_route_backward(c(l, np.float32), c(idx, np.int32), c(u, np.float32), score, renorm, 1.0,
                               c(load, np.float32), aux).cpu().numpy().astype(np.float64)
    _ok()
    want, size = _parts(l.astype(np.float32).astype(np.float64), idx, u, score, renorm, load, aux)
    assert np.isfinite(got).all() and (k == 1 or (np.abs(want) > 0).any())   # one gate alone is always 1
    tol = 128 * U * size + floor * size.max(1, keepdims=True) + 1.2e-38
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("at", [0.0, 6.0, 8.0, 12.0, 16.0, 20.0, 30.0])
@pytest.mark.parametrize("score", ["sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("E", [64, 37, 896])
def test_balance_gradient_of_experts_that_are_hard_on(at, score, E):
    """Logits around `at`: the sigmoid's derivative is down to e^-at and has to keep its digits."""
    l = at + np.random.default_rng(int(at) + E).standard_normal((5, E)) * 0.5
    _relative(l, score, gates=False)
    _relative(l, score, k=6)


@pytest.mark.parametrize("at", [-30.0, -60.0, -88.0, -100.0, -150.0, -300.0, -700.0])
@pytest.mark.parametrize("score", ["sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("E,k", [(64, 6), (37, 5), (896, 16), (12, 1)])
def test_gradient_of_scores_that_fp32_cannot_hold(at, score, E, k):
    """Rows far below 0, whose scores' ratios are ordinary numbers: the routing gives them ordinary
    gates, and the gradient follows.  A score below e^-87 of the largest counts as 0."""
    l = at + np.random.default_rng(int(-at) + E).standard_normal((7, E)) * 1.5
    _relative(l, score, True, k, gates=False, floor=1e-30)
    _relative(l, score, True, k, balance=False, floor=1e-30)
    _relative(l, score, True, k, floor=1e-30)


@pytest.mark.parametrize("E", [64, 61])
def test_gradient_of_sqrt_softplus_below_zero(E):
    """Not divided by a sum, and next to larger ones: exp(l / 2) is a number of fp32 down to -174."""
    rng = np.random.default_rng(E)
    l = rng.uniform(-170.0, 10.0, (9, E))
    _relative(l, "sqrt_softplus", False, balance=False)
    _relative(l, "sqrt_softplus", True)
    _relative(rng.uniform(-170.0, -90.0, (9, E)), "sqrt_softplus", False, balance=False)
    _relative(rng.uniform(-80.0, 10.0, (9, E)), "sigmoid", False, balance=False)


@pytest.mark.parametrize("score", ["sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("shift", [0.0, -100.0, -150.0])
def test_masked_experts_and_rows_with_a_balance_term(score, shift):
    rng = np.random.default_rng(9)
    l = shift + rng.standard_normal((6, 32))
    l[0, ::3] = -np.inf
    l[1, 1:] = -np.inf                                       # one expert left
    l[2] = -np.inf                                           # none
    l[3] = -800.0                                            # no score is a number of fp64: gates 0
    _relative_masked(l, score)


def _relative_masked(l, score):
    M = _M()
    rng = np.random.default_rng(1)
    T, E = l.shape
    idx = np.stack([rng.permutation(E)[:4] for _ in range(T)])
    u = rng.standard_normal((T, 4)).astype(np.float32)
    load = (rng.random(E) * 4 / E).astype(np.float32)
    c = lambda a, t: torch.from_numpy(np.ascontiguousarray(a.astype(t))).cuda()
    got = M.moe_route_backward(c(l, np.float32), c(idx, np.int32), c(u, np.float32), score, True, 1.0,
                               c(load, np.float32), 0.25).cpu().numpy().astype(np.float64)
    _ok()
    l32 = l.astype(np.float32).astype(np.float64)
    dead = ~(l32 > -745.0).any(1)
    live = l32 > -np.inf
    u = np.where(np.take_along_axis(live, idx, 1), u, 0.0)
    for t in range(T):
        if dead[t]:
            assert (got[t] == 0).all()
            continue
        want, size = np.zeros((1, E)), np.zeros((1, E))
        s, ds = _score64(l32[t], score)
        S, c_ = s.sum(), 0.25 * E / T
        mean = (s * load).sum() / S
        want[0] += c_ * ds / S * (load - mean)
        size[0] += c_ * ds / S * (load + mean)
        si = s[idx[t]]
        if si.sum() > 0:
            mu, ma = (si * u[t]).sum() / si.sum(), (si * np.abs(u[t])).sum() / si.sum()
            want[0, idx[t]] += ds[idx[t]] / si.sum() * (u[t] - mu)
            size[0, idx[t]] += ds[idx[t]] / si.sum() * (np.abs(u[t]) + ma)
        want[0, ~live[t]] = 0.0
        tol = 128 * U * size[0] + 1e-30 * size.max() + 1.2e-38
        assert (np.abs(got[t] - want[0]) <= tol).all() and (got[t][~live[t]] == 0).all()


# ---------------------------------------------------------------- the routing's gates
@pytest.mark.parametrize("T,E,k,G,kept", [(64, 896, 16, 16, 4), (64, 1024, 8, 1, 1), (33, 255, 5, 3, 2), (64, 8, 2, 4, 2)])
@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0, 12.0])
def test_full_softmax_gates_are_within_the_stated_bound(T, E, k, G, kept, spread):
    """Without renormalising: the denominator over all experts is within 120 * 2^-24 (at spread 0
    with a bias every key is equal, and a token is taken in fp64, or its terms are few and all 1)."""
    M = _M()
    l = (np.random.default_rng(E).standard_normal((T, E)) * spread).astype(np.float32)
    for bias in (None, np.zeros(E, np.float32)):
        on = None if bias is None else torch.from_numpy(bias).cuda()
        for gs in ("max", "top2"):
            i, g = M.moe_route_grouped(torch.from_numpy(l).cuda(), k, G, kept, gs, "softmax", False, 1.0, on)
            _ok()
            p = np.exp(l.astype(np.float64) - l.max(1, keepdims=True))
            want = np.take_along_axis(p / p.sum(1, keepdims=True), i.cpu().numpy().astype(np.int64), 1)
            err = np.abs(g.cpu().numpy() - want) / want
            assert err.max() <= 121 * U
            if spread == 0.0 and bias is not None:
                assert err.max() <= U * 1.001               # rounded once


# ---------------------------------------------------------------- the 8-bit products
@pytest.mark.parametrize("call", ["gate_up", "gather", "down"])
@pytest.mark.parametrize("tiles", ["tokens", "weights"])
def test_bad_offsets_between_good_experts(call, tiles, monkeypatch):
    """Two entries out of the buffer: the experts on both sides of each are skipped and recorded, all
    others' rows are right, and nothing else is written.  More tiles than CTA pairs, empty experts
    among them, so that every role walks past the gaps."""
    M = _M()
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", tiles)
    d, F, E = (256, 1040, 60) if call != "down" else (1040, 640, 60)
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 40, E)
    counts[[0, 7, 8, 30, E - 1]] = [3, 0, 300, 0, 17]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1])
    N, K = (2 * F, d) if call != "down" else (d, F)
    T = 50 if call == "gather" else rows
    q = rng.integers(-127, 128, (T, K)).astype(np.int8)
    scale = ((rng.random(T) + 0.5) * 1e-2).astype(np.float32)
    W = rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    ws = ((rng.random((E, N)) + 0.5) * (2e-2 / np.sqrt(K))).astype(np.float32)
    tok = rng.integers(0, T, rows).astype(np.int32) if call == "gather" else None
    bad = off.copy()
    bad[12], bad[41] = rows + 50, -3
    c = lambda a: torch.from_numpy(a).cuda()
    out = torch.full((rows, F if call != "down" else d), 7.0, dtype=torch.bfloat16, device="cuda")
    if call == "down":
        M.moe_expert_down_i8(c(q), c(scale), c(bad), c(W), c(ws), rows, y_rows=out)
    else:
        M.moe_expert_gate_up_i8(c(q), c(scale), c(bad), c(W), c(ws), rows, out, None if tok is None else c(tok))
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 3
    rq, rs = (q, scale) if tok is None else (q[tok], scale[tok])
    want = (B.down_i8 if call == "down" else B.gate_up_i8)(rq, rs, off, W, ws)
    for e in (11, 12, 40, 41):
        want[off[e]:off[e + 1]] = 7.0
    tol = 4 * U + 2.0 ** -8 if call == "down" else 2.0 ** -8 + 2.0 ** -17
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) * tol + 1e-30).all()


@pytest.mark.parametrize("tiles", ["tokens", "weights"])
def test_more_rows_than_any_tile_and_most_experts_empty(tiles, monkeypatch):
    """896 experts of which five have rows: the walk to the next tile's expert passes hundreds."""
    M = _M()
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", tiles)
    E, d, F = 896, 128, 272
    counts = np.zeros(E, np.int64)
    counts[[0, 3, 400, 894, 895]] = [1, 700, 257, 5, 130]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1])
    rng = np.random.default_rng(5)
    q, scale = rng.integers(-127, 128, (rows, d)).astype(np.int8), (rng.random(rows) * 0.05).astype(np.float32)
    W, ws = rng.integers(-127, 128, (E, 2 * F, d)).astype(np.int8), (rng.random((E, 2 * F)) * 1e-3).astype(np.float32)
    c = lambda a: torch.from_numpy(a).cuda()
    h = M.moe_expert_gate_up_i8(c(q), c(scale), c(off), c(W), c(ws), rows)
    _ok()
    want = B.gate_up_i8(q, scale, off, W, ws)
    assert (np.abs(h.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()
