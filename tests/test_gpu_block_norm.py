"""The norms around a block and their gradients against the float64 reference.

Bars.  A sum over a row has at most 16 elements a thread, then 5 + 5 shuffles: under 32 roundings;
a norm takes its square root, and each output a dozen products more.  So an output is within
64 * 2^-24 (96 for what passed two norms, 128 for gradients) of the sizes of the terms it is made
of, plus its type's half step.  Column sums: one fp32 addition for each token a block has (every
token, at worst) on top, relative to the sum of the terms' sizes.
"""
import numpy as np
import pytest
import torch

from oracle import block_ops as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


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


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _make(T, d, G, y, r, n, post, pre, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + d)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    return dict(r=rnd(T, d).to(r), y=None if y is None else (rnd(T, d) * 0.3).to(y), post=rnd(d) if post else None,
                pre=rnd(d) if pre else None, gate=rnd(G, d) if G else None, dx=(rnd(T, d) * 0.1).to(r),
                dn=(rnd(T, d) * 0.1).to(n) if pre else None)


def _close(got, want, size, factor, dtype, what):
    err = np.abs(_np(got) - want)
    tol = factor * U * size + HALF[dtype] * np.abs(want) + 1e-30
    assert (err <= tol).all(), (what, float((err / tol).max()))


def _sizes(v, y, alpha):
    """|alpha r| + |gate b| and that over rms(x'), times |pre|."""
    b = np.abs(y)
    if v["post"] is not None:
        b = np.abs(_np(v["post"])) * b / np.sqrt((y * y).mean(1, keepdims=True) + EPS)
    if v["gate"] is not None:
        b = b * np.repeat(np.abs(_np(v["gate"])), len(y) // v["gate"].shape[0], axis=0)
    return abs(alpha) * np.abs(_np(v["r"])) + b


TYPES = [(BF, BF, BF), (F32, F32, F32), (BF, F32, BF), (F32, BF, F32)]
SHAPES = [(1, 8, 1), (3, 64, 0), (5, 264, 5), (12, 2048, 3), (7, 2056, 1), (4, 7168, 2), (2, 8192, 0), (600, 136, 4)]


@pytest.mark.parametrize("T,d,G", SHAPES)
@pytest.mark.parametrize("yt,rt,nt", TYPES)
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_forward(T, d, G, yt, rt, nt, post, pre):
    M = _M()
    v = _make(T, d, G, yt, rt, nt, post, pre)
    x, n = M.moe_block_norm(v["r"], v["y"], v["post"], v["gate"], 0.7, v["pre"], EPS, n_dtype=nt)
    _ok()
    alpha = float(np.float32(0.7))
    wx, wn = B.block_norm(_np(v["r"]), _np(v["y"]), _np(v["post"]), _np(v["gate"]), alpha, _np(v["pre"]), EPS)
    size = _sizes(v, _np(v["y"]), alpha)
    assert x.dtype == rt
    _close(x, wx, size, 64, rt, "x")
    if pre:
        assert n.dtype == nt
        rms = np.sqrt((wx * wx).mean(1, keepdims=True) + EPS)
        # an error of x' also moves its norm: by at most the largest relative one of the row's sizes
        total = np.sqrt((size * size).mean(1, keepdims=True)) / rms
        _close(n, wn, np.abs(_np(v["pre"])) * (size / rms + np.abs(wx) / rms * total), 96, nt, "n")
    else:
        assert n is None


@pytest.mark.parametrize("T,d", [(1, 8), (9, 2048), (3, 7168)])
@pytest.mark.parametrize("rt", [BF, F32])
def test_first_pre_norm_alone(T, d, rt):
    M = _M()
    v = _make(T, d, 0, None, rt, BF, False, True)
    x, n = M.moe_block_norm(v["r"], pre_weight=v["pre"])
    assert x is None and n.dtype == BF
    wx, wn = B.block_norm(_np(v["r"]), pre=_np(v["pre"]))
    _close(n, wn, np.abs(wn), 64, BF, "n")
    _ok()


@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (5, 264, 3), (33, 2048, 8), (6, 7168, 16), (4, 128, 32), (700, 64, 2)])
@pytest.mark.parametrize("yt,rt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("extra", [False, True])
def test_combine_in_front(T, d, k, yt, rt, extra):
    M = _M()
    v = _make(T, d, 1, None, rt, BF, True, True)
    g = torch.Generator(device="cuda").manual_seed(T + k)
    rows = (torch.randn(T * k, d, device="cuda", generator=g) * 0.3).to(yt)
    row_of = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32).view(T, k).clone()
    row_of[torch.rand(T, k, device="cuda", generator=g) < 0.2] = -1
    row_of[0] = -1                                           # a token that lost every slot
    gate = torch.rand(T, k, device="cuda", generator=g) if extra else None
    sh = torch.randn(T, d, device="cuda", generator=g).to(yt) if extra else None
    y_out = torch.empty(T, d, dtype=yt, device="cuda")
    x, n = M.moe_combine_norm(v["r"], rows, row_of, T * k, gate, sh, v["post"], v["gate"], 1.0, v["pre"], EPS, y_out)
    _ok()
    rn, ro = _np(rows), row_of.cpu().numpy()
    y = B.combine_sum(rn, ro, _np(gate), _np(sh))
    ysize = B.combine_sum(np.abs(rn), ro, _np(gate), None if sh is None else np.abs(_np(sh)))
    _close(y_out, y, ysize, 2 * k + 2, yt, "y")
    wx, wn = B.block_norm(_np(v["r"]), y, _np(v["post"]), _np(v["gate"]), 1.0, _np(v["pre"]), EPS)
    rms = np.sqrt((y * y).mean(1, keepdims=True) + EPS)
    pg = np.abs(_np(v["post"])) * np.abs(_np(v["gate"]))
    spread = np.sqrt((ysize * ysize).mean(1, keepdims=True)) / rms
    size = np.abs(_np(v["r"])) + pg * (ysize + np.abs(y) * spread) / rms
    _close(x, wx, size, 64 + 2 * k, rt, "x")
    rx = np.sqrt((wx * wx).mean(1, keepdims=True) + EPS)
    total = np.sqrt((size * size).mean(1, keepdims=True)) / rx
    _close(n, wn, np.abs(_np(v["pre"])) * (size / rx + np.abs(wx) / rx * total), 96 + 2 * k, BF, "n")
    # the plain form on the combine's own fp32 sum agrees bit for bit
    if yt == F32:
        x2, n2 = M.moe_block_norm(v["r"], y_out, v["post"], v["gate"], 1.0, v["pre"], EPS)
        assert torch.equal(x, x2) and torch.equal(n, n2)


def test_combine_matches_moe_combine_bit_for_bit():
    M = _M()
    T, k, d = 50, 4, 512
    rows = torch.randn(T * k, d, device="cuda")
    row_of = torch.randperm(T * k, device="cuda").to(torch.int32).view(T, k)
    y_out = torch.empty(T, d, device="cuda")
    M.moe_combine_norm(torch.zeros(T, d, device="cuda"), rows, row_of, T * k, y_out=y_out)
    assert torch.equal(y_out, M.moe_combine(rows, row_of, T, T * k))
    row_of[0, 0] = T * k + 5                                 # past the rows: skipped and recorded
    M.moe_combine_norm(torch.zeros(T, d, device="cuda"), rows, row_of, T * k, y_out=y_out)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 3


def test_rows_of_zeros_and_one_bad_row():
    M = _M()
    r = torch.zeros(4, 64, device="cuda")
    y = torch.randn(4, 64, device="cuda")
    y[0] = 0.0
    y[2, 3] = float("nan")
    w = torch.ones(64, device="cuda")
    x, n = M.moe_block_norm(r, y, w, None, 1.0, w, n_dtype=F32)
    _ok()
    assert (x[0] == 0).all() and (n[0] == 0).all()
    assert torch.isnan(n[2]).all() and torch.isfinite(n[[0, 1, 3]]).all()


def test_in_place_residual():
    M = _M()
    v = _make(9, 2048, 1, BF, BF, BF, True, True)
    x, n = M.moe_block_norm(v["r"], v["y"], v["post"], v["gate"], 0.5, v["pre"])
    keep = v["r"].clone()
    x2, n2 = M.moe_block_norm(keep, v["y"], v["post"], v["gate"], 0.5, v["pre"], x_out=keep)
    assert x2.data_ptr() == keep.data_ptr() and torch.equal(x, keep) and torch.equal(n, n2)
    _ok()


@pytest.mark.parametrize("T,d,G", SHAPES + [(5000, 64, 1), (4096, 8, 4096), (301, 2048, 7)])
@pytest.mark.parametrize("yt,rt,nt", TYPES)
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_backward(T, d, G, yt, rt, nt, post, pre):
    M = _M()
    v = _make(T, d, G, yt, rt, nt, post, pre)
    alpha = float(np.float32(0.7))
    a = dict(post_weight=v["post"], gate=v["gate"], alpha=0.7, pre_weight=v["pre"], eps=EPS)
    got = M.moe_block_norm_backward(v["dx"], v["dn"], v["r"], v["y"], **a)
    again = M.moe_block_norm_backward(v["dx"], v["dn"], v["r"], v["y"], **a)
    _ok()
    for k in got:                                            # repeats bit for bit
        assert (got[k] is None) == (again[k] is None) and (got[k] is None or torch.equal(got[k], again[k])), k
    n = {k: _np(v[k]) for k in v}
    want = B.block_norm_backward(n["dx"], n["dn"], n["r"], n["y"], n["post"], n["gate"], alpha, n["pre"], EPS)
    x, y = n["r"], n["y"]
    u = np.abs(n["dx"])
    if pre:
        rx = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + EPS)
        gsz = np.abs(n["dn"] * n["pre"])
        u = u + rx * (gsz + np.abs(x * rx) * (gsz * np.abs(x * rx)).mean(1, keepdims=True))
        _close(got["d_pre_weight"], want["d_pre_weight"], np.abs(n["dn"] * x * rx).sum(0), 128 + T, F32, "pre")
    _close(got["d_residual"], want["d_residual"], alpha * u, 128, rt, "residual")
    yr = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + EPS)
    b = np.abs(y) if not post else np.abs(y * yr * n["post"])
    ug = u
    if G:
        size = (u * b).reshape(G, -1, d).sum(1)
        _close(got["d_gate"], want["d_gate"], size, 256 + T // G, F32, "gate")
        ug = u * np.repeat(np.abs(n["gate"]), T // G, axis=0)
    if post:
        _close(got["d_post_weight"], want["d_post_weight"], (ug * np.abs(y * yr)).sum(0), 256 + T, F32, "post")
        h = ug * np.abs(n["post"])
        size = yr * (h + np.abs(y * yr) * (h * np.abs(y * yr)).mean(1, keepdims=True))
        _close(got["d_y"], want["d_y"], size, 256, yt, "y")
    else:
        _close(got["d_y"], want["d_y"], ug, 160, yt, "y")
    assert (got["d_gate"] is None) == (G == 0) and (got["d_post_weight"] is None) == (not post)


def test_backward_parts():
    """No branch, no d_x, in place, and an empty batch."""
    M = _M()
    v = _make(11, 264, 0, BF, F32, F32, True, True)
    g = M.moe_block_norm_backward(None, v["dn"], v["r"], pre_weight=v["pre"])
    want = B.block_norm_backward(None, _np(v["dn"]), _np(v["r"]), pre=_np(v["pre"]))
    err = np.abs(_np(g["d_residual"]) - want["d_residual"]).max()
    assert err <= 128 * U * 4 * np.abs(_np(v["dn"]) * _np(v["pre"])).max() / np.sqrt((_np(v["r"]) ** 2).mean(1)).min()
    assert g["d_y"] is None and g["d_gate"] is None and g["d_post_weight"] is None
    a = M.moe_block_norm_backward(v["dx"], v["dn"], v["r"], v["y"], v["post"], None, 0.5, v["pre"])
    dx = v["dx"].clone()
    b = M.moe_block_norm_backward(dx, v["dn"], v["r"], v["y"], v["post"], None, 0.5, v["pre"], d_residual=dx)
    assert torch.equal(a["d_residual"], dx) and torch.equal(a["d_y"], b["d_y"])
    e = torch.empty(0, 264, device="cuda")
    c = M.moe_block_norm_backward(e, e, e, e, v["post"], None, 0.5, v["pre"])
    _ok()
    assert (c["d_post_weight"] == 0).all() and (c["d_pre_weight"] == 0).all() and c["d_y"].shape == (0, 264)
    x, n = M.moe_block_norm(e, e, v["post"], None, 1.0, v["pre"])
    assert x.shape == (0, 264) and n.shape == (0, 264)


def test_gradients_through_autograd_of_the_formula():
    M = _M()
    v = _make(24, 256, 3, F32, F32, F32, True, True)
    p = {k: v[k].double().requires_grad_(True) for k in ("r", "y", "post", "pre", "gate")}
    y = p["y"] / torch.sqrt(p["y"].pow(2).mean(1, keepdim=True) + EPS) * p["post"]
    x = 0.5 * p["r"] + p["gate"].repeat_interleave(8, 0) * y
    n = x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + EPS) * p["pre"]
    ((x * v["dx"].double()).sum() + (n * v["dn"].double()).sum()).backward()
    xo, _ = M.moe_block_norm(v["r"], v["y"], v["post"], v["gate"], 0.5, v["pre"], EPS, n_dtype=F32)
    g = M.moe_block_norm_backward(v["dx"], v["dn"], xo, v["y"], v["post"], v["gate"], 0.5, v["pre"], EPS)
    _ok()
    for key, name in (("r", "d_residual"), ("y", "d_y"), ("post", "d_post_weight"), ("pre", "d_pre_weight"),
                      ("gate", "d_gate")):
        w = p[key].grad
        # sums of at most 24 terms of the gradient's own size, 256 roundings each at worst
        assert (g[name].double() - w).abs().max() <= 256 * U * 24 * w.abs().max(), name


def test_refusals():
    M = _M()
    r = torch.randn(6, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(M.MoEError):
        M.moe_block_norm(r, r, gate=torch.ones(4, 64, device="cuda"))       # 4 does not divide 6
    with pytest.raises(M.MoEError):
        M.moe_block_norm(r)                                                  # nothing to write
    with pytest.raises(M.MoEError):
        M.moe_block_norm(r, pre_weight=w, eps=0.0)
    with pytest.raises(M.MoEError):
        M.moe_block_norm(r, post_weight=w, pre_weight=w)                     # a post-norm of nothing
    with pytest.raises(M.MoEError):
        M.moe_block_norm(torch.randn(2, 8200, device="cuda"), pre_weight=torch.ones(8200, device="cuda"))
    with pytest.raises(ValueError):
        M.moe_block_norm(r, r, post_weight=torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        M.moe_block_norm(r, r[:3])
    with pytest.raises(ValueError):
        M.moe_block_norm(r.t(), pre_weight=torch.ones(6, device="cuda"))
    with pytest.raises(M.MoEError):
        M.moe_block_norm_backward(r, None, r, r, w, None, 1.0, w)            # pre_weight without d_n


def test_two_graphs_and_another_stream():
    M = _M()
    v = _make(300, 256, 2, BF, BF, BF, True, True)
    args = (v["post"], v["gate"], 0.5, v["pre"])

    def step(dx):
        return M.moe_block_norm_backward(dx, v["dn"], v["r"], v["y"], *args)

    want = step(v["dx"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step(v["dx"])
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    outs, graphs, bufs = [], [], []
    for _ in range(2):                                       # each capture holds a workspace of its own
        buf = torch.zeros_like(v["dx"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(buf))
        graphs.append(g)
        bufs.append(buf)
    for b in bufs:
        b.copy_(v["dx"])
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], want[k]) for k in want)
    _ok()


def test_an_empty_gate_is_refused():
    M = _M()
    x = torch.ones((4, 64), device="cuda")
    with pytest.raises(ValueError):
        M.moe_block_norm(x, x, gate=torch.empty((0, 64), device="cuda"))


def test_a_given_streams_call_allocates_on_it(monkeypatch):
    """Every call with stream= allocates its outputs and its workspace while that stream is current."""
    M = _M()
    st, seen = torch.cuda.Stream(), []
    real_new, real_like = M._new, torch.empty_like
    monkeypatch.setattr(M, "_new", lambda *a: (seen.append(torch.cuda.current_stream()), real_new(*a))[1])
    monkeypatch.setattr(torch, "empty_like",
                        lambda *a, **k: (seen.append(torch.cuda.current_stream()), real_like(*a, **k))[1])
    x, w = torch.randn(8, 128, device="cuda"), torch.ones(128, device="cuda")
    l = torch.randn(8, 32, device="cuda")
    torch.cuda.synchronize()
    idx, gate = M.moe_route_grouped(l, 4, 4, 2, stream=st)
    M.moe_route_backward(l, idx, gate, stream=st)
    q, s = M.moe_quantize_rows_i8(x, stream=st)
    xo, n = M.moe_block_norm(x, x, post_weight=w, pre_weight=w, stream=st)
    M.moe_block_norm_backward(x, n, xo, x, post_weight=w, pre_weight=w, stream=st)
    assert len(seen) >= 12 and all(c == st for c in seen)
    assert torch.cuda.current_stream() != st
    torch.cuda.synchronize()
    _ok()
