"""A whole block as it is used: pre-norm, router with groups and a bias, 8-bit experts, shared
expert, combine with post-norm, gate, residual and the next norm; each stage against the float64
reference of what the GPU gave it (a rounding that flips in one stage then stays there)."""
import numpy as np
import pytest
import torch

from oracle import block_ops as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
T, D, E, K, F, FS = 300, 256, 16, 4, 144, 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _block(dispatch, capacity=-1, shared=True, overlap=True):
    from routing_dispatch_expert_moe_b200 import moe as M
    from routing_dispatch_expert_moe_b200.layer import MoEBlock, MoELayer, MoEWeights
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    bf = torch.bfloat16
    w = MoEWeights(Wg=rnd(D, E) * 0.1, W_gu=None, W_dn=None, select_bias=rnd(E) * 0.05,
                   W_gu_i8=M.quantize_experts_i8(rnd(E, 2 * F, D) * 0.08),
                   W_dn_i8=M.quantize_experts_i8((rnd(E, D, F) * 0.08).to(bf)))
    if shared:
        w.W_gu_s, w.W_dn_s = (rnd(1, 2 * FS, D) * 0.05).to(bf), (rnd(1, D, FS) * 0.05).to(bf)
    lay = MoELayer(w, K, T, "sigmoid", True, 2.0, capacity, rows_dtype=bf, out_dtype=bf, dispatch=dispatch,
                   overlap=overlap, n_groups=4, groups_kept=2)
    blk = MoEBlock(lay, 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D), rnd(3, D), 0.5, 1 + 0.1 * rnd(D))
    r = rnd(T, D).to(bf)
    return M, w, lay, blk, r


def _n(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dispatch", ["permute", "gather"])
@pytest.mark.parametrize("capacity", [-1, 60])
def test_stages(dispatch, capacity):
    M, w, lay, blk, r = _block(dispatch, capacity)
    x, nn = blk.forward(r)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
    # the pre-norm
    _, want = B.block_norm(_n(r), pre=_n(blk.pre_weight))
    n = blk.n[:T]
    assert (np.abs(_n(n) - want) <= (2.0 ** -8 + 64 * U) * np.abs(want)).all()
    # routing of the GPU's own logits
    idx, gate, margin = B.route_grouped(lay.logits.cpu().numpy(), K, 4, 2, "top2", "sigmoid", True, 2.0,
                                        w.select_bias.cpu().numpy())
    sure = margin > 1e-13
    assert sure.all() and np.array_equal(lay.topk_idx.cpu().numpy(), idx)
    assert (np.abs(_n(lay.topk_gate) - gate) <= 2 * U * gate).all()
    # dispatch and 8 bits
    off, row_of, tok = (t.cpu().numpy() for t in (lay.offsets, lay.row_of, lay.token_of_row))
    used = int(off[-1])
    q, s = B.quantize_rows(n.float().cpu().numpy())
    if dispatch == "permute":
        assert np.array_equal(lay.x_q.cpu().numpy()[:used], q[tok[:used]])
        assert np.array_equal(lay.x_scale.cpu().numpy()[:used], s[tok[:used]])
    else:
        assert np.array_equal(lay.x_q.cpu().numpy()[:T], q) and np.array_equal(lay.x_scale.cpu().numpy()[:T], s)
    if capacity > 0:
        assert used < T * K                                   # something was dropped
    # the expert products
    wh = B.gate_up_i8(q[tok[:used]], s[tok[:used]], off, *(t.cpu().numpy() for t in w.W_gu_i8))
    h = lay.h[:used]
    assert (np.abs(_n(h) - wh) <= np.abs(wh) * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()
    hq, hs = B.quantize_rows(h.float().cpu().numpy())
    assert np.array_equal(lay.h_q.cpu().numpy()[:used], hq)
    wy = B.down_i8(hq, hs, off, *(t.cpu().numpy() for t in w.W_dn_i8), lay.gate_of_row.cpu().numpy()[:used])
    assert (np.abs(_n(lay.y_perm[:used]) - wy) <= np.abs(wy) * (2.0 ** -8 + 5 * U)).all()
    # combine, post-norm, gate, residual, next norm: of the GPU's rows
    rows = np.zeros((T * K, D))
    rows[:used] = _n(lay.y_perm[:used])
    y = B.combine_sum(rows, row_of, None, _n(lay.y_s[:T]))
    wx, wn = B.block_norm(_n(r), y, _n(blk.post_weight), _n(blk.gate), 0.5, _n(blk.next_weight))
    ysum = B.combine_sum(np.abs(rows), row_of, None, np.abs(_n(lay.y_s[:T])))
    rms = np.sqrt((y * y).mean(1, keepdims=True))
    spread = np.sqrt((ysum * ysum).mean(1, keepdims=True)) / rms
    pg = np.abs(_n(blk.post_weight)) * np.repeat(np.abs(_n(blk.gate)), T // 3, axis=0)
    size = 0.5 * np.abs(_n(r)) + pg * (ysum + np.abs(y) * spread) / rms
    assert (np.abs(_n(x) - wx) <= 80 * U * size + 2.0 ** -8 * np.abs(wx)).all()
    rx = np.sqrt((wx * wx).mean(1, keepdims=True))
    total = np.sqrt((size * size).mean(1, keepdims=True)) / rx
    tol = np.abs(_n(blk.next_weight)) * (size + np.abs(wx) * total) / rx
    assert (np.abs(_n(nn) - wn) <= 110 * U * tol + 2.0 ** -8 * np.abs(wn)).all()


def test_dispatch_forms_agree_and_a_chain_skips_the_norm():
    M, w, lay, blk, r = _block("permute")
    a, an = (t.clone() for t in blk.forward(r))
    M2, w2, lay2, blk2, r2 = _block("gather")
    b, bn = (t.clone() for t in blk2.forward(r2))
    # both dispatch forms take weight-major tiles here (75 rows an expert): the same products
    assert torch.equal(a, b) and torch.equal(an, bn)
    # a second block fed with the first one's n' equals one that norms x' itself, but for that norm's
    # rounding of x' (bf16): the n' given is closer to the truth; it only has to run and be finite
    x2, n2 = blk.forward(a, n=an)
    assert torch.isfinite(x2).all() and torch.isfinite(n2).all()
    assert M.moe_get_device_error() == 0


@pytest.mark.parametrize("overlap", [True, False])
def test_smaller_batches_streams_and_graph(overlap):
    M, w, lay, blk, r = _block("permute", overlap=overlap)
    want = {}
    for t in (3, 30, 300):
        x, n = blk.forward(r[:t])
        want[t] = (x.clone(), n.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, n = blk.forward(r[:30], stream=s)
    s.synchronize()
    assert torch.equal(x, want[30][0]) and torch.equal(n, want[30][1])
    buf = torch.zeros_like(r[:300])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            x, n = blk.forward(buf, stream=side)
    buf.copy_(r)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want[300][0]) and torch.equal(n, want[300][1])
    assert M.moe_get_device_error() == 0


def test_launch_count():
    _, _, lay, _, _ = _block("permute", shared=False)
    _, _, lay2, _, _ = _block("gather", shared=False)
    # router, grouped top-k, rank, scatter, x to 8 bits, gate/up, h to 8 bits, down, combine
    assert lay.launches_per_forward(False) == 9 and lay2.launches_per_forward(False) == 9


@pytest.mark.parametrize("T,form", [(256, "gather"), (2048, "permute")])
def test_auto_dispatch_of_8_bit_experts_follows_their_tiles(T, form):
    """48 and 384 rows an expert on average."""
    from routing_dispatch_expert_moe_b200.layer import MoELayer, MoEWeights
    from routing_dispatch_expert_moe_b200 import moe as M
    E, d, F, k = 16, 256, 128, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    w = MoEWeights(Wg=rnd(d, E) * 0.1, W_gu=None, W_dn=None, W_gu_i8=M.quantize_experts_i8(rnd(E, 2 * F, d)),
                   W_dn_i8=M.quantize_experts_i8(rnd(E, d, F)))
    x = rnd(T, d).bfloat16()
    out = {}
    for dispatch in ("auto", form):
        lay = MoELayer(w, k=k, T_max=T, dispatch=dispatch)
        assert dispatch != "auto" or lay.dispatch_mode == form
        out[dispatch] = lay.forward(x).clone()
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
    assert torch.equal(out["auto"], out[form])


FIRST_CALLS = """
import torch
from routing_dispatch_expert_moe_b200 import moe as M
l, x = torch.randn(64, 896, device="cuda"), torch.randn(64, 256, device="cuda").bfloat16()
w, off = torch.ones(256, device="cuda"), torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
Wq, ws = torch.ones((2, 256, 256), dtype=torch.int8, device="cuda"), torch.ones((2, 256), device="cuda")

def route():
    i, g = M.moe_route_grouped(l, 8, 8, 4)
    return g, M.moe_route_backward(l, i, g, "sigmoid", z_coef=0.1)

def i8():
    q, s = M.moe_quantize_rows_i8(x)
    h = M.moe_expert_gate_up_i8(q, s, off, Wq, ws, 64)
    return h, M.moe_expert_down_i8(q[:, :128].contiguous(), s, off, Wq[:, :, :128].contiguous(), ws, 64)

def norm():
    xo, n = M.moe_block_norm(x, x, w, None, 1.0, w)
    return n, M.moe_block_norm_backward(x, x, xo, x, w, None, 1.0, w)["d_post_weight"]

for f in (route, i8, norm):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, f())), f.__name__
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
print("captured")
"""


def test_a_process_first_calls_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("rows", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t", [300, 33])
def test_a_block_keeps_what_its_norms_gradients_take(rows, t):
    """y as the combine sums it, rounded once; the gradients behind the layer from it and x'."""
    from routing_dispatch_expert_moe_b200.layer import MoEBlock, MoELayer
    M, w, lay, blk, r = _block("permute")
    lay = MoELayer(w, K, T, "sigmoid", True, 2.0, -1, rows_dtype=rows, n_groups=4, groups_kept=2)
    args = (blk.pre_weight, blk.post_weight, blk.gate, 0.5, blk.next_weight)
    kept = MoEBlock(lay, *args, keep_y=True)
    x, n = (v.clone() for v in MoEBlock(lay, *args).forward(r[:t]))
    x2, n2 = kept.forward(r[:t])
    y = kept.y[:t]
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
    assert torch.equal(x, x2) and torch.equal(n, n2)         # keeping y changes nothing else
    row_of = lay.row_of[:t].cpu().numpy()
    used = int(lay.offsets[-1])
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.1
    want_y = B.combine_sum(_n(lay.y_perm[:used]), row_of, None, _n(lay.y_s[:t]))
    size = B.combine_sum(np.abs(_n(lay.y_perm[:used])), row_of, None, np.abs(_n(lay.y_s[:t])))
    half = 2.0 ** -8 if rows == torch.bfloat16 else U
    assert y.dtype == rows and (np.abs(_n(y) - want_y) <= (K + 1) * U * size + half * np.abs(want_y)).all()
    dx, dn = rnd(t, D).bfloat16(), rnd(t, D).bfloat16()
    got = M.moe_block_norm_backward(dx, dn, x2, y, blk.post_weight, blk.gate, 0.5, blk.next_weight, kept.eps)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
    want = B.block_norm_backward(_n(dx), _n(dn), _n(x2), _n(y), _n(blk.post_weight), _n(blk.gate), 0.5,
                                 _n(blk.next_weight), kept.eps)
    # the bars of the norms' own tests: (256 + T) roundings of the sums of the terms' sizes
    rx = 1.0 / np.sqrt((_n(x2) ** 2).mean(1, keepdims=True) + kept.eps)
    xh, gs = np.abs(_n(x2)) * rx, np.abs(_n(dn) * _n(blk.next_weight))
    u = np.abs(_n(dx)) + rx * (gs + xh * (gs * xh).mean(1, keepdims=True))
    yr = 1.0 / np.sqrt((_n(y) ** 2).mean(1, keepdims=True) + kept.eps)
    yh = np.abs(_n(y)) * yr
    sizes = {"d_residual": 0.5 * u, "d_pre_weight": (np.abs(_n(dn)) * xh).sum(0),
             "d_gate": (u * yh * np.abs(_n(blk.post_weight))).reshape(3, -1, D).sum(1)}
    ug = u * np.repeat(np.abs(_n(blk.gate)), t // 3, axis=0)
    sizes["d_post_weight"] = (ug * yh).sum(0)
    h = ug * np.abs(_n(blk.post_weight))
    sizes["d_y"] = yr * (h + yh * (h * yh).mean(1, keepdims=True))
    for key, sz in sizes.items():
        step = {"d_residual": 2.0 ** -8, "d_y": half}.get(key, U)
        assert (np.abs(_n(got[key]) - want[key]) <= (256 + t) * U * sz + step * np.abs(want[key]) + 1e-30).all(), key


@pytest.mark.parametrize("routing", ["hash", "noisy", "uniform"])
def test_a_block_over_the_other_routing_rules(routing):
    """The rule's inputs reach the layer: the block equals its norm, the layer and the combine's norm."""
    from routing_dispatch_expert_moe_b200 import moe as M
    from routing_dispatch_expert_moe_b200.layer import MoEBlock, MoELayer, MoEWeights
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    bf, t = torch.bfloat16, 50
    w = MoEWeights(Wg=rnd(D, E) * 0.1, W_gu=(rnd(E, 2 * F, D) * 0.08).to(bf), W_dn=(rnd(E, D, F) * 0.08).to(bf),
                   W_noise=rnd(D, E) * 0.1 if routing == "noisy" else None)
    lay = MoELayer(w, K, 64, rows_dtype=bf, routing=routing)
    blk = MoEBlock(lay, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"))
    r = rnd(t, D).to(bf)
    extra = {"hash": dict(token_id=torch.arange(t, dtype=torch.int32, device="cuda")),
             "noisy": dict(noise=rnd(t, E)), "uniform": {}}[routing]
    x = blk.forward(r, **extra)[0].clone()
    if extra:
        with pytest.raises(ValueError, match="needs"):
            blk.forward(r)
    n = M.moe_block_norm(r, pre_weight=blk.pre_weight)[1]
    lay.forward(n, **extra)
    want = M.moe_combine_norm(r, lay.y_perm, lay.row_of[:t], lay.rows_max, post_weight=blk.post_weight)[0]
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 0
    assert torch.equal(x, want)


@pytest.mark.parametrize("tiles,form", [("tokens", "permute"), ("weights", "gather")])
def test_auto_dispatch_of_8_bit_experts_obeys_the_override(tiles, form, monkeypatch):
    from routing_dispatch_expert_moe_b200 import moe as M
    from routing_dispatch_expert_moe_b200.layer import MoELayer, MoEWeights
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", tiles)
    w = MoEWeights(Wg=torch.randn(D, E, device="cuda"), W_gu=None, W_dn=None,
                   W_gu_i8=M.quantize_experts_i8(torch.randn(E, 2 * F, D, device="cuda")),
                   W_dn_i8=M.quantize_experts_i8(torch.randn(E, D, F, device="cuda")))
    lay = MoELayer(w, k=K, T_max=64 if tiles == "tokens" else 2048, dispatch="auto")   # 16 and 512 rows an expert
    assert lay.dispatch_mode == form
