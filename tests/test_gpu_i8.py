"""8-bit rows and the expert GEMMs over them against the float64 reference.

Bars.  Quantized rows and scales: bit-exact.  The int32 sums are exact, so a down row has one
rounding to fp32, and one for each factor: 4 * 2^-24, plus the output type's half step.  H adds the
fast exponential ((2 + 1.2 |g|) steps) and division (2 steps): under 2^-17 for |g| < 32, next to
bf16's half step 2^-8.
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
    torch.cuda.empty_cache()


def _M():
    from routing_dispatch_expert_moe_b200 import moe as M
    return M


def _ok():
    torch.cuda.synchronize()
    assert _M().moe_get_device_error() == 0


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 512), (7, 528), (5, 1040), (33, 2048), (4, 4112), (2, 7168),
                                       (3, 8208), (2, 16384), (4000, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows(rows, cols, dtype):
    M = _M()
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(dtype)
    q, s = M.moe_quantize_rows_i8(x.cuda())
    _ok()
    wq, ws = B.quantize_rows(x.float().numpy())
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


def test_quantize_special_rows():
    M = _M()
    x = torch.randn(9, 64)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 63] = float("nan")
    x[3] = 1e-45                                             # the smallest subnormal: scale 0
    x[4] = 3.4e38
    x[5, 1:] = 0.0
    x[6] = -0.0
    x[7, 9] = float("-inf")
    x[8] = 1e-38
    q, s = M.moe_quantize_rows_i8(x.cuda())
    _ok()
    wq, ws = B.quantize_rows(x.numpy())
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)


@pytest.mark.parametrize("cols", [128, 2048, 7168])
def test_quantize_fused_with_the_dispatch(cols):
    M = _M()
    T, k = 37, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, cols, device="cuda", generator=g).bfloat16()
    row_of = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32).view(T, k)
    row_of[3, 2] = row_of[7, 0] = -1
    row_of[9] = -1
    q = torch.full((T * k, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T * k,), -5.0, device="cuda")
    M.moe_quantize_rows_i8(x, row_of, T * k, q, s)
    _ok()
    q0, s0 = M.moe_quantize_rows_i8(x)
    wq = torch.full_like(q, 99)
    ws = torch.full_like(s, -5.0)
    t, j = (row_of >= 0).nonzero(as_tuple=True)
    wq[row_of[t, j].long()] = q0[t]
    ws[row_of[t, j].long()] = s0[t]
    assert torch.equal(q, wq) and torch.equal(s, ws)         # rows nothing goes to are left alone
    row_of[0, 0] = T * k                                     # past the buffer: skipped and recorded
    M.moe_quantize_rows_i8(x, row_of, T * k, q, s)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 3


def _experts(E, counts, N, K, seed, spare=3):
    rng = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(offsets[-1]) + spare
    q = rng.integers(-127, 128, (rows, K)).astype(np.int8)
    scale = ((rng.random(rows) + 0.5) * 1e-2).astype(np.float32)
    W = rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    ws = ((rng.random((E, N)) + 0.5) * (2e-2 / np.sqrt(K))).astype(np.float32)
    return offsets, rows, q, scale, W, ws


COUNTS = [[1], [0, 0, 5], [33, 0, 1, 129, 64], [300, 2, 0, 257], [1100], [7] * 40]
DIMS = [(128, 128), (144, 160), (512, 256), (1040, 272), (256, 1040)]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("d,F", DIMS)
@pytest.mark.parametrize("tiles", ["auto", "tokens", "weights"])
def test_gate_up(counts, d, F, tiles, monkeypatch):
    M = _M()
    if tiles != "auto":
        monkeypatch.setenv("MOE_B200_EXPERT_TILES", tiles)
    E = len(counts)
    off, rows, q, s, W, ws = _experts(E, counts, 2 * F, d, [d, F, E])
    h = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
    c = lambda a: torch.from_numpy(a).cuda()
    M.moe_expert_gate_up_i8(c(q), c(s), c(off), c(W), c(ws), rows, h=h)
    _ok()
    want = B.gate_up_i8(q, s, off, W, ws)
    got = h.double().cpu().numpy()
    n = int(off[-1])
    assert (got[n:] == 7.0).all()                            # rows behind the last expert's stay
    assert (np.abs(got[:n] - want[:n]) <= np.abs(want[:n]) * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()


@pytest.mark.parametrize("d,F", DIMS)
def test_gate_up_in_pairs(d, F, monkeypatch):
    M = _M()
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", "tokens")
    monkeypatch.setenv("MOE_B200_TOKEN_TILES", "pairs")
    off, rows, q, s, W, ws = _experts(3, [300, 1, 511], 2 * F, d, 3)
    c = lambda a: torch.from_numpy(a).cuda()
    h = M.moe_expert_gate_up_i8(c(q), c(s), c(off), c(W), c(ws), rows)
    _ok()
    want, n = B.gate_up_i8(q, s, off, W, ws), int(off[-1])
    assert (np.abs(h.double().cpu().numpy()[:n] - want[:n]) <= np.abs(want[:n]) * (2.0 ** -8 + 2.0 ** -17) + 1e-30).all()


@pytest.mark.parametrize("d,F", DIMS)
def test_gate_up_gathered_equals_permuted(d, F, monkeypatch):
    M = _M()
    T = 61
    off, rows, _, _, W, ws = _experts(4, [50, 0, 131, 9], 2 * F, d, 5, spare=0)
    g = torch.Generator(device="cuda").manual_seed(2)
    xq = torch.randint(-127, 128, (T, d), dtype=torch.int8, device="cuda", generator=g)
    xs = torch.rand(T, device="cuda", generator=g) * 1e-2
    tok = torch.randint(0, T, (rows,), dtype=torch.int32, device="cuda", generator=g)
    c = lambda a: torch.from_numpy(a).cuda()
    a = M.moe_expert_gate_up_i8(xq, xs, c(off), c(W), c(ws), rows, token_of_row=tok)
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", "weights")
    b = M.moe_expert_gate_up_i8(xq[tok.long()].contiguous(), xs[tok.long()].contiguous(), c(off), c(W), c(ws), rows)
    _ok()
    assert torch.equal(a, b)


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("d,F", DIMS)
@pytest.mark.parametrize("tiles", ["tokens", "weights", "pairs"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_down(counts, d, F, tiles, dtype, monkeypatch):
    M = _M()
    monkeypatch.setenv("MOE_B200_EXPERT_TILES", "weights" if tiles == "weights" else "tokens")
    monkeypatch.setenv("MOE_B200_TOKEN_TILES", "pairs" if tiles == "pairs" else "single")
    E = len(counts)
    off, rows, q, s, W, ws = _experts(E, counts, d, F, [d, F, E, 1])
    gate = np.random.default_rng(1).random(rows).astype(np.float32)
    c = lambda a: torch.from_numpy(a).cuda()
    for g in (None, gate):
        y = torch.full((rows, d), 7.0, dtype=dtype, device="cuda")
        M.moe_expert_down_i8(c(q), c(s), c(off), c(W), c(ws), rows, None if g is None else c(g), y_rows=y)
        _ok()
        want, n = B.down_i8(q, s, off, W, ws, g), int(off[-1])
        got = y.double().cpu().numpy()
        assert (got[n:] == 7.0).all()
        tol = 4 * U + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
        assert (np.abs(got[:n] - want[:n]) <= np.abs(want[:n]) * tol).all()


def test_largest_sums_are_exact():
    """Every product at its largest, at the longest row: 16384 * 127^2 = 2^27.98."""
    M = _M()
    K, d = 16384, 128
    q = torch.full((5, K), 127, dtype=torch.int8, device="cuda")
    q[1] = -127
    q[2, 1:] = 0
    W = torch.full((1, d, K), -127, dtype=torch.int8, device="cuda")
    one = torch.ones(5, device="cuda")
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    y = M.moe_expert_down_i8(q, one, off, W, torch.ones(1, d, device="cuda"), 5)
    _ok()
    want = torch.tensor([-1.0, 1.0, 0.0, -1.0, -1.0], dtype=torch.float64) * (K * 127 * 127)
    want[2] = -127 * 127
    assert torch.equal(y.cpu(), want.float()[:, None].expand(5, d))


def test_a_poisoned_row_spoils_only_itself():
    M = _M()
    x = torch.randn(40, 256, device="cuda").bfloat16()
    x[7, 100] = float("nan")
    x[20, 5] = float("inf")
    W, ws = M.quantize_experts_i8(torch.randn(2, 256, 256, device="cuda") * 0.05)
    off = torch.tensor([0, 30, 40], dtype=torch.int32, device="cuda")
    q, s = M.moe_quantize_rows_i8(x)
    h = M.moe_expert_gate_up_i8(q, s, off, W, ws, 40)
    _ok()
    bad = torch.isnan(h).any(1)
    assert bad[7] and bad[20] and int(bad.sum()) == 2
    assert torch.isnan(h[7]).all()


def test_bad_tokens_and_offsets_are_recorded():
    M = _M()
    T, d, F = 8, 128, 128
    xq = torch.ones((T, d), dtype=torch.int8, device="cuda")
    xs = torch.ones(T, device="cuda")
    W = torch.ones((1, 2 * F, d), dtype=torch.int8, device="cuda")
    ws = torch.full((1, 2 * F), 1e-3, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    tok = torch.tensor([0, 99, -1, 3], dtype=torch.int32, device="cuda")
    M.moe_expert_gate_up_i8(xq, xs, off, W, ws, 4, token_of_row=tok)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 3
    M.moe_expert_gate_up_i8(xq, xs, torch.tensor([0, 9], dtype=torch.int32, device="cuda"), W, ws, 8)
    torch.cuda.synchronize()
    assert M.moe_get_device_error() == 3


def test_nothing_to_do():
    M = _M()
    W = torch.ones((2, 256, 128), dtype=torch.int8, device="cuda")
    ws = torch.ones((2, 256), device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 128), dtype=torch.int8, device="cuda")
    h = M.moe_expert_gate_up_i8(e, torch.empty(0, device="cuda"), off, W, ws, 0)
    assert h.shape == (0, 128)
    x = torch.ones((4, 128), dtype=torch.int8, device="cuda")
    h = torch.full((4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_gate_up_i8(x, torch.ones(4, device="cuda"), off, W, ws, 4, h=h)   # rows, but no expert has one
    q, s = M.moe_quantize_rows_i8(torch.empty((0, 64), device="cuda"))
    _ok()
    assert (h == 3.0).all() and q.shape == (0, 64) and s.shape == (0,)


def test_refusals():
    M = _M()
    W = torch.ones((2, 256, 128), dtype=torch.int8, device="cuda")
    ws = torch.ones((2, 256), device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, xs = torch.ones((4, 128), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        M.moe_expert_gate_up_i8(x.float(), xs, off, W, ws, 4)
    with pytest.raises(ValueError):
        M.moe_expert_gate_up_i8(x, xs, off, W, ws, 5)        # rows_max beyond the rows
    with pytest.raises(ValueError):
        M.moe_expert_gate_up_i8(x, xs[:3], off, W, ws, 4)
    with pytest.raises(ValueError):
        M.moe_expert_gate_up_i8(x, xs, off, W, ws[:, :100].contiguous(), 4)
    with pytest.raises(ValueError):
        M.moe_expert_gate_up_i8(x[:, ::2], xs, off, W, ws, 4)
    with pytest.raises(M.MoEError):                          # rows shorter than one k-block
        M.moe_expert_down_i8(torch.ones((4, 64), dtype=torch.int8, device="cuda"), xs, off,
                             torch.ones((2, 128, 64), dtype=torch.int8, device="cuda"),
                             torch.ones((2, 128), device="cuda"), 4)
    with pytest.raises(M.MoEError):
        M.moe_quantize_rows_i8(torch.ones((2, 24), device="cuda"))


def test_graph_replay_and_other_stream():
    M = _M()
    g0 = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(100, 256, device="cuda", generator=g0).bfloat16()
    W, ws = M.quantize_experts_i8(torch.randn(3, 512, 256, device="cuda", generator=g0))
    off = torch.tensor([0, 10, 60, 100], dtype=torch.int32, device="cuda")

    def step(v):
        q, s = M.moe_quantize_rows_i8(v)
        return M.moe_expert_gate_up_i8(q, s, off, W, ws, 100)

    want = step(x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = step(x)
    st.synchronize()
    assert torch.equal(got, want)
    buf = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(buf)
    buf.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    _ok()


def test_unsafe_or_ambiguous_arguments():
    M = _M()
    x = torch.ones((4, 64), device="cuda")
    with pytest.raises(ValueError):                          # no slot: would pass for "no dispatch"
        M.moe_quantize_rows_i8(x, torch.empty((4, 0), dtype=torch.int32, device="cuda"), 1)
    with pytest.raises(ValueError):
        M.moe_quantize_rows_i8(x, torch.zeros(4, dtype=torch.int32, device="cuda"), 4)
    with pytest.raises(ValueError):                          # an odd number of weight rows
        M.moe_expert_gate_up_i8(torch.ones((4, 128), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"),
                                torch.zeros(2, dtype=torch.int32, device="cuda"),
                                torch.ones((1, 257, 128), dtype=torch.int8, device="cuda"),
                                torch.ones((1, 257), device="cuda"), 4)
