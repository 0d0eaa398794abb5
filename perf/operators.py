"""The routing, 8-bit and block-norm operators as they are measured: cases, inputs, plain forms.

Six operators, each with a small case where latency counts and a large one:

  route        group-limited top-k of router logits with gates (moe_route_grouped)
  route_grad   gradient of gates, load-balance loss and z-loss by the logits (moe_route_backward)
  gate_up_i8   bf16 expert rows -> 8-bit rows -> grouped gate/up product with SwiGLU
  down_i8      bf16 hidden rows -> 8-bit rows -> grouped down product times the row's gate
  norm         post-norm, gate, scaled residual and the next pre-norm, after a combine or a plain branch
  norm_grad    its gradients, those of the weights and of the broadcast gate among them

With `own` false, run() computes them by elementary torch operations in 32 bits (the selection
keys of the router in 64, where neighbours decide); with `own` true it calls the library.
"""
import math

import torch

own = False

_GROUP_SCORES = ("max", "top2")
_SCORES = ("softmax", "sigmoid", "sqrt_softplus")


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # decoding: four tokens of a 256-expert router with a balance bias, groups by their best two
        dict(name="route_decode", op="route", T=4, E=256, k=8, groups=8, kept=4, group_score="top2",
             score="sigmoid", renorm=True, bias=True, masked=0.0),
        # prefill of the 896-expert layer, a few experts switched off by a logit of minus infinity
        dict(name="route_prefill", op="route", T=32768, E=896, k=16, groups=16, kept=4, group_score="top2",
             score="sqrt_softplus", renorm=True, bias=True, masked=0.02),
        # a training step of the 64-expert layer: softmax gates, load-balance loss and z-loss
        dict(name="route_grad_64", op="route_grad", T=8192, E=64, k=8, score="softmax", renorm=True,
             aux=0.01, z=0.001),
        # a training step of the 896-expert layer: sigmoid gates and the load-balance loss
        dict(name="route_grad_896", op="route_grad", T=32768, E=896, k=16, score="sigmoid", renorm=True,
             aux=0.01, z=0.0),
        # decoding a batch of 16 tokens: most experts hold two rows, the weights are the work
        dict(name="gate_up_i8_decode", op="gate_up_i8", T=16, E=64, k=8, d=2048, F=1024),
        # prefill of the 64-expert layer: a thousand rows an expert, the products are the work
        dict(name="gate_up_i8_prefill", op="gate_up_i8", T=8192, E=64, k=8, d=2048, F=1024),
        # a ragged small batch with fp32 rows out
        dict(name="down_i8_ragged", op="down_i8", T=37, E=64, k=8, d=2048, F=1024, out="f32"),
        # the 896-expert layer's narrow experts, 146 rows each on average
        dict(name="down_i8_896", op="down_i8", T=8192, E=896, k=16, d=7168, F=256, out="bf16"),
        # decoding: seven tokens of a wide fp32 residual stream after a plain branch
        dict(name="norm_decode", op="norm", T=7, d=7168, k=0, G=1, alpha=1.0, y="bf16", r="f32", n="bf16",
             post=True, pre=True, dropped=0.0),
        # prefill of the 64-expert layer: the sum over eight expert rows, four sequences' gates
        dict(name="norm_combine", op="norm", T=8192, d=2048, k=8, G=4, alpha=0.5, y="bf16", r="bf16", n="bf16",
             post=True, pre=True, dropped=0.05),
        # gradients of that block, one gate for all tokens
        dict(name="norm_grad_2048", op="norm_grad", T=8192, d=2048, G=1, alpha=0.5, y="bf16", r="bf16", n="bf16",
             post=True, pre=True),
        # gradients at the widest rows, fp32 residual stream, 16 sequences' gates
        dict(name="norm_grad_7168", op="norm_grad", T=4096, d=7168, G=16, alpha=1.0, y="bf16", r="f32", n="bf16",
             post=True, pre=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "route_grad", "gate_up_i8", "down_i8", "norm", "norm_grad"))
    if op == "route":
        groups = rng.choice((1, 2, 3, 4, 6, 8, 16, 28))
        E = groups * _log(rng, 1 if groups > 8 else 4, 1024 // groups)
        kept = rng.randint(1, groups)
        k = min(_log(rng, 1, 16), kept * (E // groups))
        T = _log(rng, 1, min(32768, 32768 * 896 // E))
        return dict(op=op, T=T, E=E, k=k, groups=groups, kept=kept, group_score=rng.choice(_GROUP_SCORES),
                    score=rng.choice(_SCORES), renorm=rng.random() < 0.7, bias=rng.random() < 0.6,
                    masked=rng.choice((0.0, 0.02)))
    if op == "route_grad":
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, min(32768, 32768 * 896 // E))
        return dict(op=op, T=T, E=E, k=min(_log(rng, 1, 16), E), score=rng.choice(_SCORES),
                    renorm=rng.random() < 0.7, aux=rng.choice((0.0, 0.01)), z=rng.choice((0.0, 0.001)))
    if op in ("gate_up_i8", "down_i8"):
        while True:
            E, k = _log(rng, 4, 896), rng.choice((1, 2, 4, 6, 8, 16))
            d, F, T = 16 * _log(rng, 8, 448), 16 * _log(rng, 8, 128), _log(rng, 1, 8192)
            # no dearer than the listed prefill (its products) and the 896-expert weights
            if k <= E and T * k * d * F <= 65536 * 2048 * 1024 and E * d * F <= 896 * 7168 * 256 // 4:
                break
        case = dict(op=op, T=T, E=E, k=k, d=d, F=F)
        if op == "down_i8":
            case["out"] = rng.choice(("bf16", "f32"))
        return case
    G = rng.choice((1, 1, 2, 3, 5, 16))
    d = 8 * _log(rng, 8, 1024)
    per = _log(rng, 1, max(1, min(16384, 8192 * 2048 // d) // G))
    if rng.random() < 0.15:
        G, per = G * per, 1                      # a gate for every token
    case = dict(op=op, T=G * per, d=d, G=G, alpha=rng.choice((1.0, 0.5)), y=rng.choice(("bf16", "bf16", "f32")),
                r=rng.choice(("bf16", "f32")), n=rng.choice(("bf16", "bf16", "f32")), post=rng.random() < 0.8,
                pre=rng.random() < 0.8)
    if op == "norm":
        case["k"] = rng.choice((0, 1, 2, 4, 8))
        case["dropped"] = rng.choice((0.0, 0.1))
    return case


# ------------------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _routing(case, g):
    """Expert-contiguous rows of a skewed batch: counts after a capacity factor of 2, their
    offsets, and (for the padded plain form) the largest count."""
    E, rows = case["E"], case["T"] * case["k"]
    w = torch.exp(0.5 * torch.randn(E, generator=g, dtype=torch.float64))
    share = rows * w / w.sum()
    counts = share.floor().long()
    rest = rows - int(counts.sum())
    counts += torch.bincount(torch.randint(0, E, (rest,), generator=g), minlength=E)
    counts = counts.clamp(max=max(1, -(-2 * rows // E)))
    off = torch.zeros(E + 1, dtype=torch.int64)
    off[1:] = counts.cumsum(0)
    return off.to(torch.int32).cuda(), int(counts.max())


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]

    def rnd(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    if op in ("route", "route_grad"):
        E, k = case["E"], case["k"]
        # logits of a trained router: unit spread over the tokens, half a unit between experts
        logits = rnd(T, E) + rnd(E, scale=0.5)
        s = dict(case=case, logits=logits)
        if op == "route":
            if case["masked"]:
                off = torch.rand(E, generator=gen, device="cuda") < case["masked"]
                logits.masked_fill_(off, -math.inf)
            s["bias"] = rnd(E, scale=0.05) if case["bias"] else None
            return s
        s["topk_idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
        s["d_gate"] = rnd(T, k, scale=0.1)
        counts = torch.bincount(s["topk_idx"].reshape(-1).long(), minlength=E)
        s["load"] = (counts.double() / (T * k)).float() if case["aux"] else None
        return s

    if op in ("gate_up_i8", "down_i8"):
        E, d, F, rows = case["E"], case["d"], case["F"], T * case["k"]
        off, most = _routing(case, g)
        n, K = (2 * F, d) if op == "gate_up_i8" else (d, F)
        W = torch.empty((E, n, K), dtype=torch.int8, device="cuda")
        for e in range(0, E, 64):                # in pieces: the fp32 draws are four times the weights
            W[e:e + 64] = rnd(min(64, E - e), n, K, scale=36.0).round_().clamp_(-127, 127).to(torch.int8)
        ws = torch.rand((E, n), generator=gen, device="cuda") * 2e-4 + 5e-4
        s = dict(case=case, offsets=off, most=most, W=W, w_scale=ws, rows_max=rows)
        s["x"] = rnd(rows, K, dtype=torch.bfloat16)
        if op == "gate_up_i8":
            s["out"] = torch.zeros((rows, F), dtype=torch.bfloat16, device="cuda")
        else:
            s["gate"] = torch.rand((rows,), generator=gen, device="cuda") * 0.25
            s["out"] = torch.zeros((rows, d), dtype=_DT[case["out"]], device="cuda")
        return s

    d, G = case["d"], case["G"]
    s = dict(case=case)
    s["post"] = rnd(d, scale=0.1, shift=1.0) if case["post"] else None
    s["pre"] = rnd(d, scale=0.1, shift=1.0) if case["pre"] else None
    s["gate"] = rnd(G, d, scale=0.2, shift=0.5)
    if op == "norm":
        s["r"] = rnd(T, d, dtype=_DT[case["r"]], scale=2.0)
        k = case["k"]
        if k:
            perm = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).reshape(T, k)
            drop = torch.rand((T, k), generator=gen, device="cuda") < case["dropped"]
            s["row_of"] = torch.where(drop, torch.full_like(perm, -1), perm).contiguous()
            s["y"] = rnd(T * k, d, dtype=_DT[case["y"]], scale=0.2)
        else:
            s["y"] = rnd(T, d, dtype=_DT[case["y"]], scale=0.5)
        return s
    s["x_out"] = rnd(T, d, dtype=_DT[case["r"]], scale=2.0)
    s["y"] = rnd(T, d, dtype=_DT[case["y"]], scale=0.5)
    s["d_x"] = rnd(T, d, dtype=_DT[case["r"]], scale=0.01)
    s["d_n"] = rnd(T, d, dtype=_DT[case["n"]], scale=0.01) if case["pre"] else None
    return s


# ------------------------------------------------------------------------------ the passes
EPS = 1e-6


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from routing_dispatch_expert_moe_b200 import moe as M

        if op == "route":
            return M.moe_route_grouped(s["logits"], case["k"], case["groups"], case["kept"], case["group_score"],
                                       case["score"], case["renorm"], 1.0, s["bias"])
        if op == "route_grad":
            return M.moe_route_backward(s["logits"], s["topk_idx"], s["d_gate"], case["score"], case["renorm"], 1.0,
                                        s["load"], case["aux"], case["z"])
        if op == "gate_up_i8":
            q, qs = M.moe_quantize_rows_i8(s["x"])
            return M.moe_expert_gate_up_i8(q, qs, s["offsets"], s["W"], s["w_scale"], s["rows_max"], h=s["out"])
        if op == "down_i8":
            q, qs = M.moe_quantize_rows_i8(s["x"])
            return M.moe_expert_down_i8(q, qs, s["offsets"], s["W"], s["w_scale"], s["rows_max"], s["gate"],
                                        y_rows=s["out"])
        if op == "norm":
            args = dict(post_weight=s["post"], gate=s["gate"], alpha=case["alpha"], pre_weight=s["pre"], eps=EPS,
                        n_dtype=_DT[case["n"]])
            if case["k"]:
                out = M.moe_combine_norm(s["r"], s["y"], s["row_of"], s["y"].shape[0], **args)
            else:
                out = M.moe_block_norm(s["r"], s["y"], **args)
            return [t for t in out if t is not None]
        out = M.moe_block_norm_backward(s["d_x"], s["d_n"], s["x_out"], s["y"], post_weight=s["post"],
                                        gate=s["gate"], alpha=case["alpha"], pre_weight=s["pre"], eps=EPS)
        return {key: v for key, v in out.items() if v is not None}
    return {"route": _route, "route_grad": _route_grad, "gate_up_i8": _gate_up, "down_i8": _down, "norm": _norm,
            "norm_grad": _norm_grad}[op](s)


def _score64(l, score):
    """Scores in 64 bits: two experts next to the border between chosen and not differ by less
    than 32 bits hold."""
    l = l.double()
    if score == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        return e / e.sum(1, keepdim=True).clamp_min(1e-300)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    return torch.sqrt(l.clamp_min(0.0) + torch.log1p(torch.exp(-l.abs())))


def _route(s):
    case, l = s["case"], s["logits"]
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    n = E // G
    off = torch.isinf(l)
    low = torch.tensor(-math.inf, device=l.device, dtype=torch.float64)
    sc = _score64(l, case["score"])
    value = sc if s["bias"] is None else sc + s["bias"].double()
    key = torch.where(off, low, l.double() if s["bias"] is None else value)
    if case["group_score"] == "max":
        of_group = key.view(T, G, n).amax(2)
    else:
        two = torch.sort(torch.where(off, low, value).view(T, G, n), dim=2, descending=True).values[:, :, :2]
        of_group = torch.where(torch.isinf(two[:, :, :1]), low, torch.where(torch.isinf(two), 0.0, two)
                               .sum(2, keepdim=True)).squeeze(2)
    # stable: of equal values the lower index comes first
    keep = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :case["kept"]].sort(1).values
    cand = (keep.unsqueeze(2) * n + torch.arange(n, device=l.device)).view(T, -1)
    order = torch.sort(key.gather(1, cand), dim=1, descending=True, stable=True).indices[:, :k]
    idx = cand.gather(1, order)
    kept_l = l.gather(1, idx).double()
    dead = torch.isinf(kept_l)
    if case["score"] == "softmax" and case["renorm"]:
        m = kept_l.amax(1, keepdim=True)
        g = torch.exp(kept_l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    else:
        g = sc.gather(1, idx)
    g = torch.where(dead, torch.zeros_like(g), g)
    if case["renorm"]:
        tot = g.sum(1, keepdim=True)
        g = torch.where(tot > 0, g / tot, torch.zeros_like(g))
    return idx.to(torch.int32), g.float()


def _dscore(l, score):
    """Score and its derivative, fp32, for the two scores that act on one logit alone."""
    sig = torch.sigmoid(l)
    if score == "sigmoid":
        return sig, sig * torch.sigmoid(-l)
    root = torch.sqrt(l.clamp_min(0.0) + torch.log1p(torch.exp(-l.abs())))
    return root, sig / (2.0 * root)


def _route_grad(s):
    case, l, d_gate = s["case"], s["logits"], s["d_gate"]
    T, E = l.shape
    idx = s["topk_idx"].long()
    score, renorm = case["score"], case["renorm"]
    lse = torch.logsumexp(l, 1, keepdim=True)
    p = torch.exp(l - lse)
    out = torch.zeros_like(l)
    kept = l.gather(1, idx)
    if score == "softmax" and renorm:
        e = torch.exp(kept - kept.amax(1, keepdim=True))
        q = e / e.sum(1, keepdim=True)
        dk = q * (d_gate - (q * d_gate).sum(1, keepdim=True))
    elif score == "softmax":
        q = p.gather(1, idx)
        dk = q * d_gate
        out -= p * dk.sum(1, keepdim=True)
    else:
        sc, ds = _dscore(kept, score)
        if renorm:
            tot = sc.sum(1, keepdim=True)
            dk = ds * (d_gate - (sc * d_gate).sum(1, keepdim=True) / tot) / tot
        else:
            dk = ds * d_gate
    out.scatter_add_(1, idx, dk)
    if case["aux"]:
        f, c = s["load"], case["aux"] * E / T
        if score == "softmax":
            out += c * p * (f - (p * f).sum(1, keepdim=True))
        else:
            sc, ds = _dscore(l, score)
            tot = sc.sum(1, keepdim=True)
            out += c * ds * (f - (sc * f).sum(1, keepdim=True) / tot) / tot
    if case["z"]:
        out += case["z"] * 2.0 / T * lse * p
    return out


def _quantize(x):
    """Rows to 8 bits: 127 / amax as one factor, its inverse as the scale."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    f = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(x * f), (amax / 127.0).squeeze(1)


def _grouped(s):
    """Per-expert products of the quantized rows: sums of integers, [E, most, n] with the rows
    of each expert padded to the largest group, the place of each, and the row scales."""
    off, most, rows = s["offsets"].long(), s["most"], s["rows_max"]
    q, qs = _quantize(s["x"])
    at = off[:-1, None] + torch.arange(most, device=off.device)
    inside = at < off[1:, None]
    at = at.clamp(max=rows - 1)
    X = q[at.reshape(-1)].view(*at.shape, -1) * inside.unsqueeze(2)
    acc = torch.bmm(X, s["W"].float().transpose(1, 2))
    return acc * qs[at].unsqueeze(2) * s["w_scale"].unsqueeze(1), at, inside


def _gate_up(s):
    F = s["case"]["F"]
    a, at, inside = _grouped(s)
    g, u = a[:, :, :F], a[:, :, F:]
    h = torch.zeros((s["rows_max"], F), dtype=torch.bfloat16, device=a.device)
    h[at[inside]] = (g / (1.0 + torch.exp(-g)) * u)[inside].to(torch.bfloat16)
    return h


def _down(s):
    a, at, inside = _grouped(s)
    y = torch.zeros_like(s["out"])
    y[at[inside]] = (a * s["gate"][at].unsqueeze(2))[inside].to(y.dtype)
    return y


def _norm(s):
    case, r = s["case"], s["r"].float()
    T, d = r.shape
    y = s["y"].float()
    if case["k"]:
        row = s["row_of"].long()
        y = (y[row.clamp_min(0)] * (row >= 0).unsqueeze(2)).sum(1)
    if case["post"]:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["post"]
    x = case["alpha"] * r + (s["gate"].unsqueeze(1) * y.view(case["G"], -1, d)).view(T, d)
    out = [x.to(s["r"].dtype)]
    if case["pre"]:
        out.append((x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["pre"]).to(_DT[case["n"]]))
    return out


def _norm_grad(s):
    case = s["case"]
    x, y, dx = s["x_out"].float(), s["y"].float(), s["d_x"].float()
    T, d = x.shape
    G, out = case["G"], {}
    if case["pre"]:
        rs = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        xh, dn = x * rs, s["d_n"].float()
        out["d_pre_weight"] = (dn * xh).sum(0)
        w = dn * s["pre"]
        dx = dx + rs * (w - xh * (w * xh).mean(1, keepdim=True))
    out["d_residual"] = (case["alpha"] * dx).to(s["x_out"].dtype)
    if case["post"]:
        rs = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        yh = y * rs
        branch = yh * s["post"]
    else:
        branch = y
    out["d_gate"] = (dx * branch).view(G, -1, d).sum(1)
    u = (dx.view(G, -1, d) * s["gate"].unsqueeze(1)).view(T, d)
    if case["post"]:
        out["d_post_weight"] = (u * yh).sum(0)
        u = u * s["post"]
        u = rs * (u - yh * (u * yh).mean(1, keepdim=True))
    out["d_y"] = u.to(s["y"].dtype)
    return out


# ------------------------------------------------------------------------------ work
def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        # a score of some ten operations for every logit, and the comparisons
        return {"bytes": 4.0 * T * E + 8.0 * T * k + 4.0 * E * case["bias"], "flops": 16.0 * T * E}
    if op == "route_grad":
        E, k = case["E"], case["k"]
        return {"bytes": 8.0 * T * E + 8.0 * T * k + 4.0 * E, "flops": 16.0 * T * E}
    if op in ("gate_up_i8", "down_i8"):
        E, d, F, rows = case["E"], case["d"], case["F"], T * case["k"]
        touched = min(E, rows)                   # experts with rows: only their weights are read
        if op == "gate_up_i8":
            return {"bytes": rows * (2.0 * d + 2.0 * F) + touched * 2.0 * F * (d + 4.0),
                    "flops": 4.0 * rows * d * F}
        size = 4.0 if case["out"] == "f32" else 2.0
        return {"bytes": rows * (2.0 * F + size * d + 4.0) + touched * d * (F + 4.0), "flops": 2.0 * rows * d * F}
    size = {"bf16": 2.0, "f32": 4.0}
    d, w = case["d"], 4.0 * case["d"] * (case["G"] + case["post"] + case["pre"])
    if op == "norm":
        rows = T * case["k"] * (1.0 - case["dropped"]) if case["k"] else T
        n = rows * d * size[case["y"]] + 2.0 * T * d * size[case["r"]] + case["pre"] * T * d * size[case["n"]]
        return {"bytes": n + w + 4.0 * T * case["k"], "flops": 10.0 * T * d + rows * d}
    n = T * d * (3.0 * size[case["r"]] + 2.0 * size[case["y"]] + case["pre"] * size[case["n"]])
    return {"bytes": n + 2.0 * w, "flops": 24.0 * T * d}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad() if op not in ("route_grad", "norm_grad") else torch.enable_grad():
        return {"route": _exact_route, "route_grad": _exact_route_grad, "gate_up_i8": _exact_experts,
                "down_i8": _exact_experts, "norm": _exact_norm, "norm_grad": _exact_norm_grad}[op](s, case)


def _scores_of(l, score):
    if score == "softmax":
        return torch.softmax(l, 1)
    if score == "sigmoid":
        return torch.sigmoid(l)
    return torch.nn.functional.softplus(l, threshold=1e9).sqrt()


def _exact_route(s, case):
    l = s["logits"].double()
    T, E = l.shape
    G, n = case["groups"], E // case["groups"]
    dead = l == -math.inf
    sc = torch.nan_to_num(_scores_of(l, case["score"]), nan=0.0)
    plus = sc + (0.0 if s["bias"] is None else s["bias"].double())
    key = (l if s["bias"] is None else plus).masked_fill(dead, -math.inf)
    per = (key if case["group_score"] == "max" else plus.masked_fill(dead, -math.inf)).view(T, G, n)
    first = per.max(2)
    value = first.values
    if case["group_score"] == "top2" and n > 1:
        second = per.scatter(2, first.indices.unsqueeze(2), -math.inf).max(2).values
        value = value + torch.where(torch.isinf(second) | torch.isinf(value), torch.zeros_like(second), second)
    # one choice after another: argmax of what is left, the first among equals
    chosen = torch.zeros((T, G), dtype=torch.bool, device=l.device)
    place = torch.arange(G, device=l.device)
    for _ in range(case["kept"]):
        best = value.masked_fill(chosen, -math.inf).max(1, keepdim=True).values
        ok = ~chosen & ((value == best) | torch.isinf(best))
        at = torch.where(ok, place, G).min(1, keepdim=True).values
        chosen.scatter_(1, at, True)
    open_ = chosen.repeat_interleave(n, 1)
    place = torch.arange(E, device=l.device)
    idx = []
    for _ in range(case["k"]):
        best = key.masked_fill(~open_, -math.inf).max(1, keepdim=True).values
        at = torch.where(open_ & (key == best), place, E).min(1, keepdim=True).values
        idx.append(at)
        open_.scatter_(1, at, False)
    idx = torch.cat(idx, 1)
    kept = l.gather(1, idx)
    if case["score"] == "softmax" and case["renorm"]:
        g = torch.softmax(kept, 1)
    else:
        g = sc.gather(1, idx)
        g = g / g.sum(1, keepdim=True) if case["renorm"] else g
    return idx.to(torch.int32), torch.nan_to_num(g, nan=0.0)


def _exact_route_grad(s, case):
    l = s["logits"].double().requires_grad_(True)
    T, E = l.shape
    idx = s["topk_idx"].long()
    q = _scores_of(l, case["score"])
    if case["score"] == "softmax" and case["renorm"]:
        g = torch.softmax(l.gather(1, idx), 1)
    else:
        g = q.gather(1, idx)
        g = g / g.sum(1, keepdim=True) if case["renorm"] else g
    loss = (g * s["d_gate"].double()).sum()
    if case["aux"]:
        share = q / q.sum(1, keepdim=True)
        loss = loss + case["aux"] * E * (share.mean(0) * s["load"].double()).sum()
    if case["z"]:
        loss = loss + case["z"] * torch.logsumexp(l, 1).square().mean()
    return torch.autograd.grad(loss, l)[0]


def _exact_experts(s, case):
    if case["E"] * s["W"][0].numel() > 2 * 10 ** 9:
        return None
    off = s["offsets"].tolist()
    # the 8-bit rows are whole numbers, fixed by the definition: the row times the fp32 factor
    # 127 / amax in fp32, to the nearest even (half of amax is 63.5, so the factor's own
    # rounding decides); everything after them is in 64 bits
    x = s["x"].float()
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x * torch.where(amax > 0, 127.0 / amax, 0.0 * amax)).double()
    amax = amax.double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        v = (q[a:b] @ s["W"][e].double().T) * (amax[a:b] / 127.0) * s["w_scale"][e].double()
        if case["op"] == "gate_up_i8":
            v = torch.nn.functional.silu(v[:, :case["F"]]) * v[:, case["F"]:]
        else:
            v = v * s["gate"][a:b, None].double()
        out[a:b] = v
    return out


def _block64(case, r, y, post, gate, pre):
    T, d = r.shape
    if post is not None:
        y = y / torch.sqrt(y.pow(2).mean(1, keepdim=True) + EPS) * post
    x = case["alpha"] * r + y * gate.repeat_interleave(T // case["G"], 0)
    return x, None if pre is None else x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + EPS) * pre


def _wide(t):
    return None if t is None else t.double()


def _exact_norm(s, case):
    y = s["y"].double()
    if case["k"]:
        row = s["row_of"].long()
        tot = torch.zeros(s["r"].shape, dtype=torch.float64, device=y.device)
        for j in range(case["k"]):
            tot += torch.where(row[:, j:j + 1] >= 0, y[row[:, j].clamp_min(0)], 0.0)
        y = tot
    x, n = _block64(case, s["r"].double(), y, _wide(s["post"]), s["gate"].double(), _wide(s["pre"]))
    return [x] if n is None else [x, n]


def _exact_norm_grad(s, case):
    # the residual that gives the saved x_out, so that autograd passes through that very value
    names = ("y", "post", "gate", "pre")
    v = {n: None if s[n] is None else s[n].double().requires_grad_(True) for n in names}
    with torch.no_grad():
        r = torch.zeros(s["x_out"].shape, dtype=torch.float64, device="cuda")
        branch, _ = _block64(case, r, v["y"], v["post"], v["gate"], None)
        r = (s["x_out"].double() - branch) / case["alpha"]
    r.requires_grad_(True)
    x, n = _block64(case, r, v["y"], v["post"], v["gate"], v["pre"])
    loss = (x * s["d_x"].double()).sum()
    if n is not None:
        loss = loss + (n * s["d_n"].double()).sum()
    keys = [("d_residual", r), ("d_y", v["y"]), ("d_post_weight", v["post"]), ("d_gate", v["gate"]),
            ("d_pre_weight", v["pre"])]
    keys = [(name, t) for name, t in keys if t is not None]
    return {name: g for (name, _), g in zip(keys, torch.autograd.grad(loss, [t for _, t in keys]))}
