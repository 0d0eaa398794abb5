"""Plain float64 references of the group-limited routing and its gradient, the 8-bit expert
products, and the norms around a block with their gradients.

Written from the formulas, one token or one expert at a time; shares no code with the library.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ routing by groups
def _clean(l):
    """NaN counts as masked (-inf), +inf as the largest float32."""
    l = np.asarray(l, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, float(np.finfo(np.float32).max))


def score_of(l, score: str):
    """Scores of one token's clean logits; 0 where masked."""
    l = np.asarray(l, np.float64)
    live = l > -np.inf
    s = np.zeros_like(l)
    if not live.any():
        return s
    v = l[live]
    if score == "softmax":
        e = np.exp(v - v.max())
        s[live] = e / e.sum()
    elif score == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-v))
    elif score == "sqrt_softplus":
        s[live] = np.sqrt(np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v))))
    else:
        raise ValueError(score)
    return s


def route_grouped(logits, k, n_groups, groups_kept, group_score="top2", score="sigmoid", renormalize=True, scale=1.0,
                  select_bias=None):
    """(idx [T, k], gates [T, k], margin [T]): margin is the smallest key distance that decides
    the token (the kept groups' border, and each pair of neighbours down to the first left out),
    relative to the largest finite key, score and bias of the row."""
    T, E = logits.shape
    n = E // n_groups
    idx = np.zeros((T, k), np.int64)
    gate = np.zeros((T, k))
    margin = np.full(T, np.inf)

    def gap(a, b):
        return np.inf if np.isinf(a) or np.isinf(b) else abs(a - b)

    for t in range(T):
        l = _clean(logits[t])
        live = l > -np.inf
        s = score_of(l, score)
        plus = s if select_bias is None else s + np.asarray(select_bias, np.float64)
        key = np.where(live, l if select_bias is None else plus, -np.inf)
        worth = []
        for g in range(n_groups):
            at = slice(g * n, (g + 1) * n)
            if not live[at].any():
                worth.append(-np.inf)
            elif group_score == "max":
                worth.append(key[at].max())
            else:
                worth.append(np.sort(plus[at][live[at]])[::-1][:2].sum())
        order = sorted(range(n_groups), key=lambda g: (-worth[g], g))
        if groups_kept < n_groups:
            margin[t] = gap(worth[order[groups_kept - 1]], worth[order[groups_kept]])
        pool = [e for g in sorted(order[:groups_kept]) for e in range(g * n, (g + 1) * n)]
        ranked = sorted(pool, key=lambda e: (-key[e], e))
        for a, b in zip(ranked[:k], ranked[1:k + 1]):
            margin[t] = min(margin[t], gap(key[a], key[b]))
        idx[t] = ranked[:k]
        size = np.abs(np.concatenate([key[live], s[live], [] if select_bias is None else select_bias, [1e-300]])).max()
        margin[t] /= size
        if score == "softmax" and renormalize:
            q = score_of(l[idx[t]], "softmax")
        else:
            q = s[idx[t]]
            if renormalize:
                q = q / q.sum() if q.sum() > 0 else np.zeros(k)
        gate[t] = q * scale
    return idx, gate, margin


def routing_loss(logits, topk_idx, d_gate, score, renormalize, scale, load, aux_coef, z_coef):
    """The scalar whose gradient moe_route_backward gives: sum(gates * d_gate) + aux_coef * aux +
    z_coef * z, for finite logits."""
    T, E = logits.shape
    total = 0.0
    P = np.zeros(E)
    for t in range(T):
        l = _clean(logits[t])
        s = score_of(l, score)
        if d_gate is not None:
            i = topk_idx[t]
            if score == "softmax" and renormalize:
                q = score_of(l[i], "softmax")
            else:
                q = s[i] / (s[i].sum() if renormalize else 1.0)
            total += scale * float(q @ np.asarray(d_gate[t], np.float64))
        P += s / s.sum() / T
        m = l.max()
        total += z_coef * (m + np.log(np.exp(l - m).sum())) ** 2 / T
    if aux_coef:
        total += aux_coef * E * float(P @ np.asarray(load, np.float64))
    return total


def route_backward(logits, topk_idx, d_gate, score, renormalize, scale, load=None, aux_coef=0.0, z_coef=0.0):
    """Gradient of routing_loss by the logits; masked logits have gradient 0."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = _clean(logits[t])
        live = l > -np.inf
        if not live.any():
            continue
        s = score_of(l, score)
        p = score_of(l, "softmax")
        sig = score_of(l, "sigmoid")
        # J[a, b] = d s_a / d l_b
        if score == "softmax":
            J = np.diag(p) - np.outer(p, p)
        elif score == "sigmoid":
            J = np.diag(sig * (1.0 - sig))
        else:
            with np.errstate(divide="ignore", invalid="ignore"):
                J = np.diag(np.where(s > 0, sig / (2.0 * s), 0.0))
        ds = np.zeros(E)                       # dL / ds
        if d_gate is not None:
            i = topk_idx[t]
            u = np.where(live[i], scale * np.asarray(d_gate[t], np.float64), 0.0)   # a masked slot's is not used
            if score == "softmax" and renormalize:
                q = score_of(l[i], "softmax")
                np.add.at(out[t], i, q * (u - q @ u))
            else:
                si = s[i]
                if renormalize:
                    S = si.sum()
                    if S > 0:
                        np.add.at(ds, i, u / S - (si @ u) / S ** 2)
                else:
                    np.add.at(ds, i, u)
        if aux_coef:
            f, S = np.asarray(load, np.float64), s.sum()
            if S > 0:
                ds += aux_coef * E / T * (f / S - (s @ f) / S ** 2)
        out[t] += J.T @ ds
        m = l.max()
        lse = m + np.log(np.exp(l - m).sum())
        out[t] += 2.0 * z_coef / T * lse * p
        out[t][~live] = 0.0
    return out


# ------------------------------------------------------------------ 8-bit rows and products
def quantize_rows(x):
    """(q int8, scale) by the definition's float32 steps."""
    x = np.asarray(x, np.float32)
    q = np.zeros(x.shape, np.int8)
    scale = np.zeros(x.shape[0], np.float32)
    for r in range(x.shape[0]):
        if not np.isfinite(x[r]).all():
            scale[r] = np.nan
            continue
        a = np.abs(x[r]).max()
        if a >= 2.0 ** -120:                     # 127 / a stays finite
            scale[r] = a / np.float32(127.0)
            f = np.float32(127.0) * (np.float32(1.0) / a)
            q[r] = np.rint(x[r] * f).astype(np.int8)
    return q, scale


def gate_up_i8(q, scale, offsets, W, w_scale):
    """H [rows, F] (float64) of the rows that belong to an expert, NaN elsewhere."""
    E, F2, _ = W.shape
    F = F2 // 2
    out = np.full((q.shape[0], F), np.nan)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        acc = q[a:b].astype(np.float64) @ W[e].astype(np.float64).T
        v = acc * scale[a:b, None].astype(np.float64) * w_scale[e].astype(np.float64)
        g, u = v[:, :F], v[:, F:]
        with np.errstate(over="ignore"):
            out[a:b] = g / (1.0 + np.exp(-g)) * u
    return out


def down_i8(q, scale, offsets, W, w_scale, gate=None):
    E, d, _ = W.shape
    out = np.full((q.shape[0], d), np.nan)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        acc = q[a:b].astype(np.float64) @ W[e].astype(np.float64).T
        out[a:b] = acc * scale[a:b, None].astype(np.float64) * w_scale[e].astype(np.float64)
        if gate is not None:
            out[a:b] *= gate[a:b, None].astype(np.float64)
    return out


# ------------------------------------------------------------------ norms around a block
def block_norm(residual, y=None, post=None, gate=None, alpha=1.0, pre=None, eps=1e-6):
    """(x', n or None) in float64; gate [G, d]."""
    r = np.asarray(residual, np.float64)
    T, d = r.shape
    x = alpha * r
    if y is not None:
        b = np.asarray(y, np.float64)
        if post is not None:
            b = np.asarray(post, np.float64) * b / np.sqrt((b * b).mean(1, keepdims=True) + eps)
        if gate is not None:
            b = b * np.repeat(np.asarray(gate, np.float64), T // gate.shape[0], axis=0)
        x = x + b
    n = None if pre is None else np.asarray(pre, np.float64) * x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    return x, n


def combine_sum(y_rows, row_of, topk_gate=None, shared_y=None):
    T, k = row_of.shape
    out = np.zeros((T, y_rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if row_of[t, j] >= 0:
                out[t] += (1.0 if topk_gate is None else float(topk_gate[t, j])) * y_rows[row_of[t, j]].astype(
                    np.float64)
        if shared_y is not None:
            out[t] += shared_y[t]
    return out


def _rms_grad(g, v, eps):
    """Gradient by v of sum(g * v / rms(v))."""
    r = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    vh = v * r
    return r * (g - vh * (g * vh).mean(1, keepdims=True))


def block_norm_backward(d_x, d_n, x_out, y=None, post=None, gate=None, alpha=1.0, pre=None, eps=1e-6):
    """dict of the gradients in float64, from the saved x_out and y."""
    f = lambda a: None if a is None else np.asarray(a, np.float64)
    d_x, d_n, x, y, post, gate, pre = map(f, (d_x, d_n, x_out, y, post, gate, pre))
    T, d = x.shape
    u = np.zeros((T, d)) if d_x is None else d_x.copy()
    out = dict(d_y=None, d_post_weight=None, d_gate=None, d_pre_weight=None)
    if pre is not None:
        xh = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
        out["d_pre_weight"] = (d_n * xh).sum(0)
        u += _rms_grad(d_n * pre, x, eps)
    out["d_residual"] = alpha * u
    if y is not None:
        yh = y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        b = y if post is None else yh * post
        ug = u
        if gate is not None:
            out["d_gate"] = (u * b).reshape(gate.shape[0], -1, d).sum(1)
            ug = u * np.repeat(gate, T // gate.shape[0], axis=0)
        if post is None:
            out["d_y"] = ug
        else:
            out["d_post_weight"] = (ug * yh).sum(0)
            out["d_y"] = _rms_grad(ug * post, y, eps)
    return out
