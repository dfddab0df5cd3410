"""Plain CPU oracle of the router, the 8-bit products and the layer for a few
tokens.

TEST INFRASTRUCTURE ONLY, like ``moe_oracle``: the definitions in float64
numpy, one expert or one token at a time, sharing nothing with the CUDA
library.  Results are not rounded to the storage dtype; the tests add the
rounding to their bounds.
"""

from __future__ import annotations

import numpy as np

__all__ = ["router_topk", "router_topk_grad", "quantize_rows", "linear_int8",
           "gate_up_swiglu_int8", "layer_few_tokens"]

F32_MAX = float(np.finfo(np.float32).max)


def _silu(x):
    return x * _sigmoid(x)


def _sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _clean(logits):
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    return np.minimum(l, F32_MAX)


def _scores(row, scoring: str):
    """Scores of one row of cleaned logits; masked (-inf) logits score 0."""
    if scoring == "sigmoid":
        return np.where(np.isneginf(row), 0.0, _sigmoid(np.where(np.isneginf(row), 0.0, row)))
    m = row.max()
    if np.isneginf(m):
        return np.zeros_like(row)
    e = np.exp(row - m)
    return e / e.sum()


def _log_scores(row):
    """log sigmoid, which does not underflow."""
    return np.minimum(row, 0.0) - np.log1p(np.exp(-np.abs(row)))


def _selected(row, sel, scoring: str, renormalize: bool):
    """Weights (before the scale) of the selected logits of one row."""
    if not renormalize:
        return _scores(row, scoring)[sel]
    s = row[sel] if scoring == "softmax" else _log_scores(np.maximum(row[sel], -F32_MAX))
    on = ~np.isneginf(row[sel])
    if not on.any():
        return np.zeros(len(sel))
    e = np.where(on, np.exp(np.where(on, s, 0.0) - s[on].max()), 0.0)
    return e / e.sum()


def router_topk(logits, K: int, scoring: str, renormalize: bool, scale: float):
    """(expert_ids [T, K], probs [T, K]): the K largest logits in descending
    order, ties to the lowest index, and their weights."""
    l = _clean(logits)
    T = l.shape[0]
    ids = np.zeros((T, K), dtype=np.int64)
    probs = np.zeros((T, K))
    for t in range(T):
        ids[t] = np.argsort(-l[t], kind="stable")[:K]
        probs[t] = scale * _selected(l[t], ids[t], scoring, renormalize)
    return ids, probs


def router_topk_grad(grad_probs, logits, expert_ids, scoring: str, renormalize: bool,
                     scale: float):
    """Gradient of sum(grad_probs * probs) by the logits, the selection held
    fixed, through the Jacobian of each token's weights."""
    l = _clean(logits)
    T, E = l.shape
    d = np.zeros((T, E))
    for t in range(T):
        sel = np.asarray(expert_ids[t])
        row = l[t]
        p = _scores(row, scoring)
        on = ~np.isneginf(row)
        if scoring == "softmax" and not renormalize:
            J = np.diag(p) - np.outer(p, p)                 # dp_i / dl_j
            d[t] = scale * np.asarray(grad_probs[t], dtype=np.float64) @ J[sel]
        else:
            q = _selected(row, sel, scoring, renormalize)
            slope = np.ones(len(sel)) if scoring == "softmax" else 1.0 - p[sel]  # d log p / dl
            if renormalize:
                J = (np.diag(q) - np.outer(q, q)) * slope[None, :]
            else:
                J = np.diag(q * slope)
            np.add.at(d[t], sel, scale * np.asarray(grad_probs[t], dtype=np.float64) @ J)
        d[t][~on] = 0.0
    return d


def quantize_rows(x):
    """(q, scale): q = rint(127 x / top), scale = top / 127 with top the row's
    largest magnitude; zeros for a row of zeros, NaN scale for a row that is
    not finite.  127 x and the quotient are float32 operations, which is exact
    enough to decide every tie of bfloat16 rows, and the definition for
    float32 rows."""
    x = np.asarray(x, dtype=np.float32)
    q = np.zeros(x.shape, dtype=np.int64)
    scale = np.zeros(x.shape[0], dtype=np.float32)
    for t, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scale[t] = np.nan
            continue
        top = np.max(np.abs(row)) if row.size else np.float32(0)
        if top == 0:
            continue
        scale[t] = top / np.float32(127)
        by = np.float32(2.0 ** -10 if top >= 2.0 ** 119 else 1.0)   # 127 x stays in range
        q[t] = np.rint(row * (np.float32(127) * by) / (top * by)).astype(np.int64)
    return q, scale


def linear_int8(q, row_scale, offsets, W_q, channel_scale):
    """y[i, n] = row_scale[i] channel_scale[e, n] sum_k q[i, k] W_q[e, n, k]
    for the rows i of expert e."""
    q = np.asarray(q, dtype=np.float64)
    E, Nout, _ = W_q.shape
    y = np.zeros((q.shape[0], Nout))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        s = q[lo:hi] @ np.asarray(W_q[e], dtype=np.float64).T      # exact integers
        y[lo:hi] = (np.asarray(row_scale[lo:hi], dtype=np.float64)[:, None] * s
                    * np.asarray(channel_scale[e], dtype=np.float64)[None, :])
    return y


def gate_up_swiglu_int8(q, row_scale, offsets, Wg_q, gs, Wu_q, us):
    """(act, g, u)."""
    g = linear_int8(q, row_scale, offsets, Wg_q, gs)
    u = linear_int8(q, row_scale, offsets, Wu_q, us)
    return _silu(g) * u, g, u


def layer_few_tokens(x, ids, probs, Wg, Wu, Wd, E: int, num_special: int = 0, mask=None,
                     shared=None, gs=None, us=None, ds=None):
    """(out [T, H], bound [T, H]).  bound: what fp32 sums in any order and one
    rounding of act to bfloat16 can add up to, without the rounding of out:
      dg  = (H + 4) 2^-24 sum |w x|,  du alike  (the scale's product included)
      dact <= |silu'(g) u| dg + |silu(g)| du + dg du + (2^-9 + 2^-20) |act|
              (silu' is in [-0.1, 1.1])
      dout <= sum_k |p| (|Wd| dact + (I + 2 K + 8) 2^-24 |Wd| |act|)
    """
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    K = ids.shape[1]
    u32 = 2.0 ** -24
    out = np.zeros((T, H)) if shared is None else np.asarray(shared, dtype=np.float64).copy()
    bound = np.abs(out) * 2 * u32
    m = np.ones((T, K), bool) if mask is None else np.broadcast_to(
        np.asarray(mask).astype(bool).reshape(T, -1), (T, K))
    for t in range(T):
        seen = set()
        for k in range(K):
            e = int(ids[t, k])
            if e in seen or e < 0 or e >= E or not m[t, k]:
                seen.add(e)
                continue
            seen.add(e)
            wg, wu, wd = (np.asarray(w[e], dtype=np.float64) for w in (Wg, Wu, Wd))
            I = wg.shape[0]
            if gs is not None:
                wg = wg * np.asarray(gs[e], dtype=np.float64)[:, None]
                wu = wu * np.asarray(us[e], dtype=np.float64)[:, None]
                wd = wd * np.asarray(ds[e], dtype=np.float64)[:, None]
            g, u = wg @ x[t], wu @ x[t]
            act = _silu(g) * u
            p = float(probs[t, k])
            out[t] += p * (wd @ act)
            dg = (H + 4) * u32 * (np.abs(wg) @ np.abs(x[t]))
            du = (H + 4) * u32 * (np.abs(wu) @ np.abs(x[t]))
            dact = 1.1 * np.abs(u) * dg + np.abs(_silu(g)) * du + 1.1 * dg * du \
                + (2.0 ** -9 + 2.0 ** -20) * np.abs(act)
            bound[t] += abs(p) * (np.abs(wd) @ (dact * (1 + 2.0 ** -10))
                                  + (I + 2 * K + 8) * u32 * (np.abs(wd) @ np.abs(act)))
    return out, bound
