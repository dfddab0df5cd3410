"""Plain CPU oracle of the router, the 8-bit products and the layer for a few
tokens.

TEST INFRASTRUCTURE ONLY, like ``moe_oracle``: the definitions in float64
numpy, one expert or one token at a time, sharing nothing with the CUDA
library.  Results are not rounded to the storage dtype; the tests add the
rounding to their bounds.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import round_to_bf16

__all__ = ["router_topk", "router_topk_grouped", "router_topk_grad", "quantize_rows", "linear_int8",
           "gate_up_swiglu_int8", "quantize_weights_int4", "pack_int4", "unpack_int4", "weights_int4",
           "linear_float", "layer_few_tokens"]

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


def router_topk_grouped(logits, bias, K: int, groups: int, top_groups: int, group_top: int,
                        scoring: str, renormalize: bool, scale: float):
    """(expert_ids, probs): the K largest scores plus bias of the top_groups best
    groups, weights from the scores alone.  With no bias, and no sums of two that
    matter, the logits are compared."""
    l = _clean(logits)
    T, E = l.shape
    size = E // groups
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    b = np.where(b < np.inf, b, -np.inf)  # +inf, NaN: out
    plain = bias is None and (group_top == 1 or top_groups == groups)
    ids = np.zeros((T, K), dtype=np.int64)
    probs = np.zeros((T, K))
    for t in range(T):
        c = l[t] if plain else np.where(np.isneginf(l[t]), -np.inf, _scores(l[t], scoring) + b)
        value = []
        for g in range(groups):
            best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_top]
            left = best[~np.isneginf(best)]
            value.append((-len(left), -left.sum() if len(left) else 0.0, g))
        kept = [g for _, _, g in sorted(value)[:top_groups]]
        among = sorted((-c[j], j) for g in kept for j in range(g * size, (g + 1) * size))
        ids[t] = [j for _, j in among[:K]]
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


# The inputs of eight whose values a byte holds: (lower, upper four bits).
_BYTES = ((0, 2), (4, 6), (1, 3), (5, 7))


def pack_int4(q):
    """Whole numbers [..., k] in [-8, 7] as bytes [..., k / 2]."""
    q = np.asarray(q) & 15
    p = np.zeros(q.shape[:-1] + (q.shape[-1] // 2,), dtype=np.uint8)
    for i, (a, b) in enumerate(_BYTES):
        p[..., i::4] = q[..., a::8] | q[..., b::8] << 4
    return p


def unpack_int4(p):
    """The whole numbers of pack_int4's bytes."""
    p = np.asarray(p).astype(np.int64)
    q = np.zeros(p.shape[:-1] + (p.shape[-1] * 2,), dtype=np.int64)
    for i, (a, b) in enumerate(_BYTES):
        q[..., a::8], q[..., b::8] = p[..., i::4] & 15, p[..., i::4] >> 4
    return np.where(q > 7, q - 16, q)


def quantize_weights_int4(W, group: int):
    """(q [E, n, k] whole numbers, scale [E, k / group, n] float32) of weights
    [E, n, k] in float32 arithmetic, as the format defines it."""
    W = np.asarray(W, dtype=np.float32)
    w = W.reshape(W.shape[:2] + (-1, group))
    top = np.max(np.abs(w), axis=-1)
    bad = ~np.all(np.isfinite(w), axis=-1)
    top = np.where(bad, np.float32(0), top)
    t = top * np.float32(1.0 / 7.0)
    # five significant bits, ties to even, and at least 2^-130
    step = np.ldexp(1.0, np.maximum(np.frexp(t.astype(np.float64))[1] - 5, -130))
    scale = (np.rint(t.astype(np.float64) / step) * step).astype(np.float32)
    s = np.where(scale > 0, scale, np.float32(1))[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.clip(np.rint((w / s).astype(np.float32)), -8, 7)
    q = np.where((scale > 0)[..., None], q, 0).astype(np.int64)
    scale = np.where(bad, np.float32(np.nan), scale)
    return q.reshape(W.shape), np.swapaxes(scale, 1, 2)


def weights_int4(W_q, scale):
    """The weights [E, n, k] that bytes and scales [E, k / group, n] stand for:
    q * scale rounded to bf16."""
    q = unpack_int4(W_q)
    s = np.swapaxes(np.asarray(scale, dtype=np.float64), 1, 2)
    return round_to_bf16(q * np.repeat(s, q.shape[2] // s.shape[2], axis=2))


def linear_float(x, offsets, W):
    """y[i] = W[e] x[i] for the rows i of expert e."""
    x = np.asarray(x, dtype=np.float64)
    y = np.zeros((x.shape[0], W.shape[1]))
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y[lo:hi] = x[lo:hi] @ np.asarray(W[e], dtype=np.float64).T
    return y


def layer_few_tokens(x, ids, probs, Wg, Wu, Wd, E: int, num_special: int = 0, mask=None,
                     shared=None, gs=None, us=None, ds=None, act_rounding=2.0 ** -9, exact_sums=False):
    """(out [T, H], bound [T, H]).  bound: what fp32 sums in any order and act's
    rounding add up to, without the rounding of out:
      dg  = (H + 4) 2^-24 sum |w x|,  du alike  (the scale's product included);
            0 with exact_sums, for data whose sums are exact in fp32
      dact <= |silu'(g) u| dg + |silu(g)| du + dg du + (act_rounding + 2^-20) |act|
              (silu' is in [-0.1, 1.1])
      dout <= sum_k |p| (|Wd| dact + (I + 2 K + 8) 2^-24 |Wd| |act|)
    act_rounding: 2^-9 for act in one bfloat16, half of what a single rounding can
    reach and more than a sum of I of them does; 2^-16 for act as a bfloat16 and
    the bfloat16 of what that leaves, each off by 2^-8 of its value at most.
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
            dg = (0 if exact_sums else H + 4) * u32 * (np.abs(wg) @ np.abs(x[t]))
            du = (0 if exact_sums else H + 4) * u32 * (np.abs(wu) @ np.abs(x[t]))
            dact = 1.1 * np.abs(u) * dg + np.abs(_silu(g)) * du + 1.1 * dg * du \
                + (act_rounding + 2.0 ** -20) * np.abs(act)
            bound[t] += abs(p) * (np.abs(wd) @ (dact * (1 + 2.0 ** -10))
                                  + (I + 2 * K + 8) * u32 * (np.abs(wd) @ np.abs(act)))
    return out, bound
