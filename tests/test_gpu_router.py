"""GPU parity of the router and its gradient against the float64 oracle.

Bounds.  e^(l - m) in fp32: the difference rounds once (|l - m| 2^-24 in the
exponent) and expf is within 2 ulp; the sum over E / 32 + 5 additions; a few
products and divisions.  So a weight is within
(R + E / 32 + 24) 2^-23 of itself, R the spread of the logits that matter
(at most 104: e^-104 underflows), and a gradient within the same share of
q (|g| + sum |g q|).  Results under 1e-37 are subnormal: an absolute 1e-37.
"""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import np64, ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"
MODES = [(s, r) for s in ("softmax", "sigmoid") for r in (False, True)]


def _rel(l, E):
    fin = l[np.isfinite(l)]
    spread = min(104.0, float(fin.max() - fin.min())) if fin.size else 0.0
    return (spread + E / 32 + 24) * 2.0 ** -23


def _check(lib, logits, K, scoring, renorm, scale, grad_seed=0, status=None):
    E = logits.shape[1]
    l = np64(logits)
    kw = dict(scoring=scoring, renormalize=renorm, scale=scale)
    st = lib.new_status()
    ids, probs = lib.moe_router_topk(logits, K, dev_status=st, **kw)
    w_ids, w_p = S.router_topk(l, K, scoring, renorm, scale)
    assert np.array_equal(np64(ids), w_ids)
    rel = _rel(l, E)
    assert np.all(np.abs(np64(probs) - w_p) <= rel * np.abs(w_p) + 1e-37)
    gp = torch.from_numpy(np.random.default_rng(grad_seed).standard_normal(w_p.shape)).float().to(DEV)
    d = lib.moe_router_topk_grad(gp, logits, ids, dev_status=st, **kw)
    assert d.dtype == logits.dtype
    w_d = S.router_topk_grad(np64(gp), l, w_ids, scoring, renorm, scale)
    g = np.abs(scale * np64(gp))
    q = np.abs(w_p / scale)
    mag = np.zeros_like(l)
    D = (g * q).sum(1, keepdims=True)
    if scoring == "softmax" and not renorm:
        mag += np.stack([S._scores(r, scoring) for r in S._clean(l)]) * D
    np.add.at(mag, (np.arange(len(l))[:, None], w_ids), q * (g + (D if scoring == "softmax" or renorm else 0)))
    bound = rel * mag + 1e-37
    if logits.dtype == torch.bfloat16:
        bound = bound + ulp(np.maximum(np.abs(np64(d)), np.abs(w_d)), "bf16")
    assert np.all(np.abs(np64(d) - w_d) <= bound)
    assert lib.moe_check_status(st) == (lib.MOE_OK if status is None else status)


@pytest.mark.parametrize("scoring,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 128, 8), (5, 1, 1), (37, 33, 6), (130, 200, 16), (9, 64, 1),
                                   (3, 1024, 8), (65, 257, 7), (4, 16, 16), (2, 1000, 3)])
def test_router(lib, T, E, K, dtype, scoring, renorm):
    g = np.random.default_rng(T * E + K)
    logits = torch.from_numpy(g.standard_normal((T, E)) * 2).to(dtype).to(DEV)
    _check(lib, logits, K, scoring, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("scoring,renorm", MODES)
def test_router_masked_rows_ties_and_extremes(lib, scoring, renorm):
    inf, big = float("inf"), float(np.finfo(np.float32).max)
    rows = [[0.0] * 40, [-inf] * 40, [-inf] * 38 + [1.0, -2.0], [-big] * 40, [big] * 40,
            [inf] + [0.0] * 38 + [inf], [-0.0, 0.0] * 20, [100.0] + [-100.0] * 39,
            [-inf] * 20 + [-big] * 20, [-90.0] * 40, [1e-40, 2e-40] * 20]
    logits = torch.tensor(rows, dtype=torch.float32, device=DEV)
    _check(lib, logits, 4, scoring, renorm, 1.0)


def test_router_flags_nan_and_bad_ids(lib):
    l = torch.randn(3, 20, device=DEV)
    l[1, 4] = float("nan")
    _check(lib, l, 5, "softmax", True, 1.0, status=lib.MOE_ERR_INVALID_ARG)
    l = torch.randn(2, 20, device=DEV)
    ids = torch.tensor([[3, 25], [-1, 2]], dtype=torch.int32, device=DEV)
    st = lib.new_status()
    d = lib.moe_router_topk_grad(torch.ones(2, 2, device=DEV), l, ids, renormalize=False, dev_status=st)
    assert lib.moe_check_status(st) == lib.MOE_ERR_BAD_ID
    p = torch.softmax(l.double(), 1)
    for t, e in ((0, 3), (1, 2)):
        want = -p[t] * p[t, e]
        want[e] += p[t, e]
        assert torch.allclose(d[t].double(), want, rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("scoring,renorm", MODES)
def test_router_grad_against_differences(lib, scoring, renorm):
    """Central differences of the kernel's own forward.  h = 2^-6: the
    difference quotient is off by h^2 / 6 times a third derivative (below 1
    for these scores) and by the forward's rounding, 2 * 24 * 2^-23 / 2h."""
    g = np.random.default_rng(7)
    l = torch.from_numpy(g.permutation(24).reshape(1, 24) * 0.125 - 1).float().to(DEV)  # no swaps under h
    gp = torch.from_numpy(g.standard_normal((1, 4))).float().to(DEV)
    kw = dict(scoring=scoring, renormalize=renorm)
    ids, _ = lib.moe_router_topk(l, 4, **kw)
    d = lib.moe_router_topk_grad(gp, l, ids, **kw)[0]
    h = 2.0 ** -6
    many = l.repeat(48, 1)
    for j in range(24):
        many[2 * j, j] += h
        many[2 * j + 1, j] -= h
    i2, p2 = lib.moe_router_topk(many, 4, **kw)
    assert torch.equal(i2, ids.expand(48, -1))
    v = (p2.double() * gp.double()).sum(1)
    fd = (v[0::2] - v[1::2]) / (2 * h)
    lim = float(gp.abs().sum()) * (h * h / 6 + 48 * 2.0 ** -23 / (2 * h))
    assert float((fd - d.double()).abs().max()) <= lim


def test_router_large_batch_and_second_stream(lib):
    g = torch.Generator(device=DEV).manual_seed(3)
    l = torch.randn(20000, 256, generator=g, device=DEV)
    ids, p = lib.moe_router_topk(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids2, p2 = lib.moe_router_topk(l, 8)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ids, ids2) and torch.equal(p, p2)
    want = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :8]
    assert torch.equal(ids.long(), want)


# ids of a row whose K slots name an expert more than once: neighbours, the first
# and the last, half of the slots apart, three times, all the same
REPEATED = [
    [3, 3], [5, 5, 5], [7, 1, 7], [2, 9, 9, 4], [8, 1, 2, 8], [6, 0, 6, 0], [4, 11, 13, 4, 11, 13],
    [1, 2, 3, 4, 1, 6, 7, 8], [10, 0, 10, 3, 10, 5, 6, 7], [12] * 8, [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 0],
    [0, 1, 2, 3, 4, 5, 6, 7, 0, 1, 2, 3, 4, 5, 6, 7],
]


@pytest.mark.parametrize("scoring,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [16, 40, 257])
def test_router_grad_of_repeated_ids(lib, E, dtype, scoring, renorm):
    """An expert that several slots name collects their gradients, whatever their
    places and whatever order the slots are in: the Jacobian of each slot's
    weight, in 64 bits.  The bound is the one above, for K slots."""
    g = np.random.default_rng(E)
    for row in REPEATED:
        K = len(row)
        ids = np.array([row, row[::-1], np.roll(row, 1), g.permutation(row)], dtype=np.int32)
        logits = torch.from_numpy(g.standard_normal((4, E)) * 2).to(dtype)
        logits[3, row[0]] = -np.inf                                     # a masked one among them
        l, gp = np64(logits), g.standard_normal((4, K)).astype(np.float32)
        d = lib.moe_router_topk_grad(torch.from_numpy(gp).to(DEV), logits.to(DEV), torch.from_numpy(ids).to(DEV),
                                     scoring=scoring, renormalize=renorm, scale=2.0)
        want = S.router_topk_grad(gp, l, ids, scoring, renorm, 2.0)
        mag = np.zeros_like(l)
        for t in range(4):
            q = np.abs(S._selected(S._clean(l)[t], ids[t], scoring, renorm))
            gk = np.abs(2.0 * gp[t].astype(np.float64))
            D = (gk * q).sum()
            if scoring == "softmax" and not renorm:
                mag[t] += S._scores(S._clean(l)[t], scoring) * D
            np.add.at(mag[t], ids[t], q * (gk + (D if scoring == "softmax" or renorm else 0)))
        bound = (_rel(l, E) + K * 2.0 ** -23) * mag + 1e-37
        if dtype == torch.bfloat16:
            bound = bound + ulp(np.maximum(np.abs(np64(d)), np.abs(want)), "bf16")
        assert np.all(np.abs(np64(d) - want) <= bound)
