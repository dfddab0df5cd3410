"""GPU parity of the router with a bias and groups against the float64 oracle.

The ids have to be the oracle's.  Weights and gradients are bounded as the
plain router's are: (R + E / 32 + 24) 2^-23 of themselves, R the spread of the
logits that matter, and an absolute 1e-37 for subnormal results.
"""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import np64, ulp
from test_gpu_router import MODES, _rel

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _check(lib, logits, bias, K, G, top, each, scoring, renorm, scale=1.0, status=None, grad=True):
    l = np64(logits)
    st = lib.new_status()
    kw = dict(scoring=scoring, renormalize=renorm, scale=scale)
    ids, p = lib.moe_router_topk_grouped(logits, K, bias=bias, num_groups=G, top_groups=top, group_top=each,
                                         dev_status=st, **kw)
    assert ids.dtype == torch.int32 and p.dtype == torch.float32
    b = None if bias is None else np64(bias)
    w_ids, w_p = S.router_topk_grouped(l, b, K, G, top, each, scoring, renorm, scale)
    assert np.array_equal(np64(ids), w_ids)
    rel = _rel(l, l.shape[1])
    assert np.all(np.abs(np64(p) - w_p) <= rel * np.abs(w_p) + 1e-37)
    if grad:
        g = np.random.default_rng(K).standard_normal(w_p.shape).astype(np.float32)
        d = lib.moe_router_topk_grad(torch.from_numpy(g).to(DEV), logits, ids, dev_status=st, **kw)
        want = S.router_topk_grad(g, l, w_ids, scoring, renorm, scale)
        gk, q = np.abs(scale * g.astype(np.float64)), np.abs(w_p / scale)
        D = (gk * q).sum(1, keepdims=True)
        mag = np.zeros_like(l)
        if scoring == "softmax" and not renorm:
            mag += np.stack([S._scores(r, scoring) for r in S._clean(l)]) * D
        np.add.at(mag, (np.arange(len(l))[:, None], w_ids), q * (gk + (D if scoring == "softmax" or renorm else 0)))
        bound = rel * mag + 1e-37
        if logits.dtype == torch.bfloat16:
            bound = bound + ulp(np.maximum(np.abs(np64(d)), np.abs(want)), "bf16")
        assert np.all(np.abs(np64(d) - want) <= bound)
    assert lib.moe_check_status(st) == (lib.MOE_OK if status is None else status)


@pytest.mark.parametrize("scoring,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,K,G,top,each", [
    (1, 256, 8, 8, 4, 2), (37, 160, 6, 8, 3, 1), (9, 64, 8, 1, 1, 1), (5, 32, 4, 32, 9, 1), (3, 1024, 16, 16, 5, 2),
    (64, 96, 5, 3, 2, 2), (6, 40, 16, 4, 2, 2), (130, 200, 8, 5, 5, 2), (11, 72, 2, 9, 1, 1), (2, 2, 1, 2, 1, 1),
    (3, 1, 1, 1, 1, 1), (4, 768, 7, 3, 1, 2), (50, 512, 8, 4, 2, 1)])
def test_selection_and_weights(lib, T, E, K, G, top, each, biased, dtype, scoring, renorm):
    g = np.random.default_rng(T * E + K)
    logits = torch.from_numpy(g.standard_normal((T, E)) * 1.5).to(dtype).to(DEV)
    bias = torch.from_numpy(g.standard_normal(E) * 0.1).float().to(DEV) if biased else None
    _check(lib, logits, bias, K, G, top, each, scoring, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("scoring,renorm", MODES)
@pytest.mark.parametrize("each", [1, 2])
def test_masked_groups_ties_and_extremes(lib, each, scoring, renorm):
    """Groups of 5 with none, one or two experts left; every score equal; the two
    ends of the range; a bias that takes experts out."""
    inf, big = float("inf"), float(np.finfo(np.float32).max)
    rows = [[0.0] * 20, [-inf] * 20, [-inf] * 18 + [1.0, -2.0], [-big] * 20, [big] * 20,
            [inf] + [0.0] * 18 + [inf], [-0.0, 0.0] * 10, [100.0] + [-100.0] * 19, [-inf] * 10 + [-big] * 10,
            [0.5] + [-inf] * 4 + [2.0] + [-inf] * 4 + [-1.0, -1.0] + [-inf] * 8, [1e-40, 2e-40] * 10,
            [-720.0] * 10 + [-719.0] * 10, [3.0, -inf, -inf, -inf, -inf] * 4]
    logits = torch.tensor(rows, dtype=torch.float32, device=DEV)
    biases = [None, [0.0] * 20, [0.25] * 20, [0.0] * 5 + [-inf] * 5 + [0.0] * 9 + [-inf], [-inf] * 20, [1e30] * 20]
    for b in biases:
        bias = None if b is None else torch.tensor(b, dtype=torch.float32, device=DEV)
        _check(lib, logits, bias, 4, 4, 2, each, scoring, renorm, grad=False)
        _check(lib, logits, bias, 10, 4, 2, each, scoring, renorm, grad=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_scores_that_32_bits_cannot_tell_apart(lib, scoring):
    """Logits and biases a few steps of fp32 apart: the fp32 pass must leave such
    rows to the 64-bit one.  Two sums of scores are equal only where they sum the
    same levels and biases (no two pairs of the levels have one sum), and then to
    the bit (a score plus a bias is exact here: multiples of 2^-24 below 2^-18,
    far from a power of two), so the oracle and the kernel see the same ties."""
    g = np.random.default_rng(5)
    T, E = 40, 48
    levels = np.array([0, 1, 3, 9, 27, 81], dtype=np.float32) * np.float32(2.0 ** -24)
    l = np.float32(0.7) + levels[g.integers(0, 6, (T, E))] * (1 + np.arange(T, dtype=np.float32) % 3)[:, None]
    for step in (0.0, 2.0 ** -24, 2.0 ** -20):
        bias = (g.integers(0, 3, E) * step).astype(np.float32)
        for G, top, each in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
            _check(lib, torch.from_numpy(l).to(DEV), torch.from_numpy(bias).to(DEV), 8, G, top, each, scoring, True,
                   grad=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [64.0, 1e3, 3e4])
def test_biases_that_cancel_in_a_group(lib, scoring, size):
    """A group's two largest are s + size and s' - size: their sum is of the size
    of a score, its error in fp32 of the biases'."""
    g = np.random.default_rng(int(size))
    T, E, G = 400, 64, 8
    logits = torch.from_numpy(g.standard_normal((T, E))).float().to(DEV)
    bias = torch.full((E,), -size)
    bias[::E // G] = size
    _check(lib, logits, bias.to(DEV), 4, G, 3, 2, scoring, True, grad=False)


def test_biases_whose_sums_pass_the_range(lib):
    """Sums of two beyond fp32's largest, of either sign, beside a group without experts."""
    of = [2e38, 3e38, 2.5e38, 0.0, -2e38, -3e38, -2.5e38, -float("inf")]
    bias = torch.tensor(of, dtype=torch.float32, device=DEV).repeat_interleave(4)
    logits = torch.from_numpy(np.random.default_rng(8).standard_normal((5, 32))).float().to(DEV)
    for top in range(1, 8):
        for order in (list(range(32)), list(range(31, -1, -1))):
            _check(lib, logits, bias[order], 4, 8, top, 2, "sigmoid", True, grad=False)
            _check(lib, logits, bias[order], min(16, 4 * top), 8, top, 2, "softmax", True, grad=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K,G,top,each", [(256, 8, 8, 4, 2), (512, 16, 4, 2, 1), (96, 9, 1, 1, 1), (40, 3, 10, 3, 2)])
def test_rows_of_one_logit(lib, E, K, G, top, each, dtype, scoring):
    """Padding rows: every logit and every bias the same, all but one of them, all but
    the first, and all masked."""
    l = torch.zeros(7, E)
    l[1] = 2.5
    l[2, E - 1] = 2.0 ** -7
    l[3, 0] = -1.0
    l[4] = -float("inf")
    l[5] = float("inf")
    l[6, E // 2] = -float("inf")
    flat, last = torch.full((E,), 0.125), torch.full((E,), 0.125)
    last[E - 1] = 0.25
    for b in (None, torch.zeros(E), flat, last, torch.full((E,), -float("inf"))):
        _check(lib, l.to(dtype).to(DEV), None if b is None else b.to(DEV), K, G, top, each, scoring, True, grad=False)


def test_many_rows_in_order(lib):
    """A training step's rows: each row's selection against a 64-bit sort."""
    T, E, K, G, top = 16384, 256, 8, 8, 4
    g = torch.Generator(device=DEV).manual_seed(3)
    l = torch.randn(T, E, generator=g, device=DEV) * 1.5
    bias = torch.randn(E, generator=g, device=DEV) * 0.1
    ids, p = lib.moe_router_topk_grouped(l, K, bias=bias, num_groups=G, top_groups=top, group_top=2)
    s = torch.sigmoid(l.double())
    c = s + bias.double()
    v = c.view(T, G, -1).topk(2, dim=2).values.sum(2)
    keep = v.topk(top, dim=1).indices
    out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter(1, keep, False).repeat_interleave(E // G, dim=1)
    want = c.masked_fill(out, -1.0).topk(K, dim=1).indices
    assert torch.equal(ids.long(), want)
    w = s.gather(1, want)
    w = w / w.sum(1, keepdim=True)
    assert float(((p.double() - w) / w).abs().max()) <= _rel(np.array([-8.0, 8.0]), E)
    # the same from another stream, twice at once
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        again = lib.moe_router_topk_grouped(l, K, bias=bias, num_groups=G, top_groups=top, group_top=2)
    here = lib.moe_router_topk_grouped(l, K, bias=bias, num_groups=G, top_groups=top, group_top=2)
    torch.cuda.current_stream().wait_stream(other)
    for a, b in zip(again, here):
        assert torch.equal(a, b)
    assert torch.equal(again[0], ids) and torch.equal(again[1], p)


def test_one_group_without_bias_is_the_plain_router(lib):
    g = torch.Generator(device=DEV).manual_seed(9)
    for dtype in (torch.float32, torch.bfloat16):
        l = torch.randn(300, 128, generator=g, device=DEV).to(dtype)
        for scoring, renorm in MODES:
            kw = dict(scoring=scoring, renormalize=renorm, scale=1.5)
            a, b = lib.moe_router_topk(l, 8, **kw), lib.moe_router_topk_grouped(l, 8, **kw)
            assert torch.equal(a[0], b[0])
            assert torch.allclose(a[1], b[1], rtol=2.0 ** -20, atol=0)


def test_flags_nan_and_bad_bias(lib):
    l = torch.randn(3, 24, device=DEV)
    l[1, 4] = float("nan")
    bias = torch.zeros(24, device=DEV)
    _check(lib, l, bias, 5, 4, 2, 2, "sigmoid", True, status=lib.MOE_ERR_INVALID_ARG)
    l = torch.randn(3, 24, device=DEV)
    for bad in (float("nan"), float("inf")):
        bias = torch.zeros(24, device=DEV)
        bias[7] = bad
        _check(lib, l, bias, 5, 4, 2, 2, "softmax", True, status=lib.MOE_ERR_INVALID_ARG)


def test_no_rows(lib):
    ids, p = lib.moe_router_topk_grouped(torch.empty(0, 64, device=DEV), 4, num_groups=4, top_groups=2)
    assert ids.shape == p.shape == (0, 4)


def test_in_a_graph(lib):
    l, bias = torch.zeros(70, 96, device=DEV), torch.zeros(96, device=DEV)
    kw = dict(bias=bias, num_groups=6, top_groups=2, group_top=2)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lib.moe_router_topk_grouped(l, 4, **kw)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    st = lib.new_status()
    with torch.cuda.graph(graph, stream=s):
        got = lib.moe_router_topk_grouped(l, 4, dev_status=st, **kw)
    for seed in range(3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        l.copy_(torch.randn(70, 96, generator=g, device=DEV))
        bias.copy_(torch.randn(96, generator=g, device=DEV) * 0.1)
        graph.replay()
        torch.cuda.synchronize()
        want = lib.moe_router_topk_grouped(l, 4, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lib.moe_check_status(st) == lib.MOE_OK
