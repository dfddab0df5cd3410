"""Padding rows, whose logits are all the same, under biases that balancing has moved:
each is a small multiple of one step, so that many experts and groups tie exactly and
the biases alone, then the index, decide."""

import numpy as np
import pytest
import torch

from test_gpu_router_grouped import _check

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _bias(E, steps, seed, rate=1e-3):
    """Biases after some steps of + or - rate, as float32 sums."""
    g = np.random.default_rng(seed)
    b = np.zeros(E, dtype=np.float32)
    for _ in range(steps):
        b += np.float32(rate) * np.sign(g.standard_normal(E)).astype(np.float32)
    return torch.from_numpy(b)


def _rows(E, dtype):
    """One logit each, and rows that differ in one place or by masks."""
    l = torch.zeros(9, E)
    l[1], l[2], l[3], l[4] = 2.5, -30.0, float("inf"), 1e-30
    l[5, E - 1] = 2.0 ** -7
    l[6, 0] = -float("inf")
    l[7] = -float("inf")
    l[8, ::2] = -0.0
    return l.to(dtype).to(DEV)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("steps", [1, 3, 100])
@pytest.mark.parametrize("E,K,G,top,each", [
    (256, 8, 8, 4, 2), (512, 16, 4, 2, 1), (96, 9, 1, 1, 1), (40, 3, 10, 3, 2), (160, 6, 8, 3, 2), (1024, 16, 32, 5, 2),
    (32, 4, 32, 9, 1), (72, 2, 9, 1, 1), (5, 5, 1, 1, 2)])
def test_rows_of_one_logit(lib, E, K, G, top, each, steps, dtype, scoring):
    _check(lib, _rows(E, dtype), _bias(E, steps, E + steps).to(DEV), K, G, top, each, scoring, True, grad=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("each", [1, 2])
def test_with_experts_that_a_bias_takes_out(lib, each, scoring):
    """Groups of 5 with none, one, two or all of their experts left, and a NaN."""
    inf = float("inf")
    rows = _rows(20, torch.float32)
    for out in (range(5), range(6, 10), range(10, 13), [0, 7, 19], range(18), range(20)):
        bias = _bias(20, 2, 3)
        bias[list(out)] = -inf
        for K in (1, 4, 10):
            _check(lib, rows, bias.to(DEV), K, 4, 2, each, scoring, True, grad=False)
    bias[:] = 0.001
    bias[7] = float("nan")
    _check(lib, rows, bias.to(DEV), 4, 4, 2, each, scoring, True, status=lib.MOE_ERR_INVALID_ARG, grad=False)


@pytest.mark.parametrize("size", [1e-30, 2.0 ** -53, 2.0 ** -30, 1e3, 3e38])
def test_biases_of_every_size(lib, size):
    """Sums that 64 bits round to one value tie; sums of two past fp32's range do not."""
    g = np.random.default_rng(4)
    bias = torch.from_numpy((g.integers(-2, 3, 64) * size).clip(-3.4e38, 3.4e38).astype(np.float32))
    for scoring in ("softmax", "sigmoid"):
        for each in (1, 2):
            _check(lib, _rows(64, torch.float32), bias.to(DEV), 6, 8, 3, each, scoring, True, grad=False)


def test_a_batch_that_is_half_padding(lib):
    """Against a 64-bit sort, and the ordinary rows as they are alone."""
    T, E, K, G, top = 4096, 256, 8, 8, 4
    l = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV) * 1.5
    l[T // 2:] = 0
    bias = _bias(E, 100, 5).to(DEV)
    kw = dict(bias=bias, num_groups=G, top_groups=top, group_top=2)
    ids, p = lib.moe_router_topk_grouped(l, K, **kw)
    alone = lib.moe_router_topk_grouped(l[:T // 2].contiguous(), K, **kw)
    assert torch.equal(ids[:T // 2], alone[0]) and torch.equal(p[:T // 2], alone[1])
    c = 0.5 + bias.double()
    v = c.view(G, -1).topk(2, dim=1).values.sum(1)
    keep = v.sort(descending=True, stable=True).indices[:top]
    out = torch.ones(G, dtype=torch.bool, device=DEV).index_fill_(0, keep, False).repeat_interleave(E // G)
    want = c.masked_fill(out, -9.0).sort(descending=True, stable=True).indices[:K]
    assert (ids[T // 2:].long() == want).all() and (p[T // 2:] == 0.125).all()
