"""The grouped router without a GPU: its oracle, and calls that are refused on the host."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from test_abi_exports import built_lib  # noqa: F401  (fixture)
from test_oracle_serving_pins import MODES

P, U = 0x10000, 0x10008
F32, BF16 = 0, 1
INV, SHAPE = 1, 2


@pytest.mark.parametrize("scoring,renorm", MODES)
@pytest.mark.parametrize("each", [1, 2])
def test_oracle_matches_torch(each, scoring, renorm):
    g = np.random.default_rng(4)
    T, E, K, G, top = 30, 48, 5, 6, 3
    l, b = g.standard_normal((T, E)), g.standard_normal(E) * 0.1
    ids, p = S.router_topk_grouped(l, b, K, G, top, each, scoring, renorm, 1.5)
    s = torch.softmax(torch.from_numpy(l), 1) if scoring == "softmax" else torch.sigmoid(torch.from_numpy(l))
    c = s + torch.from_numpy(b)
    v = c.view(T, G, -1).topk(each, dim=2).values.sum(2)
    out = torch.ones(T, G, dtype=torch.bool).scatter(1, v.topk(top, dim=1).indices, False)
    want = c.masked_fill(out.repeat_interleave(E // G, 1), -9.0).topk(K, dim=1).indices
    assert np.array_equal(ids, want.numpy())
    w = s.gather(1, want)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    assert np.allclose(p, 1.5 * w.numpy(), rtol=1e-13, atol=0)


def test_oracle_masks_and_ties():
    inf = np.inf
    l = np.array([[0.0, 0.0, 0.0, 0.0, 0.0, 0.0], [3.0, -inf, 0.0, 0.0, -inf, -inf], [-inf] * 6])
    ids, p = S.router_topk_grouped(l, np.zeros(6), 2, 3, 1, 2, "sigmoid", True, 1.0)
    # a group with one expert left comes after the one with two
    assert ids.tolist() == [[0, 1], [2, 3], [0, 1]] and p[2].tolist() == [0.0, 0.0]
    ids, _ = S.router_topk_grouped(l, np.array([0, 0, -inf, 0, np.nan, 0]), 2, 3, 1, 2, "sigmoid", True, 1.0)
    assert ids.tolist() == [[0, 1], [0, 1], [0, 1]]


CHECKS = [
    # logits, dtype, bias, T, E, K, groups, top, each, scoring, renorm, scale, ids, probs, status, stream
    ((P, F32, P, -1, 64, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),     # T < 0
    ((P, F32, P, 4, 64, 0, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),      # K = 0
    ((P, F32, P, 4, 64, 4, 0, 2, 2, 0, 1, 1.0, P, P, None, None), INV),      # no groups
    ((P, F32, P, 4, 64, 4, 4, 0, 2, 0, 1, 1.0, P, P, None, None), INV),      # none kept
    ((P, 2, P, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),        # dtype
    ((P, F32, P, 4, 64, 4, 4, 2, 3, 0, 1, 1.0, P, P, None, None), INV),      # a sum of three
    ((P, F32, P, 4, 64, 4, 4, 2, 2, 2, 1, 1.0, P, P, None, None), INV),      # scoring
    ((P, F32, P, 4, 64, 17, 4, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),   # K > 16
    ((P, F32, P, 4, 1088, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),  # E > 1024
    ((P, F32, P, 4, 66, 4, 33, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),   # more than 32 groups
    ((P, F32, P, 4, 64, 4, 4, 5, 2, 0, 1, 1.0, P, P, None, None), SHAPE),    # more kept than there are
    ((P, F32, P, 4, 65, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),    # E is no multiple
    ((P, F32, P, 4, 4, 2, 4, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),     # groups of one, two asked
    ((P, F32, P, 4, 64, 9, 8, 1, 2, 0, 1, 1.0, P, P, None, None), SHAPE),    # K of eight experts
    ((P, F32, P, 4, 960, 4, 3, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),   # 320 experts in 8 lanes
    ((P, F32, P, 1 << 28, 64, 8, 4, 2, 2, 0, 1, 1.0, P, P, None, None), SHAPE),  # T K past 31 bits
    ((None, F32, P, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),
    ((U, F32, P, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),
    ((P, F32, U, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, P, P, None, None), INV),
    ((P, BF16, None, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, None, P, None, None), INV),
    ((P, BF16, None, 4, 64, 4, 4, 2, 2, 0, 1, 1.0, P, U, None, None), INV),
]


@pytest.mark.parametrize("args,status", CHECKS)
def test_refused_on_the_host(built_lib, args, status):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    assert binding.load_library(built_lib).moe_router_topk_grouped(*args) == status


def test_nothing_to_do_is_ok(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    lib = binding.load_library(built_lib)
    assert lib.moe_router_topk_grouped(None, F32, None, 0, 64, 4, 4, 2, 2, 0, 1, 1.0, None, None, None, None) == 0


def test_binding_refuses_wrong_tensors(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding as b
    l = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="bias must be"):
        b.moe_router_topk_grouped(l, 4, bias=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="bias must have shape"):
        b.moe_router_topk_grouped(l, 4, bias=torch.zeros(63))
    with pytest.raises(ValueError, match="expert_ids must be"):
        b.moe_router_topk_grouped(l, 4, expert_ids=torch.zeros(4, 4))
    with pytest.raises(ValueError, match="probs must have shape"):
        b.moe_router_topk_grouped(l, 4, probs=torch.zeros(4, 5))
