"""Pins of the router / 8-bit / few-token oracle (no GPU), and the refusals
of the entry points that are decided on the host."""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import serving_oracle as S
from test_abi_exports import built_lib  # noqa: F401  (fixture)

MODES = [(s, r) for s in ("softmax", "sigmoid") for r in (False, True)]


@pytest.mark.parametrize("scoring,renorm", MODES)
def test_router_matches_torch(scoring, renorm):
    g = np.random.default_rng(1)
    l = g.standard_normal((40, 24))
    ids, p = S.router_topk(l, 5, scoring, renorm, 1.5)
    tl = torch.from_numpy(l)
    s = torch.softmax(tl, 1) if scoring == "softmax" else torch.sigmoid(tl)
    w, i = torch.topk(s, 5, dim=1)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    assert np.array_equal(ids, i.numpy())
    assert np.allclose(p, 1.5 * w.numpy(), rtol=1e-13, atol=0)


@pytest.mark.parametrize("scoring,renorm", MODES)
def test_router_grad_matches_finite_differences_and_autograd(scoring, renorm):
    g = np.random.default_rng(2)
    l, gp = g.standard_normal((6, 12)) * 2, g.standard_normal((6, 4))
    ids, _ = S.router_topk(l, 4, scoring, renorm, 0.7)
    d = S.router_topk_grad(gp, l, ids, scoring, renorm, 0.7)
    h = 1e-6
    for t in range(6):
        for j in range(12):
            v = []
            for sgn in (1, -1):
                m = l.copy()
                m[t, j] += sgn * h
                v.append((gp[t] * 0.7 * S._selected(m[t], ids[t], scoring, renorm)).sum())
            assert abs((v[0] - v[1]) / (2 * h) - d[t, j]) < 1e-7
    tl = torch.from_numpy(l).requires_grad_()
    s = torch.softmax(tl, 1) if scoring == "softmax" else torch.sigmoid(tl)
    w = s.gather(1, torch.from_numpy(ids))
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (w * 0.7 * torch.from_numpy(gp)).sum().backward()
    assert np.allclose(d, tl.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_router_masks_ties_and_extremes():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 1.0, 1.0, 0.0], [-inf, -inf, -inf, -inf], [-inf, 2.0, -inf, -inf],
                  [nan, 1.0, 0.0, nan], [inf, 0.0, inf, 1.0], [-0.0, 0.0, -1.0, -1.0]])
    ids, p = S.router_topk(l, 2, "softmax", True, 1.0)
    assert ids.tolist() == [[0, 1], [0, 1], [1, 0], [1, 2], [0, 2], [0, 1]]
    assert p[1].tolist() == [0.0, 0.0] and p[2].tolist() == [1.0, 0.0] and p[4].tolist() == [0.5, 0.5]


def test_quantize_rows_closed_forms():
    x = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [np.inf, 1, 0, 0], [np.nan, 1, 0, 0]])
    q, s = S.quantize_rows(x)
    assert q[0].tolist() == [127, -64, 0, 2] and s[0] == 1.0
    assert q[1].tolist() == [0] * 4 and s[1] == 0.0
    assert np.isnan(s[2]) and np.isnan(s[3])


def test_quantize_rows_decides_bf16_ties_like_exact_arithmetic():
    from fractions import Fraction
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.standard_normal((40, 64)).astype(np.float32)).bfloat16().float().numpy()
    x[:20] = np.round(x[:20] * 8) / 8            # many exact ties
    q, _ = S.quantize_rows(x)
    for row, qr in zip(x, q):
        top = Fraction(float(np.max(np.abs(row))))
        for v, got in zip(row, qr):
            assert round(Fraction(float(v)) * 127 / top) == got     # Fraction rounds half to even


def test_int8_products_match_dequantized_mlp():
    g = np.random.default_rng(4)
    E, I, H, off = 3, 16, 32, np.array([0, 5, 5, 9])
    x = g.standard_normal((9, H))
    q, rs = S.quantize_rows(x)
    Wg, Wu = g.integers(-127, 128, (E, I, H)), g.integers(-127, 128, (E, I, H))
    gs, us = g.random((E, I)), g.random((E, I))
    act, _, _ = S.gate_up_swiglu_int8(q, rs, off, Wg, gs, Wu, us)
    want, _, _, _ = O.expert_mlp(q * rs[:, None].astype(np.float64), off, Wg * gs[..., None],
                                 Wu * us[..., None], g.standard_normal((E, H, I)), "f64")
    assert np.allclose(act, want, rtol=1e-10, atol=1e-12 * np.abs(want).max())


def test_layer_few_tokens_matches_permute_mlp_unpermute():
    g = np.random.default_rng(5)
    T, H, E, K, I = 7, 32, 5, 3, 16
    x = g.standard_normal((T, H))
    ids = np.argsort(g.random((T, E)), axis=1)[:, :K]
    p = g.random((T, K))
    Wg, Wu = g.standard_normal((E, I, H)), g.standard_normal((E, I, H))
    Wd, sh = g.standard_normal((E, H, I)), g.standard_normal((T, H))
    out, bound = S.layer_few_tokens(x, ids, p, Wg, Wu, Wd, E, shared=sh)
    si, rm, _, off = O.permute_routing(ids, E)
    _, y, _, _ = O.expert_mlp(O.permute_rows(x, si, K), off, Wg, Wu, Wd, "f64")
    want = O.unpermute(y, rm, p, T, K, "f64") + sh
    assert np.allclose(out, want, rtol=1e-11, atol=1e-10)
    assert np.all(bound > 0)
    mask = np.ones((T, K), np.uint8)
    mask[2] = 0
    out2, _ = S.layer_few_tokens(x, ids, p, Wg, Wu, Wd, E, mask=mask, shared=sh)
    assert np.array_equal(out2[2], sh[2]) and np.allclose(out2[3], want[3])


# ---- refusals ------------------------------------------------------------------

P, U = 0x10000, 0x10004          # never dereferenced; U is not 16-byte aligned
F32, BF16, I8 = 0, 1, 2
INV, SHAPE = 1, 2


def few(**kw):
    a = dict(x=P, ids=P, pr=P, T=4, H=128, K=2, I=64, E=8, sp=0, mask=None, md=0, wd=BF16, g=P, u=P,
             d=P, gs=None, us=None, ds=None, sh=None, out=P, ws=P, n=1 << 30, st=None, stream=None)
    a.update(kw)
    return tuple(a.values())


REFUSALS = [
    ("moe_router_topk", (P, F32, 4, 8, 9, 0, 1, 1.0, P, P, None, None), SHAPE),          # K > E
    ("moe_router_topk", (P, F32, 4, 64, 17, 0, 1, 1.0, P, P, None, None), SHAPE),        # K > 16
    ("moe_router_topk", (P, F32, 4, 1025, 8, 0, 1, 1.0, P, P, None, None), SHAPE),       # E > 1024
    ("moe_router_topk", (P, F32, 4, 64, 0, 0, 1, 1.0, P, P, None, None), INV),           # K = 0
    ("moe_router_topk", (P, I8, 4, 64, 8, 0, 1, 1.0, P, P, None, None), INV),            # dtype
    ("moe_router_topk", (P, F32, 4, 64, 8, 2, 1, 1.0, P, P, None, None), INV),           # scoring
    ("moe_router_topk", (None, F32, 4, 64, 8, 0, 1, 1.0, P, P, None, None), INV),        # no logits
    ("moe_router_topk", (P, F32, 4, 64, 8, 0, 1, 1.0, P, None, None, None), INV),        # no probs
    ("moe_router_topk", (P, F32, -1, 64, 8, 0, 1, 1.0, P, P, None, None), INV),          # T < 0
    ("moe_router_topk", (U, F32, 4, 64, 8, 0, 1, 1.0, P, P, None, None), INV),           # unaligned
    ("moe_router_topk_grad", (None, P, F32, P, 4, 64, 8, 0, 1, 1.0, P, None, None), INV),  # no gradient
    ("moe_router_topk_grad", (P, P, F32, P, 4, 64, 8, 0, 1, 1.0, None, None, None), INV),  # no output
    ("moe_quantize_rows", (P, BF16, None, 4, 24, 1, 4, P, P, None), SHAPE),              # H % 16
    ("moe_quantize_rows", (P, BF16, None, 4, 32, 2, 8, P, P, None), SHAPE),              # K without a map
    ("moe_quantize_rows", (P, BF16, None, 4, 32, 1, 3, P, P, None), SHAPE),              # N < T
    ("moe_quantize_rows", (P, I8, None, 4, 32, 1, 4, P, P, None), INV),                  # dtype
    ("moe_quantize_rows", (P, BF16, P, 4, 32, 17, 4, P, P, None), SHAPE),                # K > 16
    ("moe_quantize_rows", (P, BF16, P, 4, 32, 2, 8, U, P, None), INV),                   # q unaligned
    ("moe_gate_up_swiglu_int8", (P, P, P, 4, 24, 16, 2, P, P, P, P, P, None, None), SHAPE),   # H % 16
    ("moe_gate_up_swiglu_int8", (P, P, P, 4, 32, 8, 2, P, P, P, P, P, None, None), SHAPE),    # I % 16
    ("moe_gate_up_swiglu_int8", (P, P, None, 4, 32, 16, 2, P, P, P, P, P, None, None), INV),  # offsets
    ("moe_gate_up_swiglu_int8", (P, P, P, 4, 32, 16, 2, P, None, P, P, P, None, None), INV),  # no scale
    ("moe_gate_up_swiglu_int8", (U, P, P, 4, 32, 16, 2, P, P, P, P, P, None, None), INV),     # unaligned
    ("moe_gate_up_swiglu_int8", (P, P, P, 4, 131088, 16, 2, P, P, P, P, P, None, None), SHAPE),  # H too long
    ("moe_gate_up_swiglu_int8", (P, P, P, 4, 32, 16, 1025, P, P, P, P, P, None, None), SHAPE),   # E > 1024
    ("moe_down_proj_int8", (P, P, P, 4, 32, 16, 2, P, P, P, I8, None, None), INV),       # out dtype
    ("moe_down_proj_int8", (P, None, P, 4, 32, 16, 2, P, P, P, BF16, None, None), INV),  # no row scale
    ("moe_down_proj_int8", (P, P, P, -4, 32, 16, 2, P, P, P, BF16, None, None), INV),    # N < 0
    ("moe_layer_few_tokens", few(T=65), SHAPE),
    ("moe_layer_few_tokens", few(T=-1), INV),
    ("moe_layer_few_tokens", few(K=17, E=64), SHAPE),
    ("moe_layer_few_tokens", few(K=9), SHAPE),
    ("moe_layer_few_tokens", few(H=96), SHAPE),
    ("moe_layer_few_tokens", few(I=32), SHAPE),
    ("moe_layer_few_tokens", few(E=1025), SHAPE),
    ("moe_layer_few_tokens", few(wd=F32), INV),
    ("moe_layer_few_tokens", few(wd=I8), INV),                       # no scales
    ("moe_layer_few_tokens", few(gs=P, us=P, ds=P), INV),            # scales with bf16 weights
    ("moe_layer_few_tokens", few(mask=P, md=3), INV),
    ("moe_layer_few_tokens", few(ws=None), INV),
    ("moe_layer_few_tokens", few(n=64), INV),                        # workspace too small
    ("moe_layer_few_tokens", few(ws=U), INV),
    ("moe_layer_few_tokens", few(x=U), INV),
    ("moe_layer_few_tokens", few(pr=None), INV),
]


@pytest.mark.parametrize("name,args,status", REFUSALS, ids=[f"{c[0]}-{i}" for i, c in enumerate(REFUSALS)])
def test_entry_points_refuse_on_the_host(built_lib, name, args, status):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    assert getattr(binding.load_library(built_lib), name)(*args) == status


def test_nothing_to_do_is_ok(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    lib = binding.load_library(built_lib)
    assert lib.moe_router_topk(None, F32, 0, 64, 8, 0, 1, 1.0, None, None, None, None) == 0
    assert lib.moe_quantize_rows(None, BF16, None, 0, 32, 1, 0, None, None, None) == 0
    assert lib.moe_gate_up_swiglu_int8(None, None, P, 0, 32, 16, 2, None, None, None, None, None, None,
                                       None) == 0
    assert lib.moe_down_proj_int8(None, None, None, 0, 32, 16, 1, None, None, None, BF16, None, None) == 0
    assert lib.moe_layer_few_tokens(*few(T=0, x=None, out=None, ws=None)) == 0


def test_binding_refuses_wrong_tensors(built_lib):  # noqa: F811
    """Shapes and dtypes that would make a kernel read past a tensor."""
    from unpermute_moe_permute_gb300 import binding as b
    x, ids = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    w, wd = torch.zeros(8, 64, 128, dtype=torch.bfloat16), torch.zeros(8, 128, 64, dtype=torch.bfloat16)
    p = torch.zeros(4, 2)
    for bad in (dict(probs=p.double()), dict(probs=p[:, :1]), dict(expert_ids=ids.long()),
                dict(W_down=w), dict(W_up=w[:4]), dict(tokens=x.float()),
                dict(scales=(p, p, p)), dict(active_mask=torch.ones(3, dtype=torch.bool)),
                dict(shared_x=x[:2])):
        a = dict(tokens=x, expert_ids=ids, probs=p, W_gate=w, W_up=w, W_down=wd)
        a.update(bad)
        with pytest.raises(ValueError):
            b.moe_layer_few_tokens(**a)
    with pytest.raises(ValueError):
        b.moe_router_topk(torch.zeros(4, 8), 2, scoring="relu")
    with pytest.raises(ValueError):
        b.moe_router_topk(torch.zeros(4, 8), 2)                       # not on a GPU
    with pytest.raises(ValueError):
        b.moe_quantize_rows(x, row_map=torch.zeros(7, dtype=torch.int32), K=2)
    q, s8 = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(8, 64)
    wq = torch.zeros(8, 64, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        b.moe_gate_up_swiglu_int8(q, torch.zeros(3), torch.zeros(9, dtype=torch.int32), wq, s8, wq, s8)
    with pytest.raises(ValueError):
        b.moe_down_proj_int8(q, torch.zeros(4), None, wq, torch.zeros(8, 63))
