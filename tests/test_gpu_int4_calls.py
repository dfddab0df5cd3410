"""Calls of the grouped router and the 4-bit weights that nothing else makes: outputs
that the caller holds, nothing to do, views, two at once, offsets past 32 bits."""

import pytest
import torch

from gpu_util import assert_elementwise, np64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _weights(lib, E, n, k, group=64, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lib.moe_quantize_weights_int4(torch.randn(E, n, k, generator=g, device=DEV) * k ** -0.5, group)


def test_outputs_of_the_caller(lib):
    g = torch.Generator(device=DEV).manual_seed(1)
    l = torch.randn(50, 64, generator=g, device=DEV)
    ids, p = torch.empty(50, 4, dtype=torch.int32, device=DEV), torch.empty(50, 4, device=DEV)
    a = lib.moe_router_topk_grouped(l, 4, num_groups=8, top_groups=3, expert_ids=ids, probs=p)
    b = lib.moe_router_topk_grouped(l, 4, num_groups=8, top_groups=3)
    assert a[0] is ids and a[1] is p and torch.equal(ids, b[0]) and torch.equal(p, b[1])
    W = torch.randn(3, 40, 128, generator=g, device=DEV)
    q, s = torch.empty(3, 40, 64, dtype=torch.uint8, device=DEV), torch.empty(3, 2, 40, dtype=torch.bfloat16, device=DEV)
    a, b = lib.moe_quantize_weights_int4(W, 64, W_q=q, scale=s), lib.moe_quantize_weights_int4(W, 64)
    assert a[0] is q and torch.equal(q, b[0]) and torch.equal(s, b[1])
    w = torch.empty(3, 40, 128, dtype=torch.bfloat16, device=DEV)
    assert lib.moe_dequantize_weights_int4(q, s, W=w) is w and torch.equal(w, lib.moe_dequantize_weights_int4(q, s))


def test_nothing_to_do(lib):
    q, s = _weights(lib, 2, 128, 128)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    assert lib.moe_gate_up_swiglu_int4(x, off, q, s, q, s).shape == (0, 128)
    assert lib.moe_down_proj_int4(x, off, q, s).shape == (0, 128)
    ids, p = torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    assert lib.moe_layer_few_tokens_int4(x, ids, p, q, s, q, s, q, s).shape == (0, 128)
    # rows, but none of an expert: nothing is written
    out = torch.full((5, 128), 2.0, dtype=torch.bfloat16, device=DEV)
    lib.moe_down_proj_int4(torch.ones(5, 128, dtype=torch.bfloat16, device=DEV), off, q, s, expanded=out)
    assert (out == 2.0).all()


def test_views_are_refused(lib):
    W = torch.randn(2, 65, 128, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        lib.moe_quantize_weights_int4(W[:, :64], 64)
    with pytest.raises(ValueError, match="contiguous"):
        lib.moe_router_topk_grouped(torch.randn(64, 4, device=DEV).t(), 2, num_groups=2, top_groups=1)
    flat = torch.randn(64 * 128 + 1, device=DEV)[1:].view(64, 128)          # 4 bytes past 16
    with pytest.raises(lib.MoeError) as e:
        lib.moe_quantize_weights_int4(flat, 64)
    assert e.value.status == lib.MOE_ERR_INVALID_ARG
    with pytest.raises(lib.MoeError) as e:
        lib.moe_router_topk_grouped(flat, 2, num_groups=2, top_groups=1)
    assert e.value.status == lib.MOE_ERR_INVALID_ARG


def test_more_offsets_than_experts(lib):
    q, s = _weights(lib, 2, 64, 128)
    x = torch.randn(30, 128, device=DEV).bfloat16()
    off = torch.tensor([0, 12, 30], dtype=torch.int32, device=DEV)
    more = torch.tensor([0, 12, 30, 7, -1], dtype=torch.int32, device=DEV)
    assert torch.equal(lib.moe_down_proj_int4(x, off, q, s), lib.moe_down_proj_int4(x, more, q, s))


@pytest.mark.parametrize("rows", [19, 700, 6000])
def test_two_products_at_once(lib, rows):
    """The three forms beside each other and beside the few-token layer, on four
    streams, many times: each gives what it gives alone."""
    E, H, I = 16, 1024, 256
    (wg, gs), (wu, us), (wd, ds) = _weights(lib, E, I, H), _weights(lib, E, I, H, seed=1), _weights(lib, E, H, I, seed=2)
    g = torch.Generator(device=DEV).manual_seed(3)
    cut = torch.randint(0, rows + 1, (E - 1,), generator=g, device=DEV).sort().values
    off = torch.cat([torch.zeros(1, device=DEV), cut, torch.full((1,), rows, device=DEV)]).int()
    x = torch.randn(rows, H, generator=g, device=DEV).bfloat16()
    y = torch.randn(rows, I, generator=g, device=DEV).bfloat16()
    ids = torch.rand(7, E, generator=g, device=DEV).topk(4, dim=1).indices.int()
    p = torch.rand(7, 4, generator=g, device=DEV)
    m = lib._m
    calls = [lambda: m.moe_gate_up_swiglu_int4(x, off, wg, gs, wu, us), lambda: m.moe_down_proj_int4(y, off, wd, ds),
             lambda: m.moe_down_proj_int4(y, off, wd, ds, out_dtype=torch.float32),
             lambda: m.moe_layer_few_tokens_int4(x[:7].contiguous(), ids, p, wg, gs, wu, us, wd, ds)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, o in zip(calls, streams, got):
            with torch.cuda.stream(s):
                o.append(c())
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(v, w) for v in o)


def test_weights_past_32_bits(lib):
    """3 x 32768 x 32768 values, 1.6 GB of bytes: the last matrix is what it is alone."""
    g = torch.Generator(device=DEV).manual_seed(4)
    W = torch.empty(3, 32768, 32768, dtype=torch.bfloat16, device=DEV)
    for e in range(3):
        W[e].normal_(generator=g)
    q, s = lib.moe_quantize_weights_int4(W, 128)
    last = lib.moe_quantize_weights_int4(W[2].clone(), 128)
    assert torch.equal(q[2], last[0]) and torch.equal(s[2], last[1])
    del W
    back = lib.moe_dequantize_weights_int4(q, s)
    assert torch.equal(back[2], lib.moe_dequantize_weights_int4(*last))


def test_products_past_32_bits(lib):
    """An output of more than 2^31 elements, and experts whose bytes begin past 2^32."""
    N, K, H = 2_200_007, 64, 1024
    q, s = _weights(lib, 1, H, K)
    x = torch.randn(N, K, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).bfloat16()
    out = lib.moe_down_proj_int4(x, None, q, s)
    assert out.numel() > 2 ** 31
    assert torch.equal(out[-600:], lib.moe_down_proj_int4(x[-600:].contiguous(), None, q, s))
    del out
    E, n, k = 300, 4096, 8192
    q = torch.zeros(E, n, k // 2, dtype=torch.uint8, device=DEV)
    s = torch.zeros(E, k // 128, n, dtype=torch.bfloat16, device=DEV)
    one = _weights(lib, 1, n, k, 128)
    q[E - 1], s[E - 1] = one[0][0], one[1][0]
    assert (E - 1) * n * k // 2 > 2 ** 32
    x = torch.randn(5, k, device=DEV).bfloat16()
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 5
    # (k + 2 rounded additions of exact terms, whatever their order, and the store's rounding)
    W, xd = lib.moe_dequantize_weights_int4(*one)[0].double(), x.double()
    assert_elementwise(np64(lib.moe_down_proj_int4(x, off, q, s)), np64(xd @ W.t()), np64(xd.abs() @ W.abs().t()), k + 2,
                       "bf16", "the last expert's rows")


def test_logits_past_32_bits(lib):
    T, E = 8_400_003, 256
    l = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
    l.normal_(generator=torch.Generator(device=DEV).manual_seed(6))
    assert l.numel() > 2 ** 31
    bias = torch.randn(E, device=DEV) * 0.1
    kw = dict(bias=bias, num_groups=8, top_groups=4, group_top=2)
    ids, p = lib.moe_router_topk_grouped(l, 8, **kw)
    a, b = lib.moe_router_topk_grouped(l[-1000:].clone(), 8, **kw)
    assert torch.equal(ids[-1000:], a) and torch.equal(p[-1000:], b)


def test_rows_that_32_bits_cannot_decide_among_many(lib):
    """A training step's rows with bf16 logits, one bias for all and a masked group:
    every row in question, against a 64-bit sort."""
    T, E, K, G, top = 4096, 128, 8, 8, 3
    g = torch.Generator(device=DEV).manual_seed(7)
    l = torch.randn(T, E, generator=g, device=DEV).bfloat16()
    l[:, 16:32] = float("-inf")
    bias = torch.full((E,), 0.125, device=DEV)
    for scoring in ("sigmoid", "softmax"):
        ids, _ = lib.moe_router_topk_grouped(l, K, bias=bias, num_groups=G, top_groups=top, group_top=1, scoring=scoring)
        d = l.double()
        c = (torch.sigmoid(d) if scoring == "sigmoid" else torch.softmax(d, 1)) + bias.double()
        c = c.masked_fill(torch.isinf(d), -1.0)
        v = c.view(T, G, -1).amax(2)
        keep = v.sort(dim=1, descending=True, stable=True).indices[:, :top]
        out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter(1, keep, False).repeat_interleave(E // G, 1)
        want = c.masked_fill(out, -2.0).sort(dim=1, descending=True, stable=True).indices[:, :K]
        assert torch.equal(ids.long(), want)
