"""GPU parity of the 4-bit weights and their products against the float64 oracle.

Bytes, scales and the bf16 weights are compared bit for bit.  A product's
factors are bf16, so its terms are exact in fp32 and each of the Kd additions
may round: (Kd + 4) 2^-24 of the sum of magnitudes, and the store's rounding.
"""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import U32, assert_elementwise, np64, ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _same(lib, W, group):
    q, s = lib.moe_quantize_weights_int4(W.to(DEV), group)
    w3 = np64(W) if W.dim() == 3 else np64(W)[None]
    w_q, w_s = S.quantize_weights_int4(w3, group)
    assert q.dtype == torch.uint8 and s.dtype == torch.bfloat16
    assert np.array_equal(q.cpu().numpy().reshape(w_q.shape[0], w_q.shape[1], -1), S.pack_int4(w_q))
    assert np.array_equal(np64(s).reshape(w_s.shape), w_s.astype(np.float64), equal_nan=True)
    back = lib.moe_dequantize_weights_int4(q, s)
    assert back.shape == W.shape and back.dtype == torch.bfloat16
    with np.errstate(invalid="ignore"):
        want = w_q * np.repeat(np.swapaxes(w_s.astype(np.float64), 1, 2), group, axis=2)  # (exact in bf16)
    assert np.array_equal(np64(back).reshape(want.shape), want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("E,rows,cols", [(1, 1, 128), (3, 33, 256), (2, 70, 384), (1, 200, 1152), (5, 64, 640), (2, 8, 4096)])
def test_quantize_and_back_bit_exact(lib, E, rows, cols, group, dtype):
    g = np.random.default_rng(rows + cols)
    w = g.standard_normal((E, rows, cols)) * 0.02
    w[0, 0, :group] = 0
    w[-1, -1, -1] = 3.0                                                  # an outlier in the last group
    _same(lib, torch.from_numpy(w).to(dtype), group)


def test_quantize_one_matrix_and_odd_widths(lib):
    g = np.random.default_rng(1)
    _same(lib, torch.from_numpy(g.standard_normal((48, 192))).float(), 64)
    _same(lib, torch.from_numpy(g.standard_normal((2, 40, 64))).bfloat16(), 32)
    q, s = lib.moe_quantize_weights_int4(torch.empty(0, 16, 128, device=DEV), 128)
    assert q.shape == (0, 16, 64) and s.shape == (0, 1, 16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-44, 1e-40, 3e-38, 1e-36, 1e-31, 6e-31, 1e-20, 1e20, 5e30, 1e31, 3e38])
def test_quantize_every_magnitude(lib, size, dtype):
    """Scales that underflow, reciprocals that would overflow, the two sides of the
    border to the divided form."""
    g = np.random.default_rng(3)
    w = np.clip(g.standard_normal((1, 20, 256)), -1, 1) * size
    _same(lib, torch.from_numpy(w).to(dtype), 32)


def test_quantize_ties(lib):
    """Every bf16 significand as a group's largest against every bf16 value of the
    five binades below it, both signs: quotients that lie on a tie among them."""
    m = np.arange(128, 256, dtype=np.float64)
    low = np.concatenate([m * 2.0 ** -i for i in range(1, 6)])
    rows = []
    for M in range(128, 256):
        r = np.concatenate([np.minimum(m, M), low, -np.minimum(m, M), -low])
        parts = r.reshape(-1, 31 if len(r) % 31 == 0 else 32)
        parts = np.concatenate([np.full((len(parts), 1), float(M)), parts[:, :31]], axis=1)
        rows.append(parts.reshape(-1))
    w = torch.from_numpy(np.stack(rows))[None]
    assert w.shape[2] % 64 == 0
    for scale in (1.0, 2.0 ** -9, 2.0 ** 90):
        _same(lib, (w * scale).bfloat16(), 32)
        _same(lib, (w * scale).float(), 32)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_not_finite(lib, group):
    w = torch.randn(1, 5, 256)
    w[0, 0, 3], w[0, 1, 255], w[0, 2, 128] = float("nan"), float("inf"), -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        _same(lib, w.to(dtype), group)


def test_every_nibble_with_any_scale(lib):
    """All 16 values at every place of a word; scales of all eight bits, rounded."""
    g = np.random.default_rng(2)
    q = (np.arange(16)[:, None] + np.arange(64)[None, :]) % 16 - 8
    packed = torch.from_numpy(S.pack_int4(q)).to(DEV)
    s = torch.from_numpy(g.standard_normal((2, 16)) * 3).bfloat16()
    back = lib.moe_dequantize_weights_int4(packed, s.to(DEV))
    assert np.array_equal(np64(back), S.weights_int4(packed.cpu().numpy()[None], np64(s)[None])[0])


# ---- products ------------------------------------------------------------------

def _case(seed, counts, Kd, Nout, group, five=True):
    """Rows, offsets, bytes, scales; five: scales of five significant bits."""
    g = np.random.default_rng(seed)
    E, N = len(counts), int(sum(counts))
    x = torch.from_numpy(g.standard_normal((N, Kd))).bfloat16()
    q = S.pack_int4(g.integers(-8, 8, (E, Nout, Kd)))
    s = (16 + g.integers(0, 16, (E, Kd // group, Nout))) * 2.0 ** -13 if five else \
        g.random((E, Kd // group, Nout)) * 2e-3 + 1e-4
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return x, torch.from_numpy(off), torch.from_numpy(q), torch.from_numpy(s).bfloat16()


SHAPES = [
    ([5], 64, 64, 64), ([1], 64, 128, 32), ([0, 3, 0, 130, 0], 128, 320, 64), ([64, 65, 1, 127, 128, 129], 256, 192, 128),
    ([700, 0, 20], 1024, 576, 32), ([300], 2048, 256, 128), ([0, 0], 64, 64, 32), ([257, 3], 4160, 128, 64),
    ([1500, 90, 600], 192, 768, 32), ([33, 40], 1088, 64, 64), ([19], 640, 1024, 128), ([321, 160, 161], 320, 64, 32),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("five", [True, False])
@pytest.mark.parametrize("counts,Kd,Nout,group", SHAPES)
def test_down_proj_int4(lib, counts, Kd, Nout, group, five, out_dtype):
    x, off, q, s = _case(Kd + Nout, counts, Kd, Nout, group, five)
    N = x.shape[0]
    out = torch.full((N + 3, Nout), 7.0, dtype=out_dtype, device=DEV)      # capacity past the last row
    xp = torch.cat([x, torch.full((3, Kd), float("nan"), dtype=torch.bfloat16)])
    lib.moe_down_proj_int4(xp.to(DEV), off.to(DEV), q.to(DEV), s.to(DEV), expanded=out)
    W = S.weights_int4(q.numpy(), np64(s))
    want = S.linear_float(np64(x), off.numpy(), W)
    mag = S.linear_float(np.abs(np64(x)), off.numpy(), np.abs(W))
    assert_elementwise(np64(out)[:N], want, mag, Kd + 2, "bf16" if out_dtype == torch.bfloat16 else "f32", "product")
    assert (out[N:] == 7.0).all()


@pytest.mark.parametrize("N,Kd,Nout,group", [(1, 64, 64, 64), (19, 4096, 512, 32), (200, 512, 192, 128), (1025, 320, 1088, 64)])
def test_dense_int4(lib, N, Kd, Nout, group):
    x, off, q, s = _case(N, [N], Kd, Nout, group)
    out = lib.moe_down_proj_int4(x.to(DEV), None, q.to(DEV), s.to(DEV), out_dtype=torch.float32)
    W = S.weights_int4(q.numpy(), np64(s))
    want = S.linear_float(np64(x), off.numpy(), W)
    mag = S.linear_float(np.abs(np64(x)), off.numpy(), np.abs(W))
    assert_elementwise(np64(out), want, mag, Kd + 2, "f32", "dense")


@pytest.mark.parametrize("five", [True, False])
@pytest.mark.parametrize("counts,Kd,Nout,group", SHAPES)
def test_gate_up_swiglu_int4(lib, counts, Kd, Nout, group, five):
    x, off, qg, sg = _case(Kd * 3 + Nout, counts, Kd, Nout, group, five)
    _, _, qu, su = _case(Kd * 5 + Nout, counts, Kd, Nout, group, five)
    N = x.shape[0]
    act = torch.full((N + 2, Nout), 5.0, dtype=torch.bfloat16, device=DEV)
    xp = torch.cat([x, torch.zeros(2, Kd, dtype=torch.bfloat16)])
    lib.moe_gate_up_swiglu_int4(xp.to(DEV), off.to(DEV), qg.to(DEV), sg.to(DEV), qu.to(DEV), su.to(DEV), act=act)
    Wg, Wu = S.weights_int4(qg.numpy(), np64(sg)), S.weights_int4(qu.numpy(), np64(su))
    g, u = S.linear_float(np64(x), off.numpy(), Wg), S.linear_float(np64(x), off.numpy(), Wu)
    want = S._silu(g) * u
    ax = np.abs(np64(x))
    dg = (Kd + 4) * U32 * S.linear_float(ax, off.numpy(), np.abs(Wg))
    du = (Kd + 4) * U32 * S.linear_float(ax, off.numpy(), np.abs(Wu))
    # silu' in [-0.1, 1.1]; e^-g takes |g| 2^-24 from its argument, then 8 rounded operations
    bound = 1.1 * np.abs(u) * dg + np.abs(S._silu(g)) * du + (np.abs(g) + 16) * 2 * U32 * np.abs(want)
    bound = bound + ulp(np.maximum(np.abs(np64(act)[:N]), np.abs(want)), "bf16")
    assert np.all(np.abs(np64(act)[:N] - want) <= bound)
    assert (act[N:] == 5.0).all()


def test_scale_that_is_nan_stays_in_its_channel(lib):
    x, off, q, s = _case(9, [150, 40], 128, 64, 64)
    s[1, 0, 17] = float("nan")
    out = lib.moe_down_proj_int4(x.to(DEV), off.to(DEV), q.to(DEV), s.to(DEV))
    assert torch.isnan(out[150:, 17]).all()
    out[150:, 17] = 0
    assert torch.isfinite(out).all()


def test_row_that_is_nan_stays_alone(lib):
    x, off, q, s = _case(9, [150, 40], 192, 64, 64)
    x[100, 3] = float("nan")
    out = lib.moe_down_proj_int4(x.to(DEV), off.to(DEV), q.to(DEV), s.to(DEV))
    assert torch.isnan(out[100]).all()
    out[100] = 0
    assert torch.isfinite(out).all()


def test_corrupt_offsets_stay_inside(lib):
    """Offsets that fall, pass the buffer or are negative are taken as the nearest
    ones in order: no row outside is touched."""
    x, _, q, s = _case(4, [40, 40, 40], 128, 64, 32)
    W = S.weights_int4(q.numpy(), np64(s))
    for off, eff in (([0, 50, 30, 90], [0, 50, 50, 90]), ([-5, 20, 500, 70], [0, 20, 120, 120])):
        out = torch.full((123, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        lib.moe_down_proj_int4(x.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), q.to(DEV), s.to(DEV),
                               expanded=out[:120])
        want = S.linear_float(np64(x), eff, W)
        mag = S.linear_float(np.abs(np64(x)), eff, np.abs(W))
        n = eff[-1]
        assert_elementwise(np64(out)[:n], want[:n], mag[:n], 130, "bf16", "rows")
        assert (out[n:] == 3.0).all()


@pytest.mark.parametrize("per", [160, 96, 64, 8])
def test_products_repeat_in_every_launch(lib, per):
    """Every one of thousands of launches of both products in all forms is compared,
    on the device."""
    E, H, I = 64, 1024, 768
    g = torch.Generator(device=DEV).manual_seed(per + 1)
    off = torch.arange(0, E + 1, dtype=torch.int32, device=DEV) * per
    x = torch.randn(E * per, H, device=DEV, generator=g).bfloat16()
    wg, wu = (torch.randint(0, 256, (E, I, H // 2), device=DEV, generator=g, dtype=torch.uint8) for _ in range(2))
    s = (torch.rand(E, H // 64, I, device=DEV, generator=g) * 1e-2).bfloat16()
    st = lib.new_status()
    up = lib.moe_gate_up_swiglu_int4(x, off, wg, s, wu, s, dev_status=st).clone()
    down = lib.moe_down_proj_int4(x, off, wg, s, dev_status=st).clone()
    differ = torch.zeros((), dtype=torch.bool, device=DEV)
    for _ in range(3000):
        u = lib.moe_gate_up_swiglu_int4(x, off, wg, s, wu, s, dev_status=st)
        d = lib.moe_down_proj_int4(x, off, wg, s, dev_status=st)
        differ |= (u != up).any() | (d != down).any()
    assert not bool(differ) and int(st) == 0


def test_prompt_path_in_4_bits_captured(lib):
    """Weights to 4 bits, then routing, gate/up, down and the weighted sum captured
    once and replayed with new tokens, on a stream of its own."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, H, E, K, I = 300, 256, 16, 4, 192
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    W = [rnd(E, I, H) * 0.06, rnd(E, I, H) * 0.06, rnd(E, H, I) * 0.06]
    (wg, gs), (wu, us), (wd, ds) = (lib.moe_quantize_weights_int4(w, 64) for w in W)
    logits, bias, x = rnd(T, E), rnd(E) * 0.1, rnd(T, H).bfloat16()
    st = lib.new_status()

    def step():
        ids, probs = lib.moe_router_topk_grouped(logits, K, bias=bias, num_groups=4, top_groups=2, group_top=2, dev_status=st)
        r = lib.moe_permute(x, ids, E, dev_status=st)
        act = lib.moe_gate_up_swiglu_int4(r.permuted, r.expert_offsets, wg, gs, wu, us, dev_status=st)
        y = lib.moe_down_proj_int4(act, r.expert_offsets, wd, ds, dev_status=st)
        return ids, probs, lib.moe_unpermute(y, r.row_map, probs, T, K)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    w = [lib.moe_dequantize_weights_int4(*p).double() for p in ((wg, gs), (wu, us), (wd, ds))]
    for seed in range(3):
        g2 = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g2, device=DEV))
        logits.copy_(torch.randn(T, E, generator=g2, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        ids, probs, out = got
        i, xs = ids.long(), x.double()
        h = torch.nn.functional.silu(torch.einsum("tkih,th->tki", w[0][i], xs)) * torch.einsum("tkih,th->tki", w[1][i], xs)
        want = torch.einsum("tk,tkhi,tki->th", probs.double(), w[2][i], h)
        # act, the expert's row and the result are rounded to bf16: 2^-9 / sqrt(3) rms each
        assert float((out.double() - want).norm() / want.norm()) < 0.005
    assert int(st) == 0


# Where a form begins or ends: rows of one tile and one more, tiles of 64 rows that
# all have a pair of their own, two pairs to a tile (2048 inputs and more, uneven
# halves of 9 and of 17 stages), with and without offsets.
FORMS = [(64, 2048, 1024), (65, 2048, 1024), (200, 1024, 2048), (320, 2304, 1088), (48, 4352, 256), (1, 2048, 64),
         (33, 2112, 4096), (500, 512, 512)]


@pytest.mark.parametrize("N,Kd,Nout", FORMS)
def test_dense_forms(lib, N, Kd, Nout):
    x, off, q, s = _case(N + Kd, [N], Kd, Nout, 64, five=False)
    W = S.weights_int4(q.numpy(), np64(s))
    want = S.linear_float(np64(x), off.numpy(), W)
    mag = S.linear_float(np.abs(np64(x)), off.numpy(), np.abs(W))
    for o in (None, off.to(DEV)):
        out = lib.moe_down_proj_int4(x.to(DEV), o, q.to(DEV), s.to(DEV), out_dtype=torch.float32)
        assert_elementwise(np64(out), want, mag, Kd + 2, "f32", "dense")


@pytest.mark.parametrize("counts,Kd,Nout", [([3, 0, 60, 1], 2048, 256), ([20, 64, 0, 33, 1, 0, 0, 9], 2304, 320)])
def test_two_pairs_to_a_tile_of_gate_up(lib, counts, Kd, Nout):
    x, off, qg, sg = _case(Kd + 1, counts, Kd, Nout, 64)
    _, _, qu, su = _case(Kd + 2, counts, Kd, Nout, 64)
    act = lib.moe_gate_up_swiglu_int4(x.to(DEV), off.to(DEV), qg.to(DEV), sg.to(DEV), qu.to(DEV), su.to(DEV))
    Wg, Wu = S.weights_int4(qg.numpy(), np64(sg)), S.weights_int4(qu.numpy(), np64(su))
    g, u = S.linear_float(np64(x), off.numpy(), Wg), S.linear_float(np64(x), off.numpy(), Wu)
    want, ax = S._silu(g) * u, np.abs(np64(x))
    dg = (Kd + 4) * U32 * S.linear_float(ax, off.numpy(), np.abs(Wg))
    du = (Kd + 4) * U32 * S.linear_float(ax, off.numpy(), np.abs(Wu))
    bound = 1.1 * np.abs(u) * dg + np.abs(S._silu(g)) * du + (np.abs(g) + 16) * 2 * U32 * np.abs(want)
    assert np.all(np.abs(np64(act) - want) <= bound + ulp(np.maximum(np.abs(np64(act)), np.abs(want)), "bf16"))


# Tiles of one accumulator: up to 80 and up to 128 rows per expert on average, with
# experts of none, of more than one tile takes and of more than two, and with more
# tiles than pairs.
ONE = [([70, 0, 129, 1, 33, 64, 150, 0, 40, 80], 320, 64), ([128] * 3 + [0, 0, 16], 640, 128),
       ([70, 0, 129, 1, 160, 64, 257, 0], 320, 32), ([161, 0, 320, 31], 64, 64), ([128, 128, 128], 512, 128)]


@pytest.mark.parametrize("counts,Kd,group", ONE)
def test_one_accumulator_to_a_tile(lib, counts, Kd, group):
    Nout, n = 5248, 2624
    x, off, q, s = _case(Kd, counts, Kd, Nout, group, five=False)
    ax = np.abs(np64(x))
    W = S.weights_int4(q.numpy(), np64(s))
    want, mag = S.linear_float(np64(x), off.numpy(), W), S.linear_float(ax, off.numpy(), np.abs(W))
    q, s = q.to(DEV), s.to(DEV)
    for dt, name in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        out = lib.moe_down_proj_int4(x.to(DEV), off.to(DEV), q, s, out_dtype=dt)
        assert_elementwise(np64(out), want, mag, Kd + 2, name, "rows")
    gate, up = slice(0, n), slice(n, 2 * n)
    part = [t for c in (gate, up) for t in (q[:, c].contiguous(), s[:, :, c].contiguous())]
    act = lib.moe_gate_up_swiglu_int4(x.to(DEV), off.to(DEV), *part)
    g, u = want[:, gate], want[:, up]
    dg, du = (Kd + 4) * U32 * mag[:, gate], (Kd + 4) * U32 * mag[:, up]
    act_want = S._silu(g) * u
    bound = 1.1 * np.abs(u) * dg + np.abs(S._silu(g)) * du + (np.abs(g) + 16) * 2 * U32 * np.abs(act_want)
    bound = bound + ulp(np.maximum(np.abs(np64(act)), np.abs(act_want)), "bf16")
    assert np.all(np.abs(np64(act) - act_want) <= bound)


def test_two_pairs_to_a_tile_repeat_in_every_launch(lib):
    """Sums that one pair writes into another's shared memory, thousands of times."""
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(19, 2048, device=DEV, generator=g).bfloat16()
    q = torch.randint(0, 256, (1, 4096, 1024), device=DEV, generator=g, dtype=torch.uint8)
    s = (torch.rand(1, 32, 4096, device=DEV, generator=g) * 1e-2).bfloat16()
    st = lib.new_status()
    want = lib.moe_down_proj_int4(x, None, q, s, dev_status=st).clone()
    differ = torch.zeros((), dtype=torch.bool, device=DEV)
    for _ in range(3000):
        differ |= (lib.moe_down_proj_int4(x, None, q, s, dev_status=st) != want).any()
    assert not bool(differ) and int(st) == 0
