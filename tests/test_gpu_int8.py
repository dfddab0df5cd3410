"""GPU parity of the 8-bit rows and products against the float64 oracle.

The rows are compared bit for bit.  A product's sum of exact integer products
is exact in fp32 while every partial sum stays under 2^24, which Kd <= 1040
guarantees (127^2 * 1040 < 2^24): then three rounded operations (two scales,
the conversion) and the store remain.  Past that, each of the Kd additions may
round: (Kd + 3) 2^-24 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import serving_oracle as S
from gpu_util import U32, assert_elementwise, np64, ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rows(seed, T, H, dtype):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((T, H))).to(dtype)
    if T > 4:
        x[1] = 0
        x[2, H // 2] = 1000.0
        x[3] = torch.round(x[3] * 4) / 4
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(1, 16), (7, 48), (33, 2048), (5, 7168), (3, 16384), (300, 272)])
def test_quantize_rows_bit_exact(lib, T, H, dtype):
    x = _rows(T + H, T, H, dtype)
    q, s = lib.moe_quantize_rows(x.to(DEV))
    w_q, w_s = S.quantize_rows(np64(x))
    assert np.array_equal(np64(q), w_q)
    assert np.array_equal(s.cpu().numpy(), w_s)


def test_quantize_rows_not_finite_and_tiny(lib):
    x = torch.ones(6, 64)
    x[0, 5], x[1, 63], x[2, 0] = float("inf"), float("nan"), float("-inf")
    x[3] = 1e-40                                   # subnormal rows keep their scale
    x[4] = 3e38
    x[4, 1::2] = -1e38
    q, s = lib.moe_quantize_rows(x.to(DEV))
    w_q, w_s = S.quantize_rows(x[3:6].numpy())
    assert torch.isnan(s[:3]).all() and (q[:3] == 0).all()
    assert np.array_equal(s[5:].cpu().numpy(), w_s[2:]) and np.array_equal(np64(q)[5], w_q[2])
    assert (q[3] == 127).all() and abs(float(s[3]) * 127 / 1e-40 - 1) < 1e-2
    # 127 * 3e38 would pass fp32's range
    assert abs(float(s[4]) / (3e38 / 127) - 1) < 1e-6
    assert (q[4, 0::2] == 127).all() and (q[4, 1::2] == -42).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-40, 3e-38, 2e-37, 1e-36, 1e-30, 1e37, 3e38])
def test_quantize_rows_of_every_magnitude(lib, dtype, size):
    """127 / top is out of fp32's range below 2^-121."""
    g = np.random.default_rng(5)
    x = torch.from_numpy(np.clip(g.standard_normal((9, 400)), -1, 1) * size).to(dtype)
    q, s = lib.moe_quantize_rows(x.to(DEV))
    w_q, w_s = S.quantize_rows(np64(x))
    assert np.array_equal(np64(q), w_q)
    assert np.array_equal(s.cpu().numpy(), w_s)


def test_quantize_rows_every_bf16_quotient(lib):
    """Every mantissa of a row's largest magnitude against every bf16 value of the
    nine binades below it, both signs: all the quotients there are."""
    m = np.arange(128, 256, dtype=np.float64)
    low = (m[None, :] * 2.0 ** -np.arange(1, 10)[:, None]).reshape(-1)
    rows = []
    for M in range(128, 256):
        r = np.concatenate([[M], np.minimum(m, M), low, -np.minimum(m, M), -low])
        rows.append(np.pad(r, (0, -len(r) % 16)))
    x = torch.from_numpy(np.stack(rows)).bfloat16()
    assert np.array_equal(np64(x), np.stack(rows))
    for scale in (1.0, 2.0 ** -9, 2.0 ** 100):
        q, s = lib.moe_quantize_rows((x * scale).to(DEV))
        exact = 127 * np64(x) / np64(x).max(1, keepdims=True)      # ties are exact in float64
        assert np.array_equal(np64(q), np.rint(exact))
        assert np.array_equal(np64(q), S.quantize_rows(np64(x * scale))[0])


@pytest.mark.parametrize("T,H,E,K,special", [(40, 64, 8, 4, 3), (1, 2048, 16, 8, 0), (257, 208, 24, 5, 2)])
def test_quantize_rows_into_expert_major_order(lib, T, H, E, K, special):
    g = np.random.default_rng(T)
    ids = torch.from_numpy(np.argsort(g.random((T, E + special)), axis=1)[:, :K].astype(np.int32))
    x = _rows(T, T, H, torch.bfloat16)
    r = lib.moe_permute(None, ids.to(DEV), E, special)
    q = torch.full((T * K, H), 99, dtype=torch.int8, device=DEV)
    s = torch.full((T * K,), 99.0, device=DEV)
    lib.moe_quantize_rows(x.to(DEV), row_map=r.row_map, K=K, q=q, scale=s)
    si, rm, _, off = O.permute_routing(ids.numpy(), E, special)
    n = int(off[-1])
    w_q, w_s = S.quantize_rows(np64(x))
    assert np.array_equal(np64(q)[:n], w_q[si // K]) and np.array_equal(s.cpu().numpy()[:n], w_s[si // K])
    assert (q[n:] == 99).all() and (s[n:] == 99).all()              # rows without a slot stay


def _case(seed, counts, Kd, Nout, full=False):
    g = np.random.default_rng(seed)
    E, N = len(counts), int(sum(counts))
    lo = 127 if full else 1
    q = g.integers(lo, 128, (N, Kd)) * (1 if full else g.choice([-1, 1], (N, Kd)))
    W = g.integers(-127, 128, (E, Nout, Kd))
    if full:
        W[:] = 127
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return (torch.from_numpy(q.astype(np.int8)), torch.from_numpy(g.random(N).astype(np.float32) + 0.1),
            torch.from_numpy(off), torch.from_numpy(W.astype(np.int8)),
            torch.from_numpy((g.random((E, Nout)) * 1e-2 + 1e-3).astype(np.float32)))


def _mag(q, rs, off, W, cs):
    return S.linear_int8(np.abs(np64(q)), np64(rs), off.numpy(), np.abs(np64(W)), np64(cs))


SHAPES = [
    ([5], 16, 16), ([1], 64, 48), ([0, 3, 0, 130, 0], 96, 272), ([64, 65, 1, 127, 128, 129], 256, 304),
    ([700, 0, 20], 1024, 528), ([300], 2048, 256), ([0, 0], 64, 64), ([257, 3], 4112, 80),
    ([1500, 90, 600], 192, 768),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,Kd,Nout", SHAPES)
def test_down_proj_int8(lib, counts, Kd, Nout, out_dtype):
    q, rs, off, W, cs = _case(Kd + Nout, counts, Kd, Nout)
    N = q.shape[0]
    out = torch.full((N + 3, Nout), 7.0, dtype=out_dtype, device=DEV)      # capacity past the last row
    qp = torch.cat([q, torch.ones(3, Kd, dtype=torch.int8)])
    rp = torch.cat([rs, torch.ones(3)])
    lib.moe_down_proj_int8(qp.to(DEV), rp.to(DEV), off.to(DEV), W.to(DEV), cs.to(DEV), expanded=out)
    want = S.linear_int8(np64(q), np64(rs), off.numpy(), np64(W), np64(cs))
    n = 3 if Kd <= 1040 else Kd + 3
    assert_elementwise(np64(out)[:N], want, _mag(q, rs, off, W, cs) if Kd > 1040 else np.abs(want), n,
                       "bf16" if out_dtype == torch.bfloat16 else "f32", "product")
    assert (out[N:] == 7.0).all()


def test_down_proj_int8_largest_sums(lib):
    """Every product 127^2: the sum passes 2^24, and 127^2 Kd is representable
    as rounded by any order of additions within the bound."""
    q, rs, off, W, cs = _case(1, [40], 8192, 64, full=True)
    out = lib.moe_down_proj_int8(q.to(DEV), rs.to(DEV), off.to(DEV), W.to(DEV), cs.to(DEV),
                                 out_dtype=torch.float32)
    want = S.linear_int8(np64(q), np64(rs), off.numpy(), np64(W), np64(cs))
    assert_elementwise(np64(out), want, want, 8195, "f32", "largest sums")


@pytest.mark.parametrize("N,Kd,Nout", [(1, 64, 64), (200, 512, 160), (1025, 320, 1040)])
def test_dense_int8(lib, N, Kd, Nout):
    q, rs, off, W, cs = _case(N, [N], Kd, Nout)
    out = lib.moe_down_proj_int8(q.to(DEV), rs.to(DEV), None, W.to(DEV), cs.to(DEV), out_dtype=torch.float32)
    want = S.linear_int8(np64(q), np64(rs), off.numpy(), np64(W), np64(cs))
    assert_elementwise(np64(out), want, np.abs(want), 3, "f32", "dense")


def test_int8_minus_128(lib):
    """-128 is a legal byte of either operand."""
    q = torch.full((70, 128), -128, dtype=torch.int8)
    W = torch.full((1, 32, 128), -128, dtype=torch.int8)
    W[0, 1::2] = 127
    out = lib.moe_down_proj_int8(q.to(DEV), torch.ones(70, device=DEV), None, W.to(DEV),
                                 torch.ones(1, 32, device=DEV), out_dtype=torch.float32)
    assert (out[:, 0::2] == 128.0 * 128 * 128).all() and (out[:, 1::2] == -128.0 * 127 * 128).all()


@pytest.mark.parametrize("counts,Kd,Nout", SHAPES)
def test_gate_up_swiglu_int8(lib, counts, Kd, Nout):
    q, rs, off, Wg, gs = _case(Kd * 3 + Nout, counts, Kd, Nout)
    _, _, _, Wu, us = _case(Kd * 5 + Nout, counts, Kd, Nout)
    gs = gs * (16.0 / Kd)                         # pre-activations of a few units
    N = q.shape[0]
    act = lib.moe_gate_up_swiglu_int8(q.to(DEV), rs.to(DEV), off.to(DEV), Wg.to(DEV), gs.to(DEV),
                                      Wu.to(DEV), us.to(DEV))
    want, g, u = S.gate_up_swiglu_int8(np64(q), np64(rs), off.numpy(), np64(Wg), np64(gs), np64(Wu), np64(us))
    if Kd <= 1040:
        dg, du = 4 * U32 * np.abs(g), 4 * U32 * np.abs(u)
    else:
        dg = (Kd + 4) * U32 * _mag(q, rs, off, Wg, gs)
        du = (Kd + 4) * U32 * _mag(q, rs, off, Wu, us)
    # silu' in [-0.1, 1.1]; e^-g takes |g| 2^-24 from its argument, then 8 rounded operations
    bound = 1.1 * np.abs(u) * dg + np.abs(S._silu(g)) * du + (np.abs(g) + 16) * 2 * U32 * np.abs(want)
    bound = bound + ulp(np.maximum(np.abs(np64(act)), np.abs(want)), "bf16")
    assert np.all(np.abs(np64(act) - want) <= bound)
    assert act.shape == (N, Nout)


def test_gate_up_swiglu_int8_saturated_gates(lib):
    """g far below and above the range of e^g."""
    q = torch.tensor([[127] * 16, [-127] * 16, [0] * 16], dtype=torch.int8, device=DEV)
    W = torch.full((1, 16, 16), 127, dtype=torch.int8, device=DEV)
    one = torch.ones(1, 16, device=DEV)
    act = lib.moe_gate_up_swiglu_int8(q, torch.ones(3, device=DEV), None, W, one, W, one * 1e-3)
    s = 127.0 * 127 * 16
    assert torch.allclose(act[0].float(), torch.tensor(s * s * 1e-3, device=DEV), rtol=2 ** -8)
    assert (act[1] == 0).all() and (act[2] == 0).all()


def test_row_with_nan_scale_stays_alone(lib):
    q, rs, off, W, cs = _case(9, [150, 40], 128, 64)
    rs[100] = float("nan")
    out = lib.moe_down_proj_int8(q.to(DEV), rs.to(DEV), off.to(DEV), W.to(DEV), cs.to(DEV))
    assert torch.isnan(out[100]).all()
    keep = np.arange(190) != 100
    assert torch.isfinite(out[torch.from_numpy(keep).to(DEV)]).all()


def test_int8_layer_of_a_prompt(lib):
    """router -> routing -> 8-bit gate/up -> 8-bit down -> unpermute, the way a
    prompt runs, against the same path of float weights: 8-bit rounding of
    both operands stays within 3 % of the layer's output (uniform rounding
    error of step/sqrt(12) on each factor: 1 % of the rms each for normal
    rows of this length, four factors)."""
    g = torch.Generator(device=DEV).manual_seed(5)
    T, H, E, K, I = 500, 256, 16, 4, 192
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = rnd(T, H).bfloat16()
    Wg, Wu, Wd = rnd(E, I, H) * 0.06, rnd(E, I, H) * 0.06, rnd(E, H, I) * 0.06
    ids, probs = lib.moe_router_topk(rnd(T, E), K)
    r = lib.moe_permute(None, ids, E)
    wq = [lib.moe_quantize_rows(w.reshape(-1, w.shape[2])) for w in (Wg, Wu, Wd)]
    wq = [(a.view(w.shape), s.view(w.shape[:2])) for (a, s), w in zip(wq, (Wg, Wu, Wd))]
    q, rs = lib.moe_quantize_rows(x, row_map=r.row_map, K=K)
    act = lib.moe_gate_up_swiglu_int8(q, rs, r.expert_offsets, *wq[0], *wq[1])
    aq, as_ = lib.moe_quantize_rows(act)
    y = lib.moe_down_proj_int8(aq, as_, r.expert_offsets, *wq[2])
    out = lib.moe_unpermute(y, r.row_map, probs, T, K)
    xs = x.double()[:, None]
    i = ids.long()
    h = torch.einsum("tkih,tah->tki", Wg.double()[i], xs), torch.einsum("tkih,tah->tki", Wu.double()[i], xs)
    want = torch.einsum("tk,tkhi,tki->th", probs.double(), Wd.double()[i], torch.nn.functional.silu(h[0]) * h[1])
    rel = float((out.double() - want).norm() / want.norm())
    assert rel < 0.03


@pytest.mark.parametrize("per", [96, 8])
def test_products_repeat(lib, per):
    """A late copy in one launch of thousands must not let a stage through early:
    many launches over more tiles than CTAs, in both forms (96 rows an expert, 8
    rows), give the same bytes and no error."""
    E, H, I = 64, 1024, 768
    g = torch.Generator(device=DEV).manual_seed(per)

    def ints(*shape):
        return torch.randint(-127, 128, shape, device=DEV, generator=g, dtype=torch.int8)

    off = torch.arange(0, E + 1, dtype=torch.int32, device=DEV) * per
    N = E * per
    x, wg, wu = ints(N, H), ints(E, I, H), ints(E, I, H)
    rs = torch.full((N,), 1e-3, device=DEV)
    cs = torch.full((E, I), 1e-3, device=DEV)
    st = lib.new_status()
    up = lib.moe_gate_up_swiglu_int8(x, rs, off, wg, cs, wu, cs, dev_status=st).clone()
    down = lib.moe_down_proj_int8(x, rs, off, wg, cs, dev_status=st).clone()
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(3000):
        u = lib.moe_gate_up_swiglu_int8(x, rs, off, wg, cs, wu, cs, dev_status=st)
        d = lib.moe_down_proj_int8(x, rs, off, wg, cs, dev_status=st)
        if i % 20 == 0:
            differ += (u != up).sum() + (d != down).sum()
    assert int(differ) == 0 and int(st) == 0


def test_new_outputs_are_filled_where_torch_fills_them(lib):
    """Under deterministic algorithms torch fills new memory (NaN, the largest
    integer): the rows that no call writes too, the bytes of any other memory not."""
    T, K, H, E, I = 24, 4, 64, 6, 32
    g = torch.Generator(device=DEV).manual_seed(8)
    ids = torch.rand(T, E + 4, generator=g, device=DEV).topk(K, dim=1).indices.int()
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    w = torch.randint(-127, 128, (E, I, H), generator=g, device=DEV, dtype=torch.int8)
    cs = torch.full((E, I), 1e-3, device=DEV)
    r = lib.moe_permute(None, ids, E, 4)
    n = int(r.expert_offsets[-1])
    assert 0 < n < T * K
    junk = [torch.full((T * K, m), 3, dtype=d, device=DEV)
            for m, d in ((H, torch.int8), (1, torch.float32), (I, torch.bfloat16))]
    del junk                                                        # (back to the allocator)
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        q, s = lib.moe_quantize_rows(x, row_map=r.row_map, K=K)
        act = lib.moe_gate_up_swiglu_int8(q, s, r.expert_offsets, w, cs, w, cs)
        y = lib.moe_down_proj_int8(q, s, r.expert_offsets, w, cs, out_dtype=torch.float32)
    finally:
        torch.use_deterministic_algorithms(before)
    assert (q[n:] == 127).all()
    for t in (s, act, y):
        assert torch.isnan(t[n:]).all() and torch.isfinite(t[:n]).all()


# Row lengths of every form: 1 to 4 chunks a thread at 32, 64, 128 and 256 threads
# a row, 8 chunks, and rows read twice (past 16384).
LENGTHS = [16, 256, 272, 512, 528, 768, 784, 1024, 1040, 1536, 1552, 2048, 2064, 4096, 4112, 8192, 8208, 16384,
           16400, 40000]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", LENGTHS)
def test_quantize_rows_of_every_length(lib, H, dtype):
    T, K, E = 11, 3, 5
    g = np.random.default_rng(H)
    x = _rows(H + 1, T, H, dtype)
    x[4, -1], x[5, 0], x[6, H // 2 + 1] = 50.0, -60.0, 70.0             # the largest at a row's ends
    x[7, -3] = float("nan")
    w_q, w_s = S.quantize_rows(np64(x))
    q, s = lib.moe_quantize_rows(x.to(DEV))
    assert np.array_equal(np64(q), w_q)
    assert np.array_equal(s.cpu().numpy(), w_s, equal_nan=True)
    ids = torch.from_numpy(np.argsort(g.random((T, E + 1)), axis=1)[:, :K].astype(np.int32))
    r = lib.moe_permute(None, ids.to(DEV), E, 1)                         # (one special id: rows that stay)
    q = torch.full((T * K, H), 99, dtype=torch.int8, device=DEV)
    s = torch.full((T * K,), 99.0, device=DEV)
    lib.moe_quantize_rows(x.to(DEV), row_map=r.row_map, K=K, q=q, scale=s)
    si, _, _, off = O.permute_routing(ids.numpy(), E, 1)
    n = int(off[-1])
    assert np.array_equal(np64(q)[:n], w_q[si[:n] // K])
    assert np.array_equal(s.cpu().numpy()[:n], w_s[si[:n] // K], equal_nan=True)
    assert (q[n:] == 99).all() and (s[n:] == 99).all()


@pytest.mark.parametrize("per", [96, 8])
def test_products_repeat_in_every_launch(lib, per):
    """Every one of thousands of launches of both products in both forms is
    compared, on the device."""
    E, H, I = 64, 1024, 768
    g = torch.Generator(device=DEV).manual_seed(per + 1)
    off = torch.arange(0, E + 1, dtype=torch.int32, device=DEV) * per
    N = E * per
    x = torch.randint(-127, 128, (N, H), device=DEV, generator=g, dtype=torch.int8)
    wg, wu = (torch.randint(-127, 128, (E, I, H), device=DEV, generator=g, dtype=torch.int8) for _ in range(2))
    rs, cs = torch.full((N,), 1e-3, device=DEV), torch.full((E, I), 1e-3, device=DEV)
    st = lib.new_status()
    up = lib.moe_gate_up_swiglu_int8(x, rs, off, wg, cs, wu, cs, dev_status=st).clone()
    down = lib.moe_down_proj_int8(x, rs, off, wg, cs, dev_status=st).clone()
    differ = torch.zeros((), dtype=torch.bool, device=DEV)
    for _ in range(3000):
        u = lib.moe_gate_up_swiglu_int8(x, rs, off, wg, cs, wu, cs, dev_status=st)
        d = lib.moe_down_proj_int8(x, rs, off, wg, cs, dev_status=st)
        differ |= (u != up).any() | (d != down).any()
    assert not bool(differ) and int(st) == 0
