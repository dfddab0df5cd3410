"""Products over 4-bit weights whose rows lie in both CTAs of a pair: each launch
multiplies its own rows.  Two inputs take turns, so that rows that a launch reads
before they have landed are another input's."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("E,per,Kd,Nout", [
    (64, 8, 1024, 768),     # few rows, 256-deep stages
    (1, 19, 2048, 4096),    # two pairs to a tile
    (24, 64, 1088, 1344),   # one accumulator of up to 128 rows
    (24, 96, 576, 1344),    # one accumulator of up to 160 rows
    (16, 250, 512, 1024),   # two accumulators
    (9, 321, 2112, 640),    # the same, more than one tile an expert
])
def test_each_launch_multiplies_its_own_rows(lib, E, per, Kd, Nout):
    g = torch.Generator(device=DEV).manual_seed(per)
    off = torch.arange(0, E + 1, dtype=torch.int32, device=DEV) * per
    xs = [torch.randn(E * per, Kd, device=DEV, generator=g).bfloat16() * s for s in (1.0, 64.0)]
    w = [torch.randint(0, 256, (E, Nout, Kd // 2), device=DEV, generator=g, dtype=torch.uint8) for _ in range(2)]
    s = (torch.rand(E, Kd // 64, Nout, device=DEV, generator=g) * 1e-3).bfloat16()
    st = lib.new_status()
    W = [lib.moe_dequantize_weights_int4(v, s).double() for v in w]
    want = []
    for x in xs:
        want.append((lib.moe_gate_up_swiglu_int4(x, off, w[0], s, w[1], s, dev_status=st).clone(),
                     lib.moe_down_proj_int4(x, off, w[0], s, dev_status=st).clone()))
        y = torch.bmm(x.double().view(E, per, Kd), W[0].transpose(1, 2)).view(E * per, Nout)
        u = torch.bmm(x.double().view(E, per, Kd), W[1].transpose(1, 2)).view(E * per, Nout)
        # one rounding to bf16 (2^-8 of a value at most) and fp32 sums
        for got, ref in zip(want[-1], (torch.nn.functional.silu(y) * u, y)):
            assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -8
    differ = torch.zeros((), dtype=torch.bool, device=DEV)
    for i in range(1000):
        up = lib.moe_gate_up_swiglu_int4(xs[i % 2], off, w[0], s, w[1], s, dev_status=st)
        down = lib.moe_down_proj_int4(xs[i % 2], off, w[0], s, dev_status=st)
        differ |= (up != want[i % 2][0]).any() | (down != want[i % 2][1]).any()
    assert not bool(differ) and int(st) == 0


@pytest.mark.parametrize("counts,N", [
    ({5: 1500}, 1500),                        # one of 128 experts has every row: 12 rows an expert on average
    ({0: 700, 127: 803}, 1600),               # two of them, and rows behind the last
    ({3: 5000, 70: 1, 90: 600}, 5601),        # 44 on average
    ({2: 9000, 3: 9}, 9009),                  # 71
    ({40: 13000, 41: 400}, 13400),            # 105
])
def test_rows_on_few_of_many_experts(lib, counts, N):
    """The form is chosen by the average: here most experts have no rows and some
    many times what a tile takes."""
    E, Kd, Nout = 128, 320, 640
    g = torch.Generator(device=DEV).manual_seed(N)
    n = torch.zeros(E, dtype=torch.int64)
    for e, c in counts.items():
        n[e] = c
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    x = torch.randn(N, Kd, device=DEV, generator=g).bfloat16()
    w = [torch.randint(0, 256, (E, Nout, Kd // 2), device=DEV, generator=g, dtype=torch.uint8) for _ in range(2)]
    s = (torch.rand(E, Kd // 64, Nout, device=DEV, generator=g) * 1e-2).bfloat16()
    at = off.int().to(DEV)
    down = torch.full((N, Nout), 7.0, device=DEV)
    up = torch.full((N, Nout), 7.0, dtype=torch.bfloat16, device=DEV)
    lib.moe_down_proj_int4(x, at, w[0], s, expanded=down)
    lib.moe_gate_up_swiglu_int4(x, at, w[0], s, w[1], s, act=up)
    for e in counts:
        lo, hi = int(off[e]), int(off[e + 1])
        W = [lib.moe_dequantize_weights_int4(v[e], s[e]).double() for v in w]
        xe = x[lo:hi].double()
        y, u = xe @ W[0].t(), xe @ W[1].t()
        # (Kd + 2 rounded additions of exact terms)
        assert bool(((down[lo:hi].double() - y).abs() <= (Kd + 2) * 2.0 ** -24 * (xe.abs() @ W[0].abs().t())).all())
        act = torch.nn.functional.silu(y) * u
        # one rounding to bf16, 2^-8 of a value at most
        assert float((up[lo:hi].double() - act).norm() / act.norm()) < 2.0 ** -8
    assert bool((down[int(off[E]):] == 7).all()) and bool((up[int(off[E]):] == 7).all())
