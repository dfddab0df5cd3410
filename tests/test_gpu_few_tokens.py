"""GPU parity of the layer for a few tokens against the float64 oracle, with
the oracle's own bound of what fp32 sums and one bf16 rounding of act allow."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import np64, ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _data(seed, T, H, E, K, I, weights, special=0, shared=False):
    g = np.random.default_rng(seed)
    bf = lambda *s, std=1.0: torch.from_numpy((g.standard_normal(s) * std).astype(np.float32)).bfloat16()  # noqa: E731
    d = dict(tokens=bf(T, H),
             expert_ids=torch.from_numpy(np.argsort(g.random((T, E + special)), axis=1)[:, :K].astype(np.int32)),
             probs=torch.from_numpy(g.random((T, K)).astype(np.float32)),
             shared_x=bf(T, H) if shared else None, num_special=special)
    if weights == "bf16":
        d.update(W_gate=bf(E, I, H, std=0.05), W_up=bf(E, I, H, std=0.05), W_down=bf(E, H, I, std=0.05), scales=None)
    else:
        i8 = lambda *s: torch.from_numpy(g.integers(-128, 128, s).astype(np.int8))  # noqa: E731
        sc = lambda *s: torch.from_numpy((g.random(s) * 1e-3 + 1e-4).astype(np.float32))  # noqa: E731
        d.update(W_gate=i8(E, I, H), W_up=i8(E, I, H), W_down=i8(E, H, I), scales=(sc(E, I), sc(E, I), sc(E, H)))
    return d


def _dev(d):
    return {k: (v.to(DEV) if torch.is_tensor(v) else tuple(x.to(DEV) for x in v) if isinstance(v, tuple) else v)
            for k, v in d.items()}


def _oracle(d, mask=None):
    E = d["W_gate"].shape[0]
    sc = d["scales"]
    f = lambda v: None if v is None else np64(v)  # noqa: E731
    return S.layer_few_tokens(np64(d["tokens"]), d["expert_ids"].numpy(), d["probs"].numpy(), np64(d["W_gate"]),
                              np64(d["W_up"]), np64(d["W_down"]), E, d["num_special"],
                              None if mask is None else mask.numpy(), f(d["shared_x"]),
                              *((None,) * 3 if sc is None else (f(v) for v in sc)))


def _check(out, d, mask=None):
    want, bound = _oracle(d, mask)
    got = np64(out)
    assert got.shape == want.shape and np.all(np.isfinite(got))
    lim = bound + ulp(np.maximum(np.abs(got), np.abs(want)), "bf16")
    bad = np.abs(got - want) > lim
    assert not bad.any(), (int(bad.sum()), bad.size, float((np.abs(got - want) / lim).max()))


SIZES = [  # T, H, E, K, I
    (1, 64, 4, 1, 64), (1, 2048, 16, 8, 768), (3, 128, 8, 2, 192), (16, 512, 5, 3, 128), (17, 320, 64, 6, 64),
    (64, 256, 8, 8, 256), (33, 1088, 12, 4, 448), (64, 64, 200, 16, 64), (7, 7168, 6, 2, 64), (48, 192, 1, 1, 1024),
    (8, 448, 1024, 2, 64),
]


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("T,H,E,K,I", SIZES)
def test_few_tokens(lib, T, H, E, K, I, weights):
    d = _data(T + H + E, T, H, E, K, I, weights, shared=T % 2 == 1)
    _check(lib.moe_layer_few_tokens(**_dev(d)), d)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_all_on_one_expert(lib, weights):
    d = _data(1, 64, 320, 9, 2, 192, weights)
    d["expert_ids"][:, 0], d["expert_ids"][:, 1] = 7, 3
    _check(lib.moe_layer_few_tokens(**_dev(d)), d)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("dims", [1, 2])
def test_few_tokens_masks_and_special_ids(lib, dims, weights):
    d = _data(2, 20, 192, 6, 4, 128, weights, special=3, shared=True)
    g = np.random.default_rng(3)
    mask = torch.from_numpy((g.random((20,) if dims == 1 else (20, 4)) < 0.6).astype(np.uint8))
    mask[0] = 0                                                    # a token with nothing at all
    _check(lib.moe_layer_few_tokens(**_dev(d), active_mask=mask.to(DEV)), d, mask)
    d["shared_x"] = None
    out = lib.moe_layer_few_tokens(**_dev(d), active_mask=torch.zeros_like(mask).to(DEV))
    assert (out == 0).all()
    d["expert_ids"][:, :3] = torch.arange(6, 9, dtype=torch.int32)  # special ids, one real slot each
    d["expert_ids"][:, 3] %= 6
    _check(lib.moe_layer_few_tokens(**_dev(d)), d)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_bad_ids_are_flagged_and_skipped(lib, weights):
    d = _data(4, 9, 128, 8, 3, 64, weights)
    for t, row in ((1, [2, 8, 3]), (4, [-1, 0, 1]), (6, [5, 5, 5]), (8, [2**31 - 1, -2**31, 7])):
        d["expert_ids"][t] = torch.tensor(row, dtype=torch.int32)
    st = lib.new_status()
    out = lib.moe_layer_few_tokens(**_dev(d), dev_status=st)
    assert lib.moe_check_status(st) == lib.MOE_ERR_BAD_ID
    _check(out, d)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_keep_to_their_own_rows_and_experts(lib, weights):
    """NaN and infinities in one token's row, in one token's weight and in an
    expert that only one token chose do not reach the other tokens, nor do
    those of inactive slots reach any."""
    d = _data(5, 12, 128, 10, 2, 64, weights)
    d["expert_ids"][:] = torch.tensor([0, 1], dtype=torch.int32)
    d["expert_ids"][5] = torch.tensor([1, 9], dtype=torch.int32)   # the only token of expert 9
    d["tokens"][3, 7] = float("nan")
    d["tokens"][4, 9] = float("inf")
    d["probs"][6, 0] = float("nan")
    if weights == "bf16":
        d["W_gate"][9, 3, 3], d["W_down"][9, 2, 2] = float("nan"), float("inf")
    else:
        d["scales"][0][9, 3], d["scales"][2][9, 2] = float("nan"), float("inf")
    mask = torch.ones(12, 2, dtype=torch.uint8)
    mask[6, 0] = 0                                                 # its weight is NaN
    d["tokens"][7] = float("nan")
    mask[7] = 0                                                    # a padding token
    out = lib.moe_layer_few_tokens(**_dev(d), active_mask=mask.to(DEV)).cpu()
    assert torch.isnan(out[3]).any() and not torch.isfinite(out[4]).all() and not torch.isfinite(out[5]).all()
    assert (out[7] == 0).all()
    keep = [t for t in range(12) if t not in (3, 4, 5, 7)]
    clean = dict(d)
    clean.update({k: d[k][keep] for k in ("tokens", "expert_ids", "probs")})
    _check(out[keep], clean, mask[keep])


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_repeats_bit_for_bit_with_a_dirty_workspace(lib, weights):
    d = _dev(_data(6, 31, 512, 40, 6, 256, weights, shared=True))
    n = lib.moe_layer_few_tokens_workspace_size(31, 6, 512, 256, 40)
    first = None
    for fill in (0, 255, 85):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(2):                                          # again on what the last call left
            out = lib.moe_layer_few_tokens(**d, workspace=ws)
            first = out if first is None else first
            assert torch.equal(out, first)


def test_few_tokens_two_streams_and_a_graph(lib):
    """Two calls that may overlap, each with its own workspace, and a captured
    call replayed on new inputs."""
    a, b = _dev(_data(7, 8, 256, 16, 4, 128, "bf16")), _dev(_data(8, 64, 512, 32, 8, 256, "int8"))
    want = lib.moe_layer_few_tokens(**a), lib.moe_layer_few_tokens(**b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, d in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(lib._m.moe_layer_few_tokens(**d))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib._m.moe_layer_few_tokens(**a)
    c = _dev(_data(9, 8, 256, 16, 4, 128, "bf16"))
    for k in ("tokens", "expert_ids", "probs"):
        a[k].copy_(c[k])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lib.moe_layer_few_tokens(**a))


def test_few_tokens_matches_the_prompt_path(lib):
    """The same layer through permute, grouped GEMMs and combine (each of
    their stored tensors rounds to bf16: within 1e-2 of the largest output)."""
    d = _dev(_data(10, 50, 512, 24, 6, 256, "bf16", shared=True))
    out = lib.moe_layer_few_tokens(**d)
    r = lib.moe_permute(d["tokens"], d["expert_ids"], 24)
    _, y, _ = lib.moe_expert_mlp(r.permuted, r.expert_offsets, d["W_gate"], d["W_up"], d["W_down"])
    ref = lib.moe_combine(y, r.row_map, d["expert_ids"], d["probs"], 24, shared_x=d["shared_x"])
    assert float((out.float() - ref.float()).abs().max()) <= 1e-2 * float(ref.float().abs().max())


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_leave_no_flags_behind(lib, weights):
    """Whatever a call sets to show that its counters are clear, it takes back:
    the flags (64 bits a CTA, after the epoch's word) end as zeros, and the epoch
    has moved on."""
    d = _dev(_data(11, 20, 256, 16, 4, 128, weights))
    n = lib.moe_layer_few_tokens_workspace_size(20, 4, 256, 128, 16)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        before = int(ws[:8].view(torch.int64))
        for call in range(1, 4):
            lib.moe_layer_few_tokens(**d, workspace=ws)
            words = ws[:8 * 161].view(torch.int64)
            ctas = torch.cuda.get_device_properties(0).multi_processor_count
            assert int(words[0]) == before + call and (words[1:1 + min(ctas, 160)] == 0).all()


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("T", [1, 31])
def test_few_tokens_with_the_workspace_words_written_back(lib, T, weights):
    """A small tensor that takes the workspace's memory between two calls writes
    its first bytes (here: back to what they were) and leaves the rest."""
    a, b = (_dev(_data(s, T, 512, 40, 6, 256, weights)) for s in (12, 13))
    want = [lib.moe_layer_few_tokens(**d) for d in (a, b)]
    ws = torch.zeros(lib.moe_layer_few_tokens_workspace_size(T, 6, 512, 256, 40), dtype=torch.uint8, device=DEV)
    st = lib.new_status()
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for n in (4, 8, 64, 128):
        first = ws[:n].clone()
        for i in range(100):
            ws[:n].copy_(first)
            out = lib.moe_layer_few_tokens(**(a, b)[i % 2], workspace=ws, dev_status=st)
            differ += (out != want[i % 2]).sum()
    assert int(differ) == 0 and int(st) == 0


@pytest.mark.parametrize("weights", ["bf16", "int8"])
def test_few_tokens_in_a_graph_beside_a_small_tensor(lib, weights):
    """The same inside a graph, whose addresses repeat with every replay."""
    d = _dev(_data(14, 5, 512, 40, 6, 256, weights))
    other = _dev(_data(15, 5, 512, 40, 6, 256, weights))
    inputs = [{k: v[k].clone() for k in ("tokens", "expert_ids", "probs")} for v in (d, other)]
    want = [lib.moe_layer_few_tokens(**dict(d, **i)) for i in inputs]
    ws = torch.zeros(lib.moe_layer_few_tokens_workspace_size(5, 6, 512, 256, 40), dtype=torch.uint8, device=DEV)
    st = lib.new_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws[:8].zero_()
        out = lib._m.moe_layer_few_tokens(**d, workspace=ws, dev_status=st)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(50):
        for k, v in inputs[i % 2].items():
            d[k].copy_(v)
        graph.replay()
        differ += (out != want[i % 2]).sum()
    assert int(differ) == 0 and int(st) == 0


def test_few_tokens_over_memory_of_other_uses(lib):
    """The workspace's memory as other tensors leave it: small integers, row maps
    with minus ones, zeros under any epoch."""
    d = _dev(_data(16, 12, 512, 40, 6, 256, "bf16"))
    n = lib.moe_layer_few_tokens_workspace_size(12, 6, 512, 256, 40) // 8 * 8
    want = lib.moe_layer_few_tokens(**d)
    fills = [torch.arange(n // 8, device=DEV), torch.arange(n // 8, device=DEV) - 1,
             torch.arange(n // 4, dtype=torch.int32, device=DEV), torch.full((n // 8,), -1, device=DEV)]
    for first in (-161, -2, -1, 1, 2**62):                  # zeros after another epoch
        z = torch.zeros(n // 8, dtype=torch.int64, device=DEV)
        z[0] = first
        fills.append(z)
    z = torch.full((n // 8,), -1, device=DEV)
    z[0] = 0
    fills.append(z)
    for f in fills:
        ws = torch.cat([f.view(torch.uint8), torch.zeros(64, dtype=torch.uint8, device=DEV)])
        for _ in range(3):
            assert torch.equal(lib.moe_layer_few_tokens(**d, workspace=ws), want)


# Phase 1 over equal runs of units, a tile shared by the CTAs whose runs meet in
# it ("split"): taken when there are more tiles of 128 columns than CTAs, or few
# and long ones.  Columns of an accumulator (16, 32, 64) and, on 152 CTAs, tiles,
# shared tiles (bf16 / int8) and CTAs of a shared tile.
SPLIT = [  # T, H, E, K, I
    (16, 512, 100, 8, 320),    # 16: 219 tiles, 133 / 114 shared, 2 CTAs
    (17, 320, 100, 8, 320),    # 32: 213 tiles, 121 / 101 shared, 2 CTAs
    (32, 1088, 100, 8, 256),   # 32, all in use: 186 tiles, 142 / 134 shared, 2 CTAs
    (33, 320, 100, 8, 256),    # 64, the second half of the warps with one token: 186 tiles, 120 / 100 shared, 2 CTAs
    (64, 1088, 100, 8, 256),   # 64, all in use: 200 tiles, 136 / 128 shared, 2 CTAs
    (24, 4096, 6, 2, 128),     # 32: 6 tiles of 26 CTAs each
    (50, 4096, 6, 2, 192),     # 64, half of a tile past the end: 12 tiles of 13 or 14 CTAs each
]


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("T,H,E,K,I", SPLIT)
def test_few_tokens_with_shared_tiles(lib, T, H, E, K, I, weights):
    d = _data(T + H + E, T, H, E, K, I, weights, shared=T % 2 == 1)
    _check(lib.moe_layer_few_tokens(**_dev(d)), d)


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("T,H,E,K,I", [(31, 512, 100, 6, 320), (64, 512, 100, 8, 256)])
def test_few_tokens_with_shared_tiles_repeats_bit_for_bit(lib, T, H, E, K, I, weights):
    """A dirty workspace, the last call's own words, and first words written back."""
    d, e = (_dev(_data(s, T, H, E, K, I, weights, shared=True)) for s in (17, 18))
    want = [lib.moe_layer_few_tokens(**v) for v in (d, e)]
    n = lib.moe_layer_few_tokens_workspace_size(T, K, H, I, E)
    st = lib.new_status()
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for fill in (0, 255, 85):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        first = ws[:8].clone()
        for i in range(40):
            if i % 4 == 3:
                ws[:8].copy_(first)
            out = lib.moe_layer_few_tokens(**(d, e)[i % 2], workspace=ws, dev_status=st)
            differ += (out != want[i % 2]).sum()
    assert int(differ) == 0 and int(st) == 0


def test_few_tokens_with_shared_tiles_on_two_streams_and_in_a_graph(lib):
    a = _dev(_data(19, 20, 512, 100, 8, 320, "bf16"))
    b = _dev(_data(20, 64, 512, 100, 8, 256, "int8"))
    want = lib.moe_layer_few_tokens(**a), lib.moe_layer_few_tokens(**b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, d in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(lib._m.moe_layer_few_tokens(**d))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib._m.moe_layer_few_tokens(**b)
    c = _dev(_data(21, 64, 512, 100, 8, 256, "int8"))
    for k in ("tokens", "expert_ids", "probs"):
        b[k].copy_(c[k])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.moe_layer_few_tokens(**b))


def test_few_tokens_with_shared_tiles_keep_to_their_own_rows(lib):
    """Values of one token reach no other; ids of inactive slots change at most
    the order of the sums."""
    d = _data(22, 40, 512, 100, 8, 320, "bf16")
    clean = lib.moe_layer_few_tokens(**_dev(d)).cpu()
    d["tokens"][3], d["tokens"][39, 5] = float("nan"), float("inf")
    out = lib.moe_layer_few_tokens(**_dev(d)).cpu()
    keep = [t for t in range(40) if t not in (3, 39)]
    assert torch.isnan(out[3]).all() and torch.equal(out[keep], clean[keep])
    mask = torch.ones(40, dtype=torch.uint8)
    mask[::3] = 0
    d = _data(22, 40, 512, 100, 8, 320, "bf16")
    _check(lib.moe_layer_few_tokens(**_dev(d), active_mask=mask.to(DEV)), d, mask)


def test_few_tokens_of_long_rows(lib):
    """H and I at the limit, one expert each (the sums by torch in 64 bits)."""
    g = torch.Generator(device=DEV).manual_seed(23)
    for H, I in ((2**20, 64), (64, 2**20)):
        x, wg, wu, wd = (torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16) * s[-1] ** -0.5
                         for s in ((3, H), (1, I, H), (1, I, H), (1, H, I)))
        x *= H ** 0.5
        ids, p = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.rand(3, 1, generator=g, device=DEV)
        out = lib.moe_layer_few_tokens(x, ids, p, wg, wu, wd)
        a, b = x.double() @ wg[0].double().t(), x.double() @ wu[0].double().t()
        want = p.double() * ((torch.nn.functional.silu(a) * b) @ wd[0].double().t())
        # two roundings to bf16 (act's, the output's), 2^-9 of a value at most each, and fp32 sums
        assert float((out.double() - want).norm() / want.norm()) < 2 * 2.0 ** -9


@pytest.mark.parametrize("weights", ["bf16", "int8"])
@pytest.mark.parametrize("T", [3, 20, 64])
def test_few_tokens_saturated_gates(lib, T, weights):
    """Gates far below and above the range of e^g, each alone in a column of act
    and carried to one output.  act and out round to bf16 (2^-9 each), the
    quotient is 0 where 1 + e^-g is past 2^126: 88 u 2^-126 at most is lost."""
    H = I = 64
    gate = torch.tensor([0.0, -0.0, 1, -1, 20, -20, 60, -60, 80, -80, 86, -86, 88, -88, 90, -90, 120, -120, 1000, -1000,
                         3e4, -3e4, 127, -127] + [float(i) for i in range(-20, 20)])
    u = torch.where(torch.arange(64) % 3 == 0, -3.0, 2.0)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 1, 1
    if weights == "bf16":
        wg, wu, wd = torch.zeros(1, I, H), torch.zeros(1, I, H), torch.eye(64)[None]
        wg[0, :, 0], wu[0, :, 1] = gate, u
        w, scales = [v.bfloat16() for v in (wg, wu, wd)], None
        g64 = w[0][0, :, 0].double()
    else:
        w = [torch.zeros(1, 64, 64, dtype=torch.int8) for _ in range(3)]
        w[0][0, :, 0], w[1][0, :, 1] = 1, 1
        w[2][0] = torch.eye(64).to(torch.int8)
        scales = tuple(v[None].to(DEV) for v in (gate, u, torch.ones(64)))
        g64 = gate.double()
    out = lib.moe_layer_few_tokens(x.to(DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV),
                                   torch.ones(T, 1, device=DEV), *(v.to(DEV) for v in w),
                                   scales=scales).cpu().double()
    want = (torch.nn.functional.silu(g64) * u.double()).expand(T, -1)
    assert torch.isfinite(out).all()
    assert bool(((out - want).abs() <= want.abs() * (2 ** -8 + 2 ** -16) + 88 * 3 * 2.0 ** -126).all())
