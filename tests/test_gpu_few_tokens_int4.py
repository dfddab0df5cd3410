"""GPU parity of the layer for a few tokens over 4-bit weights: the float64
oracle on the bf16 weights that they stand for, with the oracle's own bound of
what fp32 sums and one bf16 rounding of act allow."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import np64, ulp
from test_gpu_few_tokens import SIZES, SPLIT

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _group(n, want):
    return next(g for g in (want, 64, 32) if n % g == 0)


def _data(seed, T, H, E, K, I, group=128, special=0, shared=False, five=True):
    g = np.random.default_rng(seed)
    bf = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).bfloat16()  # noqa: E731
    d = dict(tokens=bf(T, H),
             expert_ids=torch.from_numpy(np.argsort(g.random((T, E + special)), axis=1)[:, :K].astype(np.int32)),
             probs=torch.from_numpy(g.random((T, K)).astype(np.float32)),
             shared_x=bf(T, H) if shared else None, num_special=special)
    for name, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
        gr = _group(k, group)
        d[f"W_{name}_q"] = torch.from_numpy(g.integers(0, 256, (E, n, k // 2)).astype(np.uint8))
        s = (16 + g.integers(0, 16, (E, k // gr, n))) * 2.0 ** -11 if five else g.random((E, k // gr, n)) * 1.5e-2 + 1e-4
        d[f"{name}_scale"] = torch.from_numpy(s).bfloat16()
    return d


def _dev(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _floats(d):
    return [S.weights_int4(d[f"W_{n}_q"].numpy(), np.nan_to_num(np64(d[f"{n}_scale"]), nan=0.0, posinf=0.0))
            for n in ("gate", "up", "down")]


def _check(out, d, mask=None):
    want, bound = S.layer_few_tokens(np64(d["tokens"]), d["expert_ids"].numpy(), d["probs"].numpy(), *_floats(d),
                                     d["W_gate_q"].shape[0], d["num_special"], None if mask is None else mask.numpy(),
                                     None if d["shared_x"] is None else np64(d["shared_x"]))
    got = np64(out)
    assert got.shape == want.shape and np.all(np.isfinite(got))
    lim = bound + ulp(np.maximum(np.abs(got), np.abs(want)), "bf16")
    bad = np.abs(got - want) > lim
    assert not bad.any(), (int(bad.sum()), bad.size, float((np.abs(got - want) / lim).max()))


def _ids(d):
    return d["W_gate_q"].shape[0]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,H,E,K,I", SIZES)
def test_few_tokens(lib, T, H, E, K, I, group):
    d = _data(T + H + E, T, H, E, K, I, group, shared=T % 2 == 1, five=group != 64)
    _check(lib.moe_layer_few_tokens_int4(**_dev(d)), d)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,H,E,K,I", SPLIT)
def test_with_shared_tiles(lib, T, H, E, K, I, group):
    d = _data(T + H + E, T, H, E, K, I, group, shared=T % 2 == 1)
    _check(lib.moe_layer_few_tokens_int4(**_dev(d)), d)


def test_two_groups_in_one_layer(lib):
    """Scales of 128 inputs before the activation, of 32 after it."""
    d = _data(3, 20, 512, 6, 2, 192, 128)
    assert d["gate_scale"].shape[1] == 4 and d["down_scale"].shape[1] == 3
    d["down_scale"] = torch.rand(6, 6, 512, generator=torch.Generator().manual_seed(1)).bfloat16() * 0.01
    _check(lib.moe_layer_few_tokens_int4(**_dev(d)), d)


def test_all_on_one_expert(lib):
    d = _data(1, 64, 320, 9, 2, 192)
    d["expert_ids"][:, 0], d["expert_ids"][:, 1] = 7, 3
    _check(lib.moe_layer_few_tokens_int4(**_dev(d)), d)


@pytest.mark.parametrize("dims", [1, 2])
def test_masks_and_special_ids(lib, dims):
    d = _data(2, 20, 192, 6, 4, 128, special=3, shared=True)
    g = np.random.default_rng(3)
    mask = torch.from_numpy((g.random((20,) if dims == 1 else (20, 4)) < 0.6).astype(np.uint8))
    mask[0] = 0                                                    # a token with nothing at all
    _check(lib.moe_layer_few_tokens_int4(**_dev(d), active_mask=mask.to(DEV)), d, mask)
    d["shared_x"] = None
    out = lib.moe_layer_few_tokens_int4(**_dev(d), active_mask=torch.zeros_like(mask).to(DEV))
    assert (out == 0).all()
    d["expert_ids"][:, :3] = torch.arange(6, 9, dtype=torch.int32)  # special ids, one real slot each
    d["expert_ids"][:, 3] %= 6
    _check(lib.moe_layer_few_tokens_int4(**_dev(d)), d)


def test_bad_ids_are_flagged_and_skipped(lib):
    d = _data(4, 9, 128, 8, 3, 64)
    for t, row in ((1, [2, 8, 3]), (4, [-1, 0, 1]), (6, [5, 5, 5]), (8, [2**31 - 1, -2**31, 7])):
        d["expert_ids"][t] = torch.tensor(row, dtype=torch.int32)
    st = lib.new_status()
    out = lib.moe_layer_few_tokens_int4(**_dev(d), dev_status=st)
    assert lib.moe_check_status(st) == lib.MOE_ERR_BAD_ID
    _check(out, d)


def test_keep_to_their_own_rows_and_experts(lib):
    """NaN and infinities in one token's row and in the scales of an expert that only
    one token chose do not reach the others."""
    d = _data(5, 12, 128, 10, 2, 64)
    d["expert_ids"][:] = torch.tensor([0, 1], dtype=torch.int32)
    d["expert_ids"][5] = torch.tensor([1, 9], dtype=torch.int32)   # the only token of expert 9
    d["tokens"][3, 7] = float("nan")
    d["tokens"][4, 9] = float("inf")
    d["gate_scale"][9, 0, 3], d["down_scale"][9, 0, 2] = float("nan"), float("inf")
    mask = torch.ones(12, 2, dtype=torch.uint8)
    d["tokens"][7] = float("nan")
    mask[7] = 0                                                    # a padding token
    out = lib.moe_layer_few_tokens_int4(**_dev(d), active_mask=mask.to(DEV)).cpu()
    assert torch.isnan(out[3]).any() and not torch.isfinite(out[4]).all() and not torch.isfinite(out[5]).all()
    assert (out[7] == 0).all()
    keep = [t for t in range(12) if t not in (3, 4, 5, 7)]
    clean = dict(d)
    clean.update({k: d[k][keep] for k in ("tokens", "expert_ids", "probs")})
    _check(out[keep], clean, mask[keep])


@pytest.mark.parametrize("T,H,E,K,I", [(1, 2048, 128, 8, 768), (31, 512, 100, 6, 320), (64, 512, 100, 8, 256), (5, 512, 40, 6, 256)])
def test_repeats_bit_for_bit(lib, T, H, E, K, I):
    """A dirty workspace, the last call's own words, first words written back, and
    every one of many launches compared on the device."""
    d, e = (_dev(_data(s, T, H, E, K, I, 64, shared=True)) for s in (17, 18))
    want = [lib.moe_layer_few_tokens_int4(**v) for v in (d, e)]
    n = lib.moe_layer_few_tokens_workspace_size(T, K, H, I, E)
    st = lib.new_status()
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for fill in (0, 255, 85):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        first = ws[:8].clone()
        for i in range(300):
            if i % 4 == 3:
                ws[:8].copy_(first)
            out = lib.moe_layer_few_tokens_int4(**(d, e)[i % 2], workspace=ws, dev_status=st)
            differ += (out != want[i % 2]).sum()
    assert int(differ) == 0 and int(st) == 0


def test_two_streams_and_a_graph(lib):
    a, b = _dev(_data(7, 8, 256, 16, 4, 128)), _dev(_data(8, 64, 512, 32, 8, 256, 32))
    want = lib.moe_layer_few_tokens_int4(**a), lib.moe_layer_few_tokens_int4(**b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, d in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(lib._m.moe_layer_few_tokens_int4(**d))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib._m.moe_layer_few_tokens_int4(**a)
    c = _dev(_data(9, 8, 256, 16, 4, 128))
    for k in ("tokens", "expert_ids", "probs"):
        a[k].copy_(c[k])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.moe_layer_few_tokens_int4(**a))


def test_bf16_weights_of_the_same_values_give_the_same_layer(lib):
    """Weights that 4 bits hold exactly: the two kernels multiply the same numbers and
    differ in the order of their fp32 sums, which may move act's and the output's
    rounding by a step each."""
    d = _dev(_data(10, 50, 512, 24, 6, 256, 64, shared=True))
    out = lib.moe_layer_few_tokens_int4(**d)
    w = [lib.moe_dequantize_weights_int4(d[f"W_{n}_q"], d[f"{n}_scale"]) for n in ("gate", "up", "down")]
    ref = lib.moe_layer_few_tokens(d["tokens"], d["expert_ids"], d["probs"], *w, shared_x=d["shared_x"])
    assert float((out.float() - ref.float()).norm() / ref.float().norm()) < 2.0 ** -8


def test_of_long_rows(lib):
    """H and I at the limit, one expert each (the sums by torch in 64 bits)."""
    g = torch.Generator(device=DEV).manual_seed(23)
    for H, I in ((2**20, 64), (64, 2**20)):
        x = torch.randn(3, H, generator=g, device=DEV).bfloat16()
        q = [lib.moe_quantize_weights_int4(torch.randn(1, n, k, generator=g, device=DEV) * k ** -0.5, 64)
             for n, k in ((I, H), (I, H), (H, I))]
        ids, p = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.rand(3, 1, generator=g, device=DEV)
        out = lib.moe_layer_few_tokens_int4(x, ids, p, *q[0], *q[1], *q[2])
        wg, wu, wd = (lib.moe_dequantize_weights_int4(*v)[0].double() for v in q)
        want = p.double() * ((torch.nn.functional.silu(x.double() @ wg.t()) * (x.double() @ wu.t())) @ wd.t())
        # two roundings to bf16 (act's, the output's), 2^-9 of a value at most each, and fp32 sums
        assert float((out.double() - want).norm() / want.norm()) < 2 * 2.0 ** -9
