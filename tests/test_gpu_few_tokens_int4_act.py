"""The activations between the two products of the layer over 4-bit weights keep 16
significant bits, for any number of tokens.

Neighbouring channels share their gate weights and differ by one step of one up
weight, and the down product subtracts them: the output is a 2^-6th of what is
summed, so that act rounded to bf16 shows (8 bits of each term) where the output's
own rounding would hide it.  Tokens are small integers and scales powers of two, so
the first products' sums are exact in fp32 and only act's rounding, the exponential
and the second product's sums are in the bound.
"""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from gpu_util import np64, ulp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _data(seed, T, H, E, K, I, group):
    g = np.random.default_rng(seed)
    x = g.integers(-2, 3, (T, H)).astype(np.float32)
    x[:, 0] = np.where(x[:, 0] < 0, -2, 2)
    ids = np.argsort(g.random((T, E)), axis=1)[:, :K].astype(np.int32)
    step = 2.0 ** -np.round(np.log2(np.sqrt(H)) + 1.5)        # gate and up sums of a size of 2 to 3
    gate = np.repeat(g.integers(-8, 8, (E, I // 2, H)), 2, axis=1)
    up = np.repeat(g.integers(-8, 7, (E, I // 2, H)), 2, axis=1)
    up[:, 1::2, 0] += 1
    down = np.repeat(g.integers(-7, 8, (E, H, I // 2)), 2, axis=2)
    down[:, :, 1::2] *= -1
    # a scale each for 2 neighbouring channels, and for the groups of inputs
    s = lambda n: np.repeat(step * 2.0 ** -g.integers(0, 2, (E, H // group, n // 2)), 2, axis=2)  # noqa: E731
    ds = 2.0 ** -g.integers(4, 6, (E, I // _down(I, group), H)).astype(np.float64)
    gs = s(I)
    return dict(tokens=torch.from_numpy(x).bfloat16(), expert_ids=torch.from_numpy(ids),
                probs=torch.from_numpy(g.random((T, K)).astype(np.float32)),
                W_gate_q=torch.from_numpy(S.pack_int4(gate)), gate_scale=torch.from_numpy(gs).bfloat16(),
                W_up_q=torch.from_numpy(S.pack_int4(up)), up_scale=torch.from_numpy(s(I)).bfloat16(),
                W_down_q=torch.from_numpy(S.pack_int4(down)), down_scale=torch.from_numpy(ds).bfloat16())


def _down(I, group):
    return next(g for g in (group, 64, 32) if I % g == 0)


def _want(d, **how):
    W = [S.weights_int4(d[f"W_{n}_q"].numpy(), np64(d[f"{n}_scale"])) for n in ("gate", "up", "down")]
    return S.layer_few_tokens(np64(d["tokens"]), d["expert_ids"].numpy(), d["probs"].numpy(), *W,
                              d["W_gate_q"].shape[0], exact_sums=True, **how)


# Whole tiles (64 columns, 128) and tiles that CTAs share, in each of the three
# forms for 16, 32 and 64 tokens.
CASES = [(1, 2048, 16, 8, 768, 128), (3, 256, 8, 2, 192, 32), (8, 64, 32, 8, 128, 64), (8, 512, 64, 8, 512, 128),
         (5, 512, 100, 8, 640, 32), (9, 512, 40, 6, 256, 64), (16, 512, 100, 8, 320, 128), (16, 64, 8, 2, 64, 32),
         (17, 320, 64, 6, 64, 64), (24, 512, 100, 8, 320, 32), (32, 64, 16, 4, 64, 64), (33, 320, 100, 8, 256, 32),
         (45, 512, 64, 8, 256, 128), (64, 512, 100, 8, 256, 64), (64, 64, 200, 16, 64, 32)]


@pytest.mark.parametrize("T,H,E,K,I,group", CASES)
def test_act_keeps_16_bits(lib, T, H, E, K, I, group):
    d = _data(T + I, T, H, E, K, I, group)
    want, bound = _want(d, act_rounding=2.0 ** -16)
    out = np64(lib.moe_layer_few_tokens_int4(**{k: v.to(DEV) for k, v in d.items()}))
    lim = bound + ulp(np.maximum(np.abs(out), np.abs(want)), "bf16")
    assert np.all(np.abs(out - want) <= lim), float((np.abs(out - want) / lim).max())


def test_a_tokens_result_with_more_tokens_beside_it(lib):
    """The same tokens alone, and as the first of 8, 9, 17, 33 and 64: the sums may
    change their order, which is within twice the bound of one."""
    T, H, E, K, I = 64, 512, 40, 6, 256
    d = _data(2, T, H, E, K, I, 64)
    want, bound = _want(d, act_rounding=2.0 ** -16)
    dev = {k: v.to(DEV) for k, v in d.items()}
    outs = []
    for t in (1, 8, 9, 17, 33, 64):
        part = dict(dev, **{k: dev[k][:t].contiguous() for k in ("tokens", "expert_ids", "probs")})
        outs.append(np64(lib.moe_layer_few_tokens_int4(**part)))
    for o in outs:
        n = len(o)
        lim = 2 * bound[:n] + ulp(np.maximum(np.abs(o), np.abs(want[:n])), "bf16")
        assert np.all(np.abs(o - outs[-1][:n]) <= lim)
