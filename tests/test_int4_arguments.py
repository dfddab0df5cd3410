"""4-bit weights without a GPU: the oracle's format, and calls that are refused on the host."""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from test_abi_exports import built_lib  # noqa: F401  (fixture)

P, U = 0x10000, 0x10008
F32, BF16 = 0, 1
INV, SHAPE = 1, 2
ROWS = 0x7f000000


def test_format_by_hand():
    q = np.array([[1, 2, 3, 4, -1, -2, -3, -8]])
    # bytes: inputs (0, 2), (4, 6), (1, 3), (5, 7)
    assert S.pack_int4(q).tolist() == [[0x31, 0xdf, 0x42, 0x8e]]
    assert S.unpack_int4(S.pack_int4(q)).tolist() == q.tolist()
    w = S.weights_int4(S.pack_int4(np.tile(q, 8))[None], np.array([[[0.5], [2.0]]]))
    assert w[0, 0, :8].tolist() == [0.5, 1, 1.5, 2, -0.5, -1, -1.5, -4] and w[0, 0, 63] == -16


def test_quantize_by_hand():
    w = np.zeros((1, 3, 64), dtype=np.float32)
    w[0, 0, :5] = [7.0, 3.5, -2.5, 1.5, -7.0]
    w[0, 1, 32] = 33 * 7            # / 7 = 33: a tie between 32 and 34
    w[0, 1, 40] = 32 * 2.5          # a tie between 2 and 3
    w[0, 2, 0] = np.inf
    q, s = S.quantize_weights_int4(w, 32)
    assert s[0, 0].tolist()[:2] == [1.0, 0.0] and np.isnan(s[0, 0, 2]) and s[0, 1].tolist() == [0.0, 32.0, 0.0]
    assert q[0, 0, :5].tolist() == [7, 4, -2, 2, -7] and q[0, 1, 32] == 7 and q[0, 1, 40] == 2
    assert not q[0, 2].any()


def test_quantize_is_within_half_a_step():
    g = np.random.default_rng(0)
    w = g.standard_normal((2, 30, 256)).astype(np.float32)
    q, s = S.quantize_weights_int4(w, 64)
    assert q.min() >= -7 and q.max() == 7
    back = S.weights_int4(S.pack_int4(q), s)
    step = np.repeat(np.swapaxes(s, 1, 2), 64, axis=2)
    assert np.array_equal(back, q * step.astype(np.float64))       # exact in bf16
    assert np.all(np.abs(back - w) <= 0.5 * step * (1 + 1e-6))


CHECKS = [
    # W, dtype, E, rows, cols, group, W_q, scale, stream
    ("moe_quantize_weights_int4", (P, 2, 1, 64, 128, 64, P, P, None), INV),
    ("moe_quantize_weights_int4", (P, F32, -1, 64, 128, 64, P, P, None), INV),
    ("moe_quantize_weights_int4", (P, F32, 1, 64, 0, 64, P, P, None), INV),
    ("moe_quantize_weights_int4", (P, F32, 1, 64, 128, 16, P, P, None), INV),
    ("moe_quantize_weights_int4", (P, F32, 1, 64, 192, 128, P, P, None), SHAPE),
    ("moe_quantize_weights_int4", (P, F32, 1, 64, 96, 32, P, P, None), SHAPE),
    ("moe_quantize_weights_int4", (P, F32, 65536, 64, 128, 32, P, P, None), SHAPE),
    ("moe_quantize_weights_int4", (P, F32, 1, 0x100001, 128, 32, P, P, None), SHAPE),
    ("moe_quantize_weights_int4", (P, F32, 1, 64, 0x100040, 32, P, P, None), SHAPE),
    ("moe_quantize_weights_int4", (U, BF16, 1, 64, 128, 32, P, P, None), INV),
    ("moe_quantize_weights_int4", (P, BF16, 1, 64, 128, 32, None, P, None), INV),
    ("moe_quantize_weights_int4", (P, BF16, 1, 64, 128, 32, P, U, None), INV),
    ("moe_dequantize_weights_int4", (P, P, 1, 64, 128, 48, P, None), INV),
    ("moe_dequantize_weights_int4", (P, P, 1, 64, 160, 32, P, None), SHAPE),
    ("moe_dequantize_weights_int4", (P, P, 1, 64, 128, 32, U, None), INV),
    # permuted, offsets, N, H, I, E, group, Wg, gs, Wu, us, act, status, stream
    ("moe_gate_up_swiglu_int4", (P, P, -1, 128, 64, 2, 64, P, P, P, P, P, None, None), INV),
    ("moe_gate_up_swiglu_int4", (P, None, 4, 128, 64, 2, 64, P, P, P, P, P, None, None), INV),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 128, 64, 2, 16, P, P, P, P, P, None, None), INV),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 192, 64, 2, 128, P, P, P, P, P, None, None), SHAPE),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 96, 64, 2, 32, P, P, P, P, P, None, None), SHAPE),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 128, 80, 2, 32, P, P, P, P, P, None, None), SHAPE),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 128, 64, 1025, 32, P, P, P, P, P, None, None), SHAPE),
    ("moe_gate_up_swiglu_int4", (P, P, ROWS + 1, 128, 64, 2, 32, P, P, P, P, P, None, None), SHAPE),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 128, 64, 2, 32, P, U, P, P, P, None, None), INV),
    ("moe_gate_up_swiglu_int4", (P, P, 4, 128, 64, 2, 32, P, P, None, P, P, None, None), INV),
    ("moe_gate_up_swiglu_int4", (U, P, 4, 128, 64, 2, 32, P, P, P, P, P, None, None), INV),
    # act, offsets, N, H, I, E, group, Wd, ds, expanded, out_dtype, status, stream
    ("moe_down_proj_int4", (P, P, 4, 64, 192, 2, 128, P, P, P, BF16, None, None), SHAPE),
    ("moe_down_proj_int4", (P, P, 4, 64, 0x100040, 2, 32, P, P, P, BF16, None, None), SHAPE),
    ("moe_down_proj_int4", (P, P, 4, 64, 128, 2, 32, P, P, P, 2, None, None), INV),
    ("moe_down_proj_int4", (P, P, 4, 64, 128, 2, 32, P, P, U, F32, None, None), INV),
    ("moe_down_proj_int4", (P, P, 4, 64, 128, 0, 32, P, P, P, F32, None, None), INV),
    ("moe_down_proj_int4", (None, P, 4, 64, 128, 2, 32, P, P, P, F32, None, None), INV),
]


@pytest.mark.parametrize("name,args,status", CHECKS, ids=[f"{c[0]}-{i}" for i, c in enumerate(CHECKS)])
def test_refused_on_the_host(built_lib, name, args, status):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    assert getattr(binding.load_library(built_lib), name)(*args) == status


def test_nothing_to_do_is_ok(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    lib = binding.load_library(built_lib)
    assert lib.moe_quantize_weights_int4(None, F32, 0, 64, 128, 32, None, None, None) == 0
    assert lib.moe_dequantize_weights_int4(None, None, 1, 0, 128, 32, None, None) == 0
    assert lib.moe_gate_up_swiglu_int4(None, None, 0, 128, 64, 1, 32, None, None, None, None, None, None, None) == 0
    assert lib.moe_down_proj_int4(None, None, 0, 128, 64, 1, 32, None, None, None, BF16, None, None) == 0


def test_binding_refuses_wrong_tensors(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding as b
    bf16 = torch.bfloat16
    x = torch.zeros(4, 128, dtype=bf16)
    w, s = torch.zeros(8, 64, 64, dtype=torch.uint8), torch.zeros(8, 4, 64, dtype=bf16)
    off = torch.zeros(9, dtype=torch.int32)
    act = torch.zeros(4, 64, dtype=bf16)
    with pytest.raises(ValueError, match="CUDA"):
        b.moe_gate_up_swiglu_int4(x, off, w, s, w, s, act=act)
    with pytest.raises(ValueError, match="gate_scale must have"):
        b.moe_gate_up_swiglu_int4(x, off, w, s[:, :3], w, s[:, :3], act=act)
    with pytest.raises(ValueError, match="W_up_q must have shape"):
        b.moe_gate_up_swiglu_int4(x, off, w, s, w[:, :32], s, act=act)
    with pytest.raises(ValueError, match="up_scale must be"):
        b.moe_gate_up_swiglu_int4(x, off, w, s, w, s.float(), act=act)
    with pytest.raises(ValueError, match="permuted must be"):
        b.moe_gate_up_swiglu_int4(x.float(), off, w, s, w, s, act=act)
    for n in (0, 8):
        with pytest.raises(ValueError, match="expert_offsets must have"):
            b.moe_down_proj_int4(x, off[:n], w, s, expanded=act)
    with pytest.raises(ValueError, match="down_scale must have shape"):
        b.moe_down_proj_int4(x, off, w, s[:, :, :32], expanded=act)
    with pytest.raises(ValueError, match="expanded must have shape"):
        b.moe_down_proj_int4(x, off, w, s, expanded=act[:, :32])
    with pytest.raises(ValueError, match="group must be"):
        b.moe_quantize_weights_int4(torch.zeros(4, 128), 48)
    with pytest.raises(ValueError, match="multiple of 64"):
        b.moe_quantize_weights_int4(torch.zeros(4, 160), 32)
    with pytest.raises(ValueError, match="two or three"):
        b.moe_quantize_weights_int4(torch.zeros(128), 32)
    with pytest.raises(ValueError, match="scale must have"):
        b.moe_dequantize_weights_int4(w, s[:, :3])
    with pytest.raises(ValueError, match="scale must be"):
        b.moe_dequantize_weights_int4(w, s.float())


FEW = [
    # tokens, ids, probs, T, H, K, I, E, specials, mask, mask_dims, group, down_group, Wg, gs, Wu, us, Wd, ds, shared,
    # out, workspace, bytes, status, stream
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 16, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 0, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 192, 2, 64, 8, 0, None, 0, 128, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 128, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 65, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 4, 96, 2, 64, 8, 0, None, 0, 32, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 4, 0x100040, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 4, 128, 17, 64, 64, 0, None, 0, 64, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), SHAPE),
    ((P, P, P, 4, 128, 2, 64, 8, 0, P, 3, 64, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, None, P, P, P, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, U, P, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, U, P, None, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, P, P, U, P, P, 1 << 30, None, None), INV),
    ((P, P, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, P, P, None, P, P, 100, None, None), INV),
    ((P, None, P, 4, 128, 2, 64, 8, 0, None, 0, 64, 64, P, P, P, P, P, P, None, P, P, 1 << 30, None, None), INV),
]


@pytest.mark.parametrize("args,status", FEW)
def test_few_tokens_refused_on_the_host(built_lib, args, status):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding
    assert binding.load_library(built_lib).moe_layer_few_tokens_int4(*args) == status


def test_few_tokens_binding_refuses_wrong_tensors(built_lib):  # noqa: F811
    from unpermute_moe_permute_gb300 import binding as b
    bf16, u8 = torch.bfloat16, torch.uint8
    x, ids, p = torch.zeros(3, 128, dtype=bf16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    w1, s1 = torch.zeros(4, 64, 64, dtype=u8), torch.zeros(4, 2, 64, dtype=bf16)
    w2, s2 = torch.zeros(4, 128, 32, dtype=u8), torch.zeros(4, 2, 128, dtype=bf16)
    ws = torch.zeros(1 << 20, dtype=u8)
    call = lambda *a, **k: b.moe_layer_few_tokens_int4(*a, out=x, workspace=ws, **k)  # noqa: E731
    for args, what in (((x, ids, p, w1, s1, w1, s1, w2, s2), "CUDA"),
                       ((x.float(), ids, p, w1, s1, w1, s1, w2, s2), "tokens must be"),
                       ((x, ids.long(), p, w1, s1, w1, s1, w2, s2), "expert_ids must be"),
                       ((x, ids, p[:2], w1, s1, w1, s1, w2, s2), "probs must have shape"),
                       ((x, ids, p, w1, s1, w1, s1[:, :1], w2, s2), "up_scale must have shape"),
                       ((x, ids, p, w1, s1[:, :0], w1, s1, w2, s2), "gate_scale must have"),
                       ((x, ids, p, w1, s1, w1, s1, w2[:, :64], s2), "W_down_q must have shape"),
                       ((x, ids, p, w1, s1, w1, s1, w2, s2.float()), "down_scale must be")):
        with pytest.raises(ValueError, match=what):
            call(*args)
    with pytest.raises(ValueError, match="shared_x must have shape"):
        call(x, ids, p, w1, s1, w1, s1, w2, s2, shared_x=x[:2])
