"""Tensors of a device that is not the current one are refused before a launch.
(One GPU is enough: what the current device is, is the host's word.)"""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_refused(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from unpermute_moe_permute_gb300 import binding as b
    if b._get_device is None:
        pytest.skip("torch does not tell the current device")
    dev, bf16 = "cuda", torch.bfloat16
    W = torch.randn(2, 64, 128, device=dev)
    q, s = b.moe_quantize_weights_int4(W, 64)
    x, off = torch.randn(4, 128, device=dev, dtype=bf16), torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    l = torch.randn(4, 8, device=dev)
    ids, p = b.moe_router_topk_grouped(l, 2, num_groups=2, top_groups=1)
    q2, s2 = b.moe_quantize_weights_int4(torch.randn(2, 128, 64, device=dev), 64)
    torch.cuda.synchronize()
    before = b.load_library().moe_kernel_launches()
    monkeypatch.setattr(b, "_get_device", lambda: 1)
    for call in (lambda: b.moe_quantize_weights_int4(W, 64), lambda: b.moe_dequantize_weights_int4(q, s),
                 lambda: b.moe_gate_up_swiglu_int4(x, off, q, s, q, s), lambda: b.moe_down_proj_int4(x, off, q, s),
                 lambda: b.moe_router_topk_grouped(l, 2, num_groups=2, top_groups=1),
                 lambda: b.moe_layer_few_tokens_int4(x, ids % 2, p, q, s, q, s, q2, s2)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()
    assert b.load_library().moe_kernel_launches() == before
