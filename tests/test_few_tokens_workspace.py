"""Sizes of the workspace of the layer for a few tokens: what it has to hold, and
that a workspace of a larger call serves every smaller one."""

import itertools
import os
import shutil

import pytest
import torch


@pytest.fixture(scope="module")
def size():
    from unpermute_moe_permute_gb300 import binding, build
    if not os.path.exists(build.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        build.build()
    return binding.load_library(build.LIB_PATH).moe_layer_few_tokens_workspace_size


def used(T, K, H, I, E, halves):
    """The parts, each rounded up to 256 bytes: an epoch and a flag for each of 160
    CTAs, counters, two phases' partial sums, act in one bf16 or two."""
    A = min(T * K, E)
    parts = (8 * 161, 4 * (A + A * -(-I // 128) + -(-H // 256) + 1), 160 * 2 * T * 1024, 160 * 2 * T * 1024,
             2 * halves * A * T * I)
    return sum(-(-n // 256) * 256 for n in parts)


def test_does_not_fall(size):
    for K, H, I, E in ((8, 7168, 2048, 256), (2, 4096, 14336, 8), (1, 64, 64, 1), (16, 512, 320, 1024), (8, 2048, 768, 128)):
        s = [size(T, K, H, I, E) for T in range(1, 65)]
        assert all(a <= b for a, b in zip(s, s[1:]))
        assert s == [used(T, K, H, I, E, 2) for T in range(1, 65)]
    grid = [(1, 7, 8, 9, 64), (1, 2, 16), (64, 2048, 7168), (64, 768, 14336), (1, 8, 256, 1024)]
    for a in itertools.product(*grid):
        for i, values in enumerate(grid):
            for v in values:
                if v > a[i]:
                    assert size(*a) <= size(*a[:i], v, *a[i + 1:])


# ---- on the GPU: what calls take and refuse ------------------------------------

def _call(lib, T, K, H, I, E, kind, workspace):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices.int()
    p = torch.rand(T, K, generator=g, device="cuda")
    w = [(torch.randn(*s, generator=g, device="cuda") * 0.05).bfloat16() for s in ((E, I, H), (E, I, H), (E, H, I))]
    if kind == "int4":
        q = [lib.moe_quantize_weights_int4(v, 64) for v in w]
        return lib.moe_layer_few_tokens_int4(x, ids, p, *q[0], *q[1], *q[2], workspace=workspace)
    if kind == "bf16":
        return lib.moe_layer_few_tokens(x, ids, p, *w, workspace=workspace)
    q = [lib.moe_quantize_rows(v.view(-1, v.shape[2])) for v in w]
    return lib.moe_layer_few_tokens(x, ids, p, *(a.view(v.shape) for (a, _), v in zip(q, w)),
                                    scales=[b.view(v.shape[:2]) for (_, b), v in zip(q, w)], workspace=workspace)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_one_workspace_for_every_batch(lib, kind):
    """Of the largest batch's size, used for smaller ones too."""
    K, H, I, E = 2, 256, 1024, 8
    for most in (9, 10, 64):
        ws = torch.empty(lib.moe_layer_few_tokens_workspace_size(most, K, H, I, E), dtype=torch.uint8, device="cuda")
        for T in (1, 7, 8, 9, most):
            assert torch.equal(_call(lib, T, K, H, I, E, kind, ws), _call(lib, T, K, H, I, E, kind, None))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 33, 64])
def test_calls_take_what_they_use(lib, T, kind):
    K, H, I, E = 2, 256, 1024, 8
    n = used(T, K, H, I, E, 2 if kind == "int4" else 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(_call(lib, T, K, H, I, E, kind, ws), _call(lib, T, K, H, I, E, kind, None))
    with pytest.raises(lib.MoeError) as e:
        _call(lib, T, K, H, I, E, kind, ws[:n - 16])
    assert e.value.status == lib.MOE_ERR_INVALID_ARG
