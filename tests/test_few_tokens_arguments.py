"""Sizes that the layer for a few tokens refuses before any CUDA call."""

import os
import shutil

import pytest

LIMIT = 0x100000


@pytest.fixture(scope="module")
def lib():
    from unpermute_moe_permute_gb300 import binding, build
    if not os.path.exists(build.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        build.build()
    return binding.load_library(build.LIB_PATH)


@pytest.mark.parametrize("H,I,refused", [(LIMIT, 64, False), (64, LIMIT, False), (LIMIT + 64, 64, True),
                                         (64, LIMIT + 64, True), (2**31 - 64, 64, True)])
def test_sizes(lib, H, I, refused):
    """Past the limit a count of elements or of a tile's bytes could pass 31 bits;
    up to it the missing tokens are what is refused."""
    from unpermute_moe_permute_gb300 import binding
    assert (lib.moe_layer_few_tokens_workspace_size(64, 16, H, I, 1) == 0) == refused
    rc = lib.moe_layer_few_tokens(None, None, None, 64, H, 1, I, 1, 0, None, 0, binding.MOE_BF16, None, None, None,
                                  None, None, None, None, None, None, 0, None, None)
    assert rc == (binding.MOE_ERR_SHAPE if refused else binding.MOE_ERR_INVALID_ARG)
