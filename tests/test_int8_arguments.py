"""Arguments of the 8-bit products that the host refuses before any CUDA call."""

import os
import shutil

import pytest

LIMIT = 0x7f000000


@pytest.fixture(scope="module")
def lib():
    from unpermute_moe_permute_gb300 import binding, build
    if not os.path.exists(build.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        build.build()
    return binding.load_library(build.LIB_PATH)


@pytest.mark.parametrize("N,what", [(LIMIT, "MOE_ERR_INVALID_ARG"), (LIMIT + 1, "MOE_ERR_SHAPE"),
                                    (2**31 - 1, "MOE_ERR_SHAPE"), (-1, "MOE_ERR_INVALID_ARG")])
def test_rows(lib, N, what):
    """Row counts that pass 31 bits where rows and tiles are added up; up to the limit
    the missing pointers are what is refused."""
    from unpermute_moe_permute_gb300 import binding
    want = getattr(binding, what)
    assert lib.moe_gate_up_swiglu_int8(None, None, None, N, 64, 64, 1, None, None, None, None, None, None,
                                       None) == want
    assert lib.moe_down_proj_int8(None, None, None, N, 64, 64, 1, None, None, None, binding.MOE_BF16, None,
                                  None) == want
