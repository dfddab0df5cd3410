"""Arguments of the 8-bit rows and products that are refused before any CUDA call."""

import os
import shutil

import pytest
import torch

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


def test_offsets_for_every_expert(lib):
    """The kernels read E + 1 offsets."""
    from unpermute_moe_permute_gb300 import binding as b
    q, rs = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    w, cs = torch.zeros(8, 64, 128, dtype=torch.int8), torch.zeros(8, 64)
    for n in (0, 1, 8):
        off = torch.zeros(n, dtype=torch.int32)
        with pytest.raises(ValueError, match="expert_offsets must have"):
            b.moe_gate_up_swiglu_int8(q, rs, off, w, cs, w, cs, act=torch.zeros(4, 64, dtype=torch.bfloat16))
        with pytest.raises(ValueError, match="expert_offsets must have"):
            b.moe_down_proj_int8(q, rs, off, w, cs, expanded=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA"):                    # enough of them: the next check
        b.moe_down_proj_int8(q, rs, torch.zeros(9, dtype=torch.int32), w, cs, expanded=torch.zeros(4, 64))


@pytest.mark.parametrize("H,what", [(0x40000000, "MOE_ERR_INVALID_ARG"), (0x40000010, "MOE_ERR_SHAPE"),
                                    (2**31 - 16, "MOE_ERR_SHAPE")])
def test_length_of_a_row(lib, H, what):
    """Rows whose last step would pass 31 bits; up to the limit the missing output
    is what is refused."""
    from unpermute_moe_permute_gb300 import binding
    for dtype in (binding.MOE_F32, binding.MOE_BF16):
        assert lib.moe_quantize_rows(0x10000, dtype, None, 1, H, 1, 1, None, None, None) == getattr(binding, what)
