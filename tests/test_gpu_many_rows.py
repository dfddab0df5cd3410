"""As many rows as 31 bits count: the last blocks' rows, and a grid that is
computed without passing 31 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = 2**31 - 1


@pytest.fixture
def room():
    """Memory for the largest case, given back afterwards."""
    if torch.cuda.mem_get_info()[0] < 130 * 2**30:
        pytest.skip("needs 130 GiB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_router_of_all_rows(lib, room):
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device=DEV)
    logits[-3:] = float("-inf")
    ids, probs = lib.moe_router_topk(logits, 1, scale=2.5)
    assert bool((probs[:-3] == 2.5).all()) and bool((probs[-3:] == 0).all())
    assert int(ids.view(-1).view(torch.uint8).max()) == 0
    grad = torch.full_like(logits, 7.0)
    lib.moe_router_topk_grad(probs, logits, ids, scoring="sigmoid", renormalize=False, grad_logits=grad)
    # g p (1 - p) = 2.5 / 4, exact in bf16
    assert bool((grad[:-3] == 0.625).all()) and bool((grad[-3:] == 0).all())


def test_quantize_all_rows(lib, room):
    x = torch.zeros(T, 16, dtype=torch.bfloat16, device=DEV)
    x[0, 3], x[-1, 5], x[-9, 15] = 127.0, -254.0, 63.5
    q, s = lib.moe_quantize_rows(x)
    for row, (h, v, scale) in {0: (3, 127, 1.0), T - 1: (5, -127, 2.0), T - 9: (15, 127, 0.5)}.items():
        want = torch.zeros(16, dtype=torch.int8)
        want[h] = v
        assert torch.equal(q[row].cpu(), want) and float(s[row]) == scale
    assert int(torch.count_nonzero(s)) == 3 and bool((q[2**30:T - 9] == 0).all())
