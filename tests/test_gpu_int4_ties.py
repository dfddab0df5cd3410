"""Weights to 4 bits: every bf16 value of a group's upper six binades under every
bf16 significand of its largest, quotients that lie on a tie among them."""

import numpy as np
import pytest
import torch

from test_gpu_int4 import _same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -9, 2.0 ** 90, 2.0 ** -120])
def test_every_value_under_every_largest(lib, scale):
    m = np.arange(128, 256, dtype=np.float64)
    values = np.concatenate([m * 2.0 ** -i for i in range(6)])
    values = np.concatenate([values, -values])
    rows = []
    for top in m:
        r = np.clip(values, -top, top)                      # (a few of the first binade are the largest's own)
        r = np.concatenate([r, np.zeros(-len(r) % 62)]).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(r), 1), top), r], axis=1).reshape(-1))
        assert np.isin(values[np.abs(values) <= top], rows[-1]).all()
    w = torch.from_numpy(np.stack(rows))[None] * scale
    assert w.shape[2] % 64 == 0 and torch.equal(w.bfloat16().double(), w)
    _same(lib, w.bfloat16(), 32)
    _same(lib, w.float(), 32)
