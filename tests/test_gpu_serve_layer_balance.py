"""The example's training step moves the biases of a grouped router, and its command
serves with biases that have moved."""

import pytest
import torch

from test_gpu_serve_layer import _off, example  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def test_a_training_step(example):  # noqa: F811
    layer = example.Layer(128, 64, 16, 2, "sigmoid", True, seed=3, groups=(4, 2, 2))
    x = torch.randn(64, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    out, saved = layer.forward(x)
    n = saved[3].tokens_per_expert.clone()
    want = layer.backward(2 * out, saved)
    got_out, got = layer.train(x, lambda o: 2 * o)
    assert torch.equal(got_out, out)
    for a, b in zip([*got[:2], *got[2]], [*want[:2], *want[2]]):
        assert torch.equal(a, b)
    assert torch.equal(torch.sign(layer.bias), torch.sign(8.0 - n.float()))
    plain = example.Layer(128, 64, 16, 2)
    plain.train(x, lambda o: o)
    assert plain.bias is None and int(layer.status) == int(plain.status) == 0


def test_the_command_balances(example, monkeypatch, capsys):  # noqa: F811
    seen = []
    prompt = example.Layer.prompt
    monkeypatch.setattr(example.Layer, "prompt",
                        lambda self, x, **k: (seen.append(None if self.bias is None else self.bias.clone()),
                                              prompt(self, x, **k))[1])
    sizes = ["--tokens", "70", "--hidden", "256", "--inter", "128", "--experts", "16", "--topk", "2"]
    example.main(sizes + ["--int4", "--groups", "4", "--top-groups", "2"])
    assert all(bool((b != 0).any()) for b in seen)
    assert "with the biases" in capsys.readouterr().out
    seen.clear()
    example.main(sizes)
    assert all(b is None for b in seen) and "with the biases" not in capsys.readouterr().out
