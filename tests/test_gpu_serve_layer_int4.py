"""The example layer with 4-bit weights and a grouped router: prompts, decoding, a
training step with its biases.

Norm of the error over the norm of the result, against float64 on the weights
that the 4 bits stand for: act, the experts' rows, the result and (decoding) the
same again, a handful of roundings of 2^-9 / sqrt(3) rms each: under 0.01.
"""

import pytest
import torch

from test_gpu_serve_layer import _double, _off, example  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

CASES = [(1, 128, 64, 8, 2, 32, (4, 2, 2)), (64, 256, 192, 16, 4, 64, (4, 3, 1)), (33, 512, 256, 40, 8, 128, (8, 4, 2)),
         (500, 256, 128, 24, 6, 64, None)]


def _weights(example, layer):  # noqa: F811
    """The layer on its 4-bit weights, for the float64 form."""
    class Of:
        pass
    of = Of()
    of.how = layer.how
    of.gate, of.up, of.down = (example.lib.moe_dequantize_weights_int4(q, s) for q, s in layer.int4)
    return of


@pytest.mark.parametrize("T,H,I,E,K,group,groups", CASES)
def test_paths_agree(example, T, H, I, E, K, group, groups):  # noqa: F811
    layer = example.Layer(H, I, E, K, "sigmoid", True, 2.5, seed=T, int4_group=group, groups=groups)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x = torch.randn(T, H, device="cuda", generator=g, dtype=torch.bfloat16)
    if groups:
        layer.bias += torch.randn(E, device="cuda", generator=g) * 0.1
    ids, _, logits = layer.route(x)
    want = _double(_weights(example, layer), x.double(), logits.double(), ids)
    assert _off(layer.prompt(x, int4=True), want) < 0.01
    for t in range(0, T, 64):
        assert _off(layer.decode(x[t:t + 64], int4=True), want[t:t + 64]) < 0.01
    # the training path routes alike; its gradient of the logits knows nothing of the bias
    leaf = logits.double().requires_grad_(True)
    out, saved = layer.forward(x)
    grad = torch.randn(T, H, device="cuda", generator=g, dtype=torch.bfloat16)
    _double(layer, x.double(), leaf, ids).backward(grad.double())
    _, grad_logits, _ = layer.backward(grad, saved)
    assert _off(grad_logits, leaf.grad) < 0.02
    assert int(layer.status) == 0


def test_biases_move_towards_the_mean(example):  # noqa: F811
    layer = example.Layer(128, 64, 16, 2, "sigmoid", True, groups=(4, 2, 2))
    x = torch.randn(64, 128, device="cuda").bfloat16()
    _, saved = layer.forward(x)
    n = saved[3].tokens_per_expert
    assert int(n.sum()) == 128
    layer.balance(n, 0.5)
    mean = 8.0
    assert (layer.bias[n > mean] == -0.5).all() and (layer.bias[n < mean] == 0.5).all() and (layer.bias[n == mean] == 0).all()


def test_decoding_in_a_graph(example):  # noqa: F811
    """Routing by groups and the 4-bit layer captured once, its workspace made inside,
    replayed with new tokens and biases; another graph with a workspace of its own
    runs in between."""
    layer = example.Layer(256, 128, 16, 2, "sigmoid", True, int4_group=64, groups=(4, 2, 2))
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.decode(x, int4=True)
    s.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            outs.append(layer.decode(x, int4=True))
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(4, 256, device="cuda", generator=g))
        layer.bias.copy_(torch.randn(16, device="cuda", generator=g) * 0.1)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = layer.decode(x, int4=True)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert int(layer.status) == 0


def test_command(example, capsys):  # noqa: F811
    example.main(["--tokens", "70", "--hidden", "256", "--inter", "128", "--experts", "16", "--topk", "2", "--int4",
                  "--groups", "4", "--top-groups", "2"])
    text = capsys.readouterr().out
    assert "4-bit off bf16" in text and "decode      64" in text and "training" in text
