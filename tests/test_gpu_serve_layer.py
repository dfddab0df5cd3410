"""The example layer: prompts in int8, decoding in one launch, a training step.

Norm of the error over the norm of the result.  bf16 paths: a handful of
independent roundings of 2^-9 / sqrt(3) rms each on the way (rows, g, u, act,
expert rows, result): under 0.01; their gradients twice as many: 0.02.  int8:
uniform rounding of 1/127 of a row's largest magnitude, 1 % of the rms on each
of four factors (two for int8 weights alone): 0.03.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serve_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _off(got, want):
    got, want = got.detach().double(), want.detach().double()
    return float((got - want).norm() / want.norm())


def _double(layer, x, logits, ids):
    """The layer in float64 on the chosen experts; logits may require a gradient."""
    chosen = torch.gather(logits, 1, ids.long())
    if layer.how["scoring"] == "softmax":
        p = torch.softmax(logits, 1).gather(1, ids.long())
    else:
        p = torch.sigmoid(chosen)
    if layer.how["renormalize"]:
        p = p / p.sum(1, keepdim=True)
    p = p * layer.how["scale"]
    i = ids.long()
    g = torch.einsum("tkih,th->tki", layer.gate.double()[i], x)
    u = torch.einsum("tkih,th->tki", layer.up.double()[i], x)
    return torch.einsum("tk,tkhi,tki->th", p, layer.down.double()[i], torch.nn.functional.silu(g) * u)


@pytest.mark.parametrize("T,H,I,E,K,scoring,renormalize,scale", [
    (1, 128, 64, 4, 2, "softmax", True, 1.0),
    (64, 256, 192, 16, 4, "sigmoid", True, 2.5),
    (33, 512, 320, 40, 8, "softmax", False, 1.0),
])
def test_paths_agree(example, T, H, I, E, K, scoring, renormalize, scale):
    layer = example.Layer(H, I, E, K, scoring, renormalize, scale, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x = torch.randn(T, H, device="cuda", generator=g, dtype=torch.bfloat16)
    ids, _, logits = layer.route(x)
    leaf_x, leaf_l = x.double().requires_grad_(True), logits.double().requires_grad_(True)
    want = _double(layer, leaf_x, leaf_l, ids)
    out, saved = layer.forward(x)
    assert _off(out, want) < 0.01
    assert _off(layer.decode(x, int8=False), want) < 0.01
    assert _off(layer.decode(x), want) < 0.03
    assert _off(layer.prompt(x), want) < 0.03
    grad = torch.randn(T, H, device="cuda", generator=g, dtype=torch.bfloat16)
    want.backward(grad.double())
    grad_x, grad_logits, _ = layer.backward(grad, saved)
    assert _off(grad_x, leaf_x.grad) < 0.02
    assert _off(grad_logits, leaf_l.grad) < 0.02
    assert int(layer.status) == 0


def test_decode_in_a_graph(example):
    """A decoding step captured once replays with new tokens."""
    layer = example.Layer(256, 128, 8, 2)
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.decode(x)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = layer.decode(x)
    for seed in range(3):
        x.copy_(torch.randn(4, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer.decode(x))


def test_command(example, capsys):
    example.main(["--tokens", "70", "--hidden", "256", "--inter", "128", "--experts", "8", "--topk", "2"])
    text = capsys.readouterr().out
    assert "prompt" in text and "decode      64" in text and "training" in text


def test_command_says_when_a_kernel_failed(example, monkeypatch):
    """The device status word ends the command with its name."""
    monkeypatch.setattr(example.lib, "moe_check_status", lambda status: example.lib.MOE_ERR_BAD_ID)
    with pytest.raises(SystemExit, match=example.lib.status_name(example.lib.MOE_ERR_BAD_ID)):
        example.main(["--tokens", "70", "--hidden", "256", "--inter", "128", "--experts", "8", "--topk", "2"])


@pytest.mark.parametrize("T", [9, 700])
def test_prompt_and_training_in_a_graph(example, T):
    """Router, rows, products and the router's gradient, whose launches overlap the
    end of the kernel before, captured once (few and many rows an expert) and
    replayed with new tokens."""
    layer = example.Layer(256, 128, 8, 2, renormalize=False)
    x, grad = (torch.zeros(T, 256, device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def step():
        out, saved = layer.forward(x)
        dx, dl, (dg, du, dd) = layer.backward(grad, saved)
        return layer.prompt(x), out, dx, dl, dg, du, dd

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, grad):
            t.copy_(torch.randn(T, 256, device="cuda", generator=g))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert int(layer.status) == 0
