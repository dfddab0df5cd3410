"""One MoE layer served and trained through the library's calls.

  python examples/serve_layer.py [--tokens 512] [--hidden 2048] [--inter 768]
                                 [--experts 128] [--topk 8] [--bf16]

Layer holds the weights (bf16, and the same in int8 with a scale per channel)
and runs
  prompts   router -> routing -> rows in int8 -> int8 gate/up + SwiGLU ->
            rows in int8 -> int8 down -> weighted sum of the K slots
  decoding  router -> the whole layer in one launch, for up to 64 tokens, over
            the int8 or the bf16 weights
  training  router -> bf16 layer forward and backward -> gradient of the
            router's logits
The command prints each path's time and how far the int8 paths are from bf16.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from unpermute_moe_permute_gb300 import binding as lib  # noqa: E402


class Layer:
    def __init__(self, H, I, E, K, scoring="softmax", renormalize=True, scale=1.0, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            w = torch.randn(*shape, device=device, generator=g, dtype=torch.bfloat16)
            return w * shape[-1] ** -0.5

        self.E, self.K = E, K
        self.how = dict(scoring=scoring, renormalize=renormalize, scale=scale)
        self.router = weights(E, H)
        self.gate, self.up, self.down = weights(E, I, H), weights(E, I, H), weights(E, H, I)
        # int8 with a scale per output channel: the row quantiser serves for them too
        self.int8 = []
        for w in (self.gate, self.up, self.down):
            q, s = lib.moe_quantize_rows(w.view(-1, w.shape[2]))
            self.int8.append((q.view(w.shape), s.view(w.shape[:2])))
        self.status = lib.new_status(device)

    def route(self, x):
        """The experts and weights of each token, and the logits."""
        logits = (x @ self.router.t()).float()
        ids, probs = lib.moe_router_topk(logits, self.K, dev_status=self.status, **self.how)
        return ids, probs, logits

    def prompt(self, x):
        """Any number of tokens [T, H], int8 weights."""
        ids, probs, _ = self.route(x)
        r = lib.moe_permute(None, ids, self.E, dev_status=self.status)
        (wg, gs), (wu, us), (wd, ds) = self.int8
        q, s = lib.moe_quantize_rows(x, row_map=r.row_map, K=self.K)
        act = lib.moe_gate_up_swiglu_int8(q, s, r.expert_offsets, wg, gs, wu, us,
                                          dev_status=self.status)
        q, s = lib.moe_quantize_rows(act)
        y = lib.moe_down_proj_int8(q, s, r.expert_offsets, wd, ds, dev_status=self.status)
        return lib.moe_unpermute(y, r.row_map, probs, x.shape[0], self.K)

    def decode(self, x, int8=True, workspace=None):
        """Up to MOE_FEW_TOKENS tokens [T, H]; the workspace may be kept between calls."""
        ids, probs, _ = self.route(x)
        (wg, gs), (wu, us), (wd, ds) = self.int8
        w = (wg, wu, wd) if int8 else (self.gate, self.up, self.down)
        return lib.moe_layer_few_tokens(x, ids, probs, *w, scales=(gs, us, ds) if int8 else None,
                                        workspace=workspace, dev_status=self.status)

    def forward(self, x):
        """bf16, with what the backward needs."""
        ids, probs, logits = self.route(x)
        r = lib.moe_permute(x, ids, self.E, dev_status=self.status)
        act, y, gu = lib.moe_expert_mlp(r.permuted, r.expert_offsets, self.gate, self.up, self.down,
                                        save=True, dev_status=self.status)
        out = lib.moe_unpermute(y, r.row_map, probs, x.shape[0], self.K)
        return out, (ids, probs, logits, r, act, y, gu)

    def backward(self, grad_out, saved):
        """Gradients of x (through the experts), the logits and the expert weights."""
        ids, probs, logits, r, act, y, gu = saved
        grad_y, grad_probs = lib.moe_unpermute_grad(grad_out, y, r.row_map, probs, self.K)
        d_perm, dWg, dWu, dWd = lib.moe_expert_mlp_grad(grad_y, r.permuted, act, gu, r.expert_offsets,
                                                        self.gate, self.up, self.down,
                                                        dev_status=self.status)
        grad_x = lib.moe_permute_grad(d_perm, r.row_map, grad_out.shape[0], self.K)
        grad_logits = lib.moe_router_topk_grad(grad_probs, logits, ids, dev_status=self.status,
                                               **self.how)
        return grad_x, grad_logits, (dWg, dWu, dWd)


def _time(f, n=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=768)
    p.add_argument("--experts", type=int, default=128)
    p.add_argument("--topk", type=int, default=8)
    p.add_argument("--bf16", action="store_true", help="decode over the bf16 weights")
    a = p.parse_args(argv)
    layer = Layer(a.hidden, a.inter, a.experts, a.topk)
    x = torch.randn(a.tokens, a.hidden, device="cuda", dtype=torch.bfloat16)
    want, saved = layer.forward(x)

    def off(y, ref):
        return float((y.float() - ref.float()).norm() / ref.float().norm())

    print(f"prompt   {a.tokens:5d} tokens  {_time(lambda: layer.prompt(x)):8.1f} us  "
          f"int8 off bf16 by {off(layer.prompt(x), want):.4f}")
    for t in (1, 8, 64):
        if t <= a.tokens:
            y = layer.decode(x[:t], int8=not a.bf16)
            print(f"decode   {t:5d} tokens  {_time(lambda: layer.decode(x[:t], int8=not a.bf16)):8.1f} us  "
                  f"off the bf16 layer by {off(y, want[:t]):.4f}")
    print(f"training {a.tokens:5d} tokens  "
          f"{_time(lambda: layer.backward(want, layer.forward(x)[1]), 5):8.1f} us forward and backward")
    status = lib.moe_check_status(layer.status)
    if status != lib.MOE_OK:
        raise SystemExit(lib.status_name(status))


if __name__ == "__main__":
    main()
