"""A stack of sparse blocks: pre-norm, experts chosen in groups by sigmoid
scores with a balance bias, post-norm, residual; then one gradient step of the
routers and norms toward given mixing weights, the experts frozen.

    python examples/sparse_block.py [--tokens 256] [--layers 2]

Run it from the repository root after building the library; it needs the GPU.
"""

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import synthetic  # noqa: E402
from nvfp4_token_quantized_gb300 import BlockNorm, ExpertRouter, MoE  # noqa: E402

SHAPE = dataclasses.replace(synthetic.CONFIGS["c0_tiny"], name="block", H=512, E=32, K=4, I=256, T=256,
                            max_num_tokens=4096, deterministic=True)


class SparseStack:
    """``layers`` blocks over a bf16 residual stream [T, H]."""

    def __init__(self, shape, layers: int, seed: int = 0):
        self.shape = shape
        self.router = ExpertRouter(shape.E, shape.K, score="sigmoid", num_groups=4, top_groups=2, group_score="top2",
                                   scale=2.5)
        self.norm = BlockNorm(shape.H, eps=1e-6)
        self.first = BlockNorm(shape.H, eps=1e-6, post=False)
        self.moe, self.gate_w, self.bias = [], [], []
        g = torch.Generator().manual_seed(seed)
        for i in range(layers):
            layer = MoE.from_shape(shape)
            w13, w2 = synthetic.make_weights(shape, seed=seed + i)
            layer.load_weights(w13.cuda(), w2.cuda())
            self.moe.append(layer)
            self.gate_w.append(synthetic.make_router(shape, seed=seed + i).cuda())
            self.bias.append((torch.randn(shape.E, generator=g) * 50).round().div(1000).cuda())
            layer.set_routing(self.router, self.bias[-1])
        # one pre-norm a layer and the one after the last, one post-norm a layer
        self.pre = [torch.ones(shape.H, dtype=torch.bfloat16, device="cuda") for _ in range(layers + 1)]
        self.post = [torch.full((shape.H,), 0.5, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]

    def forward(self, x):
        """The normed rows after the last block, and what each layer saw."""
        trace = []
        residual = x
        _, h = self.first.forward(residual, pre_weight=self.pre[0])
        for i, layer in enumerate(self.moe):
            y = layer.forward(h, self.gate_w[i])
            trace.append({"residual": residual, "h": h, "y": y, "logits": layer.debug_logits(),
                          **layer.debug_routing()})
            residual, h = self.norm.forward(residual, y, post_weight=self.post[i], pre_weight=self.pre[i + 1])
        return h, trace

    def router_step(self, step, target, lr: float):
        """Moves one layer's router and pre-norm toward the mixing weights
        ``target`` [T, K] of its chosen experts; returns the loss before."""
        i = step["layer"]
        w = step["topk_w"]
        dlogits = self.router.select_backward(step["logits"], step["topk_ids"], w, (w - target) / w.numel())
        dgate = step["h"].float().t() @ dlogits
        dh = (dlogits @ self.gate_w[i].float().t()).to(step["h"].dtype)
        _, _, _, _, dpre = self.first.backward(None, dh, step["residual"], pre_weight=self.pre[i])
        self.gate_w[i] = (self.gate_w[i].float() - lr * dgate).to(torch.bfloat16)
        self.pre[i] = (self.pre[i].float() - lr * dpre).to(torch.bfloat16)
        return 0.5 * ((w - target) ** 2).mean()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=SHAPE.T)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    stack = SparseStack(SHAPE, a.layers)
    x = synthetic.make_activations(SHAPE, T=a.tokens).cuda()
    h, trace = stack.forward(x)
    print(f"{a.layers} blocks, {a.tokens} tokens: |h| = {h.float().square().mean().sqrt().item():.4f}")
    target = torch.full_like(trace[0]["topk_w"], 2.5 / SHAPE.K)
    for n in range(3):
        loss = stack.router_step({"layer": 0, **trace[0]}, target, lr=20.0)
        print(f"router step {n}: loss {loss.item():.6f}")
        h, trace = stack.forward(x)


if __name__ == "__main__":
    main()
