"""A stack of sparse blocks: pre-norm, experts chosen in groups by sigmoid
scores with a balance bias, post-norm, residual; low-rank adapters of several
users beside the experts; then gradient steps of a router toward given mixing
weights and of the last block's adapters, norms and router (balance loss,
clipped gradients), the experts frozen.

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
from nvfp4_token_quantized_gb300 import BlockNorm, ExpertRouter, GradientClip, LowRankAdapters, MoE  # noqa: E402

SHAPE = dataclasses.replace(synthetic.CONFIGS["c0_tiny"], name="block", H=512, E=32, K=4, I=256, T=256,
                            max_num_tokens=4096, deterministic=True)


class SparseStack:
    """``layers`` blocks over a bf16 residual stream [T, H], with ``users``
    adapters beside each block's experts."""

    def __init__(self, shape, layers: int, seed: int = 0, users: int = 0, rank: int = 8):
        self.shape = shape
        self.adapters = LowRankAdapters(shape.H, shape.H, rank)
        self.clip = GradientClip(1.0)
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
        self.down, self.up = [], []
        for _ in range(layers if users else 0):
            for factors, size in ((self.down, shape.H ** -0.5), (self.up, 0.1 * rank ** -0.5)):
                factors.append((torch.randn(users, rank, shape.H, generator=g) * size).to(torch.bfloat16).cuda())

    def forward(self, x, user=None):
        """The normed rows after the last block, and what each layer saw; user:
        int32 [T], whose adapters each row takes (-1: none)."""
        trace = []
        residual = x
        _, h = self.first.forward(residual, pre_weight=self.pre[0])
        for i, layer in enumerate(self.moe):
            y, hidden = layer.forward(h, self.gate_w[i]), None
            if user is not None:
                y, hidden = self.adapters.forward(h, user, self.down[i], self.up[i], base=y, out=y, keep_hidden=True)
            trace.append({"residual": residual, "h": h, "y": y, "hidden": hidden, "logits": layer.debug_logits(),
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


    def tuning_gradients(self, step, residual_out, dh, user, balance: float = 0.01):
        """Gradients of the last block's parameters, the experts' outputs held
        fixed, from dh, the gradient of the normed rows behind it: the loss's
        balance part, the experts' counts and {name: gradient}, clipped
        together, with their norm."""
        i = len(self.moe) - 1
        _, dy, _, dpost, dpre = self.norm.backward(None, dh, residual_out, step["y"], post_weight=self.post[i],
                                                   pre_weight=self.pre[i + 1])
        _, ddown, dup = self.adapters.backward(dy, step["h"], step["hidden"], user, self.down[i], self.up[i])
        loss, counts, slope = self.router.balance_loss(step["logits"], step["topk_ids"], coefficient=balance)
        dgate = step["h"].float().t() @ self.router.balance_backward(step["logits"], slope)
        grads = {"down": ddown, "up": dup, "post": dpost, "pre": dpre, "gate": dgate}
        norm, _ = self.clip.clip(list(grads.values()))
        return loss, counts, grads, norm

    def tuning_step(self, x, user, target, lr: float):
        """Moves the last block toward normed rows ``target``; returns the
        squared error before, the balance loss and the gradients' norm."""
        h, trace = self.forward(x, user)
        i = len(self.moe) - 1
        residual_out, _ = self.norm.forward(trace[i]["residual"], trace[i]["y"], post_weight=self.post[i],
                                            pre_weight=self.pre[i + 1])
        off = h.float() - target.float()
        loss, _, grads, norm = self.tuning_gradients(trace[i], residual_out, (off * (2.0 / off.numel())).to(h.dtype), user)
        for name, p in (("down", self.down), ("up", self.up), ("post", self.post), ("gate", self.gate_w)):
            p[i] = (p[i].float() - lr * grads[name].float()).to(p[i].dtype)
        self.pre[i + 1] = (self.pre[i + 1].float() - lr * grads["pre"]).to(torch.bfloat16)
        return (off ** 2).mean(), loss, norm


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=SHAPE.T)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    stack = SparseStack(SHAPE, a.layers, users=4)
    x = synthetic.make_activations(SHAPE, T=a.tokens).cuda()
    h, trace = stack.forward(x)
    print(f"{a.layers} blocks, {a.tokens} tokens: |h| = {h.float().square().mean().sqrt().item():.4f}")
    target = torch.full_like(trace[0]["topk_w"], 2.5 / SHAPE.K)
    for n in range(3):
        loss = stack.router_step({"layer": 0, **trace[0]}, target, lr=20.0)
        print(f"router step {n}: loss {loss.item():.6f}")
        h, trace = stack.forward(x)
    user = (torch.arange(a.tokens, device="cuda") * 5 // max(1, a.tokens) - 1).int()
    for n in range(3):
        error, balance, norm = stack.tuning_step(x, user, h.roll(1, dims=1), lr=1.0)
        print(f"tuning step {n}: error {error.item():.6f}, balance {balance.item():.6f}, gradients {norm.item():.3e}")


if __name__ == "__main__":
    main()
