"""One mixture-of-experts block with a language-model head, trained for a few
steps on the library's calls alone:

    layer norm -> dispatch to experts -> MXFP8 quantize -> grouped GEMM ->
    combine -> linear cross entropy -> every gradient -> clipping -> update

The experts' weights are frozen in MXFP8 (their gradient GEMM with respect to
the activations runs on a second, transposed copy); the norm's parameters and
the head are trained.  Synthetic data: the target of a token is the one its
input was drawn from.

    python examples/moe_step.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_03_gb300 as bsq  # noqa: E402


class MoeBlock:
    def __init__(self, tokens=1024, cols=512, experts=8, k=2, vocab=1000, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.k, self.experts = k, experts
        self.router = randn(cols, experts).bfloat16()
        w = (randn(experts, cols, cols) * cols ** -0.5).bfloat16()
        self.w = w
        wq, _ = bsq.quantize(w.reshape(experts * cols, cols), "mxfp8_e4m3", "row")
        wt, _ = bsq.quantize(w.transpose(1, 2).reshape(experts * cols, cols).contiguous(), "mxfp8_e4m3", "row")
        self.forward_w, self.backward_w = bsq.group_views(wq, experts), bsq.group_views(wt, experts)
        self.gamma, self.beta = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
        self.head = (randn(vocab, cols) * 0.02).bfloat16()
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets[::17] = -100                       # padding tokens do not count
        self.x = (randn(vocab, cols)[self.targets.clamp(min=0)] + 0.5 * randn(tokens, cols)).bfloat16()
        # buffers that stay, so the list of gradients is built once
        self.grads = [torch.empty_like(self.head), torch.empty_like(self.gamma), torch.empty_like(self.beta)]
        self.clip = bsq.GradList(self.grads)

    def route(self, y):
        weights, ids = torch.softmax((y @ self.router).float(), 1).topk(self.k, 1)
        ids = ids.masked_fill((self.targets < 0)[:, None], -1)      # padding tokens go to no expert
        return ids, weights / weights.sum(1, keepdim=True)

    def step(self, lr=0.5, max_norm=1.0):
        """One training step; returns the mean loss and the gradient norm (device tensors)."""
        x, n = self.x, (self.targets >= 0).sum()
        y, mean, rstd = bsq.layer_norm(x, self.gamma, self.beta)
        ids, weights = self.route(y)
        rows, plan = bsq.moe_dispatch(y, ids, self.experts)
        a, _ = bsq.quantize(rows, "mxfp8_e4m3")
        expert_out = bsq.grouped_gemm(a, plan.offsets, self.forward_w, torch.bfloat16)
        h = x + bsq.moe_combine(expert_out, weights, plan)
        loss, lse = bsq.linear_cross_entropy(h, self.head, self.targets)

        dloss = (1.0 / n).float().expand(loss.shape).contiguous()
        dhead, dgamma, dbeta = self.grads
        dh = torch.empty_like(h)
        bsq.linear_cross_entropy_backward_into(h, self.head, self.targets, lse, dloss, dh, dhead)
        dexpert, _ = bsq.moe_combine_backward(dh, expert_out, weights, plan)
        d, _ = bsq.quantize(dexpert, "mxfp8_e5m2")
        drows = bsq.grouped_gemm(d, plan.offsets, self.backward_w, torch.bfloat16)
        dy = bsq.moe_dispatch_backward(drows, plan)
        bsq.layer_norm_backward_into(dy, x, self.gamma, mean, rstd, torch.empty_like(x), dgamma, dbeta)

        norm = bsq.clip_grad_norm(self.clip, max_norm)
        for p, grad in zip((self.head, self.gamma, self.beta), self.grads):
            p.sub_((lr * 20 if p is self.head else lr) * grad)
        return loss.sum() / n, norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    block = MoeBlock()
    for i in range(args.steps):
        loss, norm = block.step()
        if i % 5 == 0 or i == args.steps - 1:
            print(f"step {i:3d}  loss {float(loss):.4f}  gradient norm {float(norm):.4f}")
    bsq.sync_status()


if __name__ == "__main__":
    main()
