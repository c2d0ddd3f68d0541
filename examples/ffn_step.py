"""One dense feed-forward block with a language-model head, trained for a few
steps on the library's calls alone:

    layer norm -> gated projections -> down projection, added to the residual ->
    linear cross entropy -> every gradient -> their norm -> AdamW, which clips

Weights are BF16, their moments in 8 bits, both rounded stochastically; the
norm's parameters are FP32.  With --mxfp8 the forward products run on MXFP8
operands, quantized at every step.  Synthetic data: the target of a token is the
one its input was drawn from.

    python examples/ffn_step.py [--steps N] [--mxfp8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_03_gb300 as bsq  # noqa: E402


class FeedForward:
    def __init__(self, tokens=1024, cols=512, width=1408, vocab=1000, mxfp8=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.mxfp8, self.t = mxfp8, 0
        self.w_gate, self.w_up = ((randn(width, cols) * cols ** -0.5).bfloat16() for _ in range(2))
        self.w_down = (randn(cols, width) * width ** -0.5).bfloat16()
        self.b_down = torch.zeros(cols, device="cuda")
        self.gamma, self.beta = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
        self.head = (randn(vocab, cols) * 0.02).bfloat16()
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets[::17] = -100                       # padding tokens do not count
        self.x = (randn(vocab, cols)[self.targets.clamp(min=0)] + 0.5 * randn(tokens, cols)).bfloat16()
        # buffers that stay, so the lists are built once
        matrices, vectors = [self.w_gate, self.w_up, self.w_down, self.head], [self.b_down, self.gamma, self.beta]
        self.params = matrices + vectors
        self.grads = [torch.empty_like(p) for p in self.params]
        self.norms = bsq.GradList(self.grads)
        self.adam = bsq.AdamWList(self.params, self.grads, bsq.adamw_states(matrices, 8) + bsq.adamw_states(vectors, 32))

    def forward(self, y):
        """(h, gate, up, the block's output) of the normed input"""
        h, gate, up = (torch.empty((y.shape[0], self.w_gate.shape[0]), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        if not self.mxfp8:
            bsq.gated_linear_into(y, self.w_gate, self.w_up, h, "silu", gate, up)
            return h, gate, up, bsq.linear(h, self.w_down, self.b_down, self.x)

        def q(t):
            return bsq.quantize(t, "mxfp8_e4m3")[0]

        bsq.gemm_gated_into(q(y), q(self.w_gate), q(self.w_up), h, "silu", gate, up)
        return h, gate, up, bsq.gemm_linear(q(h), q(self.w_down), self.b_down, self.x)

    def gradients(self):
        """Fills the gradients of one step; returns the mean loss and their norm (device tensors)."""
        x, n = self.x, (self.targets >= 0).sum()
        dgate, dup, ddown, dhead, dbias, dgamma, dbeta = self.grads
        y, mean, rstd = bsq.layer_norm(x, self.gamma, self.beta)
        h, gate, up, out = self.forward(y)
        loss, lse = bsq.linear_cross_entropy(out, self.head, self.targets)

        dloss = (1.0 / n).float().expand(loss.shape).contiguous()
        dout, dh, dy = torch.empty_like(out), torch.empty_like(h), torch.empty_like(y)
        bsq.linear_cross_entropy_backward_into(out, self.head, self.targets, lse, dloss, dout, dhead)
        bsq.linear_backward_into(dout, h, self.w_down, dh, ddown, dbias)
        bsq.gated_linear_backward_into(dh, y, self.w_gate, self.w_up, gate, up, dy, dgate, dup)
        bsq.layer_norm_backward_into(dy, x, self.gamma, mean, rstd, torch.empty_like(x), dgamma, dbeta)
        return loss.sum() / n, bsq.grad_norm(self.norms)

    def step(self, lr=3e-4, max_norm=1.0):
        """One training step; returns the mean loss and the gradient norm (device tensors)."""
        loss, norm = self.gradients()
        self.t += 1
        bsq.adamw_step(self.adam, lr, self.t, weight_decay=0.01, norm=norm, max_norm=max_norm, seed=0)
        return loss, norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--mxfp8", action="store_true")
    args = ap.parse_args()
    block = FeedForward(mxfp8=args.mxfp8)
    for i in range(args.steps):
        loss, norm = block.step()
        if i % 5 == 0 or i == args.steps - 1:
            print(f"step {i:3d}  loss {float(loss):.4f}  gradient norm {float(norm):.4f}")
    bsq.sync_status()


if __name__ == "__main__":
    main()
