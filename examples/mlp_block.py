"""A training step of a pre-norm gated MLP block that keeps its activations in
8 bits and hands its gradients to the compressor.

    h = x + r;  y = rmsnorm(h) * w;  [g | u] = y Wgu^T;  a = silu(g) u;  out = a Wd^T

Between forward and backward the block keeps the checkpoints of the
normalised rows (for the norm's gradient and for dWgu, with w on its
columns), of g and of u (for the activation's gradient, which gives a again
as a checkpoint, for dWd): 1.03 bytes per element instead of the 2 of bf16 for
h, y, g, u and a.  The weight gradients go straight into the tensors of the
flat fp32 arena, which error-feedback Top-k then compresses.

    python examples/mlp_block.py [--tokens 8192] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_compression_gb300 as gc  # noqa: E402

EPS = 1e-5


class GatedBlock:
    """Weights in bf16 (the norm's in fp32), buffers for `tokens` rows, and the
    gradient arena: [Wgu, Wd, w] one after another."""

    def __init__(self, tokens, width, hidden, density=0.01, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        bf = dict(device=device, dtype=torch.bfloat16)
        self.tokens, self.width, self.hidden = tokens, width, hidden
        self.w = torch.ones(width, device=device)
        self.wgu = (torch.randn(2 * hidden, width, generator=gen, device=device) / width ** 0.5).to(torch.bfloat16)
        self.wd = (torch.randn(width, hidden, generator=gen, device=device) / hidden ** 0.5).to(torch.bfloat16)
        # activations of one step
        self.h, self.y = (torch.empty(tokens, width, **bf) for _ in range(2))
        self.a = torch.empty(tokens, hidden, **bf)
        self.dgu = torch.empty(tokens, 2 * hidden, **bf)
        self.dx = torch.empty(tokens, width, **bf)
        self.rstd = torch.empty(tokens, device=device)
        # what forward keeps for backward
        self.kept_norm = gc.ActCheckpoint(tokens, width, device)
        self.kept_gate, self.kept_up = (gc.ActCheckpoint(tokens, hidden, device) for _ in range(2))
        self.kept_act = gc.ActCheckpoint(tokens, hidden, device)   # written by backward, for dWd
        # the gradient arena and its compressor
        sizes = [2 * hidden * width, width * hidden, width]
        off = np.concatenate(([0], np.cumsum(sizes)))
        k = [min(n, int(np.ceil(density * n))) for n in sizes]
        self.layout = gc.Layout(off, k, device=device)
        self.grad = torch.zeros(self.layout.numel, device=device)
        self.error = torch.zeros_like(self.grad)
        self.dwgu = self.grad[:off[1]].view(2 * hidden, width)
        self.dwd = self.grad[off[1]:off[2]].view(width, hidden)
        self.dw = self.grad[off[2]:]
        self.compressor = gc.TopkCompressor(self.layout, gc.GC_EF | gc.GC_INT8, device=device)
        self.ws_norm = gc.rmsnorm_backward_workspace(tokens, width, device)
        self.ws_gu = gc.act_weight_grad_workspace(tokens, 2 * hidden, width, torch.bfloat16, device)
        self.ws_d = gc.act_weight_grad_workspace(tokens, width, hidden, torch.bfloat16, device)

    @property
    def kept_bytes(self):
        return sum(c.nbytes for c in (self.kept_norm, self.kept_gate, self.kept_up)) + 4 * self.tokens

    def forward(self, x, residual):
        """(block output, residual stream); keeps the checkpoints."""
        gc.rmsnorm(x, self.w, EPS, self.y, residual=residual, h=self.h, rstd=self.rstd, ckpt=self.kept_norm)
        gu = self.y @ self.wgu.T
        gc.gated_act(gc.GC_GATE_SILU, gu[:, :self.hidden], gu[:, self.hidden:], self.a, ckpt_gate=self.kept_gate,
                     ckpt_up=self.kept_up)
        return self.a @ self.wd.T, self.h

    def backward(self, dout, dh, accumulate=False):
        """Gradient of x (and of the residual); the weights' into the arena,
        added to what is there for a later micro-batch."""
        da = dout @ self.wd
        gc.gated_act_backward(gc.GC_GATE_SILU, da, self.kept_gate, self.kept_up, self.dgu[:, :self.hidden],
                              self.dgu[:, self.hidden:], ckpt_out=self.kept_act)
        gc.act_weight_grad(dout, self.kept_act, self.dwd, self.ws_d, accumulate=accumulate)
        gc.act_weight_grad(self.dgu, self.kept_norm, self.dwgu, self.ws_gu, col_scale=self.w, accumulate=accumulate)
        dy = self.dgu @ self.wgu
        gc.rmsnorm_backward(dy, self.kept_norm, self.rstd, self.w, self.dx, self.dw, self.ws_norm, dh=dh,
                            accumulate=accumulate)
        return self.dx

    def compress(self, step):
        """The payload of this worker's gradients: indices, int8 codes, scales."""
        idx, _, q, scale = self.compressor(self.grad, self.error, seed=1, it=step)
        return idx, q, scale


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    args = ap.parse_args()
    block = GatedBlock(args.tokens, args.width, args.hidden)
    x, r, dout, dh = (torch.randn(args.tokens, args.width, device="cuda").to(torch.bfloat16) for _ in range(4))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(args.steps):
        begin.record()
        block.forward(x, r)
        block.backward(dout, dh)
        idx, q, scale = block.compress(step)
        end.record()
        end.synchronize()
        print("step %d: %.2f ms, %d of %d gradient entries sent" % (step, begin.elapsed_time(end), idx.numel(),
                                                                    block.layout.numel))
    wide = 2 * args.tokens * (2 * args.width + 3 * args.hidden)
    print("kept for backward: %.1f MB, in bf16 (h, y, g, u, a) %.1f MB" % (block.kept_bytes / 1e6, wide / 1e6))


if __name__ == "__main__":
    main()
