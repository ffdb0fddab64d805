"""One training step and one serving step of a pre-norm MLP block, all in this library's kernels:

    h  = x + residual;  n = RMSNorm(h) as MXFP8 copies          rmsnorm_quantize
    a  = gelu(n W1^T) (fused), y = a W2^T                       linear_fwd_gelu, linear_fwd
    backward through fc2, GeLU and fc1                          linear_dgrad_dgelu, linear_bwd
    dh = dres + the norm's backward, dgamma                     rmsnorm_bwd
    the global norm of dW1, dW2 and dgamma, and clipping        grad_norm, grad_clip

The gradients are clipped in place. Serving runs the same block for any number of tokens, one
among them: the norm pads its FP8 copy to the 128 rows that the GEMM needs.

    python examples/prenorm_mlp_step.py [--tokens 1000] [--hidden 4096] [--ffn 16384]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scaled_quantize_fp8_gb300 as F  # noqa: E402

REC = F.Recipe(kind="mxfp8")


class PreNormMlp:
    """The block's weights, their MXFP8 copies and their gradients."""

    def __init__(self, hidden, ffn, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") * 0.02
            return w.to(torch.bfloat16)

        self.gamma = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        self.w1, self.w2 = weight(ffn, hidden), weight(hidden, ffn)
        self.w1_q, self.w2_q = F.quantize_group(REC, [self.w1, self.w2], ["weight", "weight"])
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.dgamma = torch.empty(hidden, dtype=torch.float32, device="cuda")
        self.grads = F.GradList([self.dw1, self.dw2, self.dgamma])

    def forward(self, x, residual, train=True):
        """y and the new residual stream; what backward needs is kept when training."""
        n_q, h, rstd, _ = F.rmsnorm_quantize(REC, x, self.gamma, residual=residual,
                                             want_col=train)
        a_q, pre_q = F.linear_fwd_gelu(REC, n_q, self.w1_q)
        y = F.linear_fwd(REC, a_q, self.w2_q)
        self.saved = (n_q, h, rstd, a_q, pre_q) if train else None
        return y[:x.shape[0]], h

    def backward(self, dy, dres):
        """The gradient of x (and of residual) from y's and the stream's; fills the weights'."""
        n_q, h, rstd, a_q, pre_q = self.saved
        rows = torch.nn.functional.pad(dy, (0, 0, 0, n_q.rows - dy.shape[0]))
        dy_q = F.quantize(REC, rows, "grad")
        dpre_q = F.linear_dgrad_dgelu(REC, dy_q, self.w2_q, pre_q)
        F.linear_bwd(REC, dy_q, a_q, None, want_dx=False, dw=self.dw2)
        dn, _ = F.linear_bwd(REC, dpre_q, n_q, self.w1_q, dw=self.dw1)
        dh, _ = F.rmsnorm_bwd(dn, h, rstd, self.gamma, dres=dres, dgamma=self.dgamma)
        return dh

    def clip(self, max_norm):
        norm, coef = F.grad_norm(self.grads, max_norm=max_norm)
        F.grad_clip(self.grads, coef)
        return norm, coef


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=16384)
    args = ap.parse_args()
    block = PreNormMlp(args.hidden, args.ffn)
    shape = (args.tokens, args.hidden)
    x, residual = (torch.randn(shape, device="cuda").to(torch.bfloat16) for _ in range(2))
    dy, dres = ((torch.randn(shape, device="cuda") * 1e-3).to(torch.bfloat16) for _ in range(2))
    y, h = block.forward(x, residual)
    dh = block.backward(dy, dres)
    norm, coef = block.clip(max_norm=0.5)
    print(f"train: {args.tokens} tokens, |y| {y.float().norm():.4g}, |dh| {dh.float().norm():.4g}, "
          f"gradient norm {norm.item():.4g}, coefficient {coef.item():.4g}")
    one, _ = block.forward(x[:1], residual[:1], train=False)
    print(f"serve: one token, the same as in the batch: {torch.equal(one[0], y[0])}")


if __name__ == "__main__":
    main()
