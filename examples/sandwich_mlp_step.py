"""A training step and a serving step of a stack of MLP blocks with a norm on both sides, a gate per
channel and a residual scale, in this library's kernels:

    n0 = RMSNorm(x) as MXFP8 copies; x kept in 8 bits            rmsnorm_quantize, checkpoint
    o  = gelu(n W1^T) W2^T                                       linear_fwd_gelu, linear_fwd
    h' = h + scale gate RMSNorm(o),  n' = RMSNorm(h')            branch_rmsnorm_quantize
    backward: dh, do from the checkpoints of h' and o            branch_rmsnorm_bwd
    the column copy of n, which wgrad reads, made again from
    the checkpoint of h instead of kept                          checkpoint_quantize
    fc2, GeLU and fc1                                            linear_dgrad_dgelu, linear_bwd
    the first norm, from x's checkpoint                          rmsnorm_bwd

Between forward and backward a block keeps one byte an element of h and of o (and 1/32 for scales),
where bf16 tensors and the column copy of n would take five. Serving runs the same stack for any
number of tokens, one among them.

    python examples/sandwich_mlp_step.py [--tokens 1000] [--hidden 4096] [--ffn 16384] [--blocks 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scaled_quantize_fp8_gb300 as F  # noqa: E402

REC = F.Recipe(kind="mxfp8")


class Block:
    """One block's weights, their MXFP8 copies and their gradients. gamma is the weight of the norm
    in front of it, gamma_post of the one behind it."""

    def __init__(self, hidden, ffn, gen):
        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") * 0.02
            return w.to(torch.bfloat16)

        def near(value):
            v = value + 0.1 * torch.randn(hidden, generator=gen, device="cuda")
            return v.to(torch.bfloat16)

        self.gamma, self.gamma_post, self.gate = near(1.0), near(1.0), near(0.5)
        self.w1, self.w2 = weight(ffn, hidden), weight(hidden, ffn)
        self.w1_q, self.w2_q = F.quantize_group(REC, [self.w1, self.w2], ["weight", "weight"])
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.dgamma, self.dgamma_post, self.dgate = (
            torch.empty(hidden, dtype=torch.float32, device="cuda") for _ in range(3))


class SandwichMlp:
    def __init__(self, hidden, ffn, blocks=2, scale=0.5, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(hidden, ffn, gen) for _ in range(blocks)]
        self.gamma = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")    # of the last norm
        self.dgamma = torch.empty(hidden, dtype=torch.float32, device="cuda")
        self.scale = scale

    def forward(self, x, train=True):
        """The last norm's output (bf16) for bf16 tokens x; what backward needs is kept when
        training."""
        rows, hidden = x.shape
        n_q, h, rstd, _ = F.rmsnorm_quantize(REC, x, self.blocks[0].gamma, want_col=False)
        self.saved = []
        h_ck = F.checkpoint(x) if train else None
        for i, b in enumerate(self.blocks):
            a_q, pre_q = F.linear_fwd_gelu(REC, n_q, b.w1_q)
            o = F.linear_fwd(REC, a_q, b.w2_q)[:rows]
            last = i + 1 == len(self.blocks)
            o_ck, next_ck = ((F.empty_checkpoint(rows, hidden), F.empty_checkpoint(rows, hidden))
                             if train else (None, None))
            n_q, h, next_rstd, rstd_o, y = F.branch_rmsnorm_quantize(
                None if last else REC, o, h, self.gamma if last else self.blocks[i + 1].gamma,
                gamma_post=b.gamma_post, gate=b.gate, scale=self.scale, want_row=not last,
                want_col=False, want_y=last, branch_ckpt=o_ck, h_ckpt=next_ck)
            if train:
                self.saved.append((h_ck, rstd, a_q, pre_q, o_ck, rstd_o))
            h_ck, rstd = next_ck, next_rstd
        self.last = (h_ck, rstd)
        return y

    def backward(self, dy):
        """The gradient of x from that of the output; fills the weights'."""
        h_ck, rstd = self.last
        gamma, dgamma, dn, dh = self.gamma, self.dgamma, dy, None
        for b, (x_ck, x_rstd, a_q, pre_q, o_ck, rstd_o) in zip(reversed(self.blocks),
                                                               reversed(self.saved)):
            dh, do, *_ = F.branch_rmsnorm_bwd(
                dn, h_ck, rstd, gamma, o_ck, rstd_branch=rstd_o, gamma_post=b.gamma_post,
                gate=b.gate, scale=self.scale, dres=dh, dgamma=dgamma, dgamma_post=b.dgamma_post,
                dgate=b.dgate)
            rows = torch.nn.functional.pad(do, (0, 0, 0, a_q.rows - do.shape[0]))
            do_q = F.quantize(REC, rows, "grad")
            dpre_q = F.linear_dgrad_dgelu(REC, do_q, b.w2_q, pre_q)
            F.linear_bwd(REC, do_q, a_q, None, want_dx=False, dw=b.dw2)
            n_q = F.checkpoint_quantize(REC, x_ck, x_rstd, b.gamma, want_row=False)
            dn, _ = F.linear_bwd(REC, dpre_q, n_q, b.w1_q, dw=b.dw1)
            h_ck, rstd, gamma, dgamma = x_ck, x_rstd, b.gamma, b.dgamma
        dx, _ = F.rmsnorm_bwd(dn, h_ck, rstd, gamma, dres=dh, dgamma=dgamma)
        return dx


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--ffn", type=int, default=16384)
    ap.add_argument("--blocks", type=int, default=2)
    args = ap.parse_args()
    m = SandwichMlp(args.hidden, args.ffn, args.blocks)
    x = torch.randn(args.tokens, args.hidden, device="cuda").to(torch.bfloat16)
    dy = (torch.randn(args.tokens, args.hidden, device="cuda") * 1e-3).to(torch.bfloat16)
    y = m.forward(x)
    dx = m.backward(dy)
    print(f"train: {args.tokens} tokens, |y| {y.float().norm():.4g}, |dx| {dx.float().norm():.4g}, "
          f"|dgate| {m.blocks[0].dgate.norm():.4g}")
    one = m.forward(x[:1], train=False)
    print(f"serve: one token, the same as in the batch: {torch.equal(one[0], y[0])}")


if __name__ == "__main__":
    main()
