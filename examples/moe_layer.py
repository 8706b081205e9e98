"""A mixture-of-experts layer trained on one GPU, every step on the library's
kernels: routing, dispatch plan, MXFP4 quantizers and grouped GEMMs, the
weighted combine, all their gradients, and clipping by the global norm.

    python examples/moe_layer.py [--tokens N] [--d-model D] [--d-ff F] [--experts E] [--top-k K] [--steps S]
                                 [--balance C]

The layer learns to reproduce a fixed random mixture of experts of the same
shape from synthetic tokens; the loss of every step is printed.  With --balance
C times the router's balance loss is added to it.  Sizes are multiples of 32.
The activation between the two expert linears (SiLU-gated) and the router's
small products are plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mxfp4_precision_numerics_amd import mx  # noqa: E402


class MoELayer:
    """y = x + sum over a token's experts of weight * down(gated(up(x)))."""

    def __init__(self, d_model, d_ff, experts, top_k, seed, balance=0.0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, device="cuda", generator=gen) * shape[-2] ** -0.5

        self.top_k, self.experts, self.balance = top_k, experts, balance
        self.router = normal(d_model, experts)
        self.up = normal(experts, d_model, 2 * d_ff)       # gate and up projections side by side
        self.down = normal(experts, d_ff, d_model)

    def parameters(self):
        return [self.router, self.up, self.down]

    def forward(self, x, padding):
        """x [tokens, d_model] bf16; the last `padding` tokens go to no expert.
        Keeps what backward needs."""
        logits = x.float() @ self.router
        if padding:
            logits[-padding:] = -float("inf")
        ids, weights = mx.route(logits, self.top_k)
        if self.balance:                                   # its loss, the experts' assignments, what backward needs
            self.balanced = mx.balance(logits, ids)
        offsets, row_index, slot = mx.route_plan(ids, self.experts)
        rows, d = row_index.numel(), x.shape[1]
        up, down = mx.quantize_2d(self.up), mx.quantize_2d(self.down)
        # tokens are quantized once and gathered, as codes, by the GEMM
        h = mx.grouped_gemm(*mx.quantize_1d(x), up[2], up[3], offsets, rows, self.up.shape[2], d,
                            a_row_index=row_index, b_scale_2d=True)
        a = self.gated(h)
        y = mx.grouped_gemm(*mx.quantize_1d(a), down[2], down[3], offsets, rows, d, a.shape[1], b_scale_2d=True)
        self.kept = (x, logits, ids, weights, offsets, row_index, slot, up, down, h, a, y)
        return mx.combine(y, slot, weights, residual=x)

    @staticmethod
    def gated(h):
        gate, up = h.float().chunk(2, dim=1)
        return (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)

    def backward(self, dout, seed):
        """Gradients of the parameters, and of x, from dout [tokens, d_model]
        bf16.  Weight gradients contract both operands, quantized along the
        tokens with the randomized Hadamard transform and stochastic rounding."""
        x, logits, ids, weights, offsets, row_index, slot, up, down, h, a, y = self.kept
        rows, d = y.shape
        col = dict(block_axis=0, group_offsets=offsets, use_rht=True, sign_mask=mx.rht_sign_mask(seed), rnd=mx.SR,
                   seed=seed)
        row = dict(rnd=mx.SR, seed=seed)
        counts = (offsets[1:] - offsets[:-1] + 31) // 32 * 32
        padded = torch.cat([counts.new_zeros(1), counts.cumsum(0, dtype=torch.int32)])
        kp = mx.padded_capacity(rows, self.experts)

        def weight_gradient(left, right, m, n):
            # (positions past the padded total are in no group)
            return mx.grouped_gemm(*left, *right, padded, m, n, kp, group_dim_k=True, out_dtype=torch.float32)

        dy, dweights = mx.combine_bwd(dout, y, slot, weights, used_rows=offsets[-1:])
        dlogits = mx.route_bwd(logits, ids, dweights)
        if self.balance:
            mx.balance_bwd(logits, self.balanced[2], scale=self.balance, add=dlogits, dlogits=dlogits)
        ddown = weight_gradient(mx.quantize_1d(a, stream_id=0, **col), mx.quantize_1d(dy, stream_id=1, **col),
                                a.shape[1], d)
        da = mx.grouped_gemm(*mx.quantize_1d(dy, stream_id=2, **row), down[0], down[1], offsets, rows, a.shape[1], d,
                             b_scale_2d=True)
        with torch.enable_grad():
            leaf = h.detach().requires_grad_()
            dh, = torch.autograd.grad(self.gated(leaf), leaf, da)
        used = torch.arange(rows, device="cuda")[:, None] < offsets[-1]
        dh = torch.where(used, dh, torch.zeros_like(dh))
        dup = weight_gradient(mx.quantize_1d(x, row_index=row_index, stream_id=3, **col),
                              mx.quantize_1d(dh, stream_id=4, **col), d, h.shape[1])
        dx_rows = mx.grouped_gemm(*mx.quantize_1d(dh, stream_id=5, **row), up[0], up[1], offsets, rows, d, h.shape[1],
                                  b_scale_2d=True)
        # x reaches its experts by the gather and the router, and the output directly
        dx = mx.combine(dx_rows, slot, residual=(dout.float() + dlogits @ self.router.t()).to(dout.dtype))
        return [x.float().t() @ dlogits, dup, ddown], dx


def train(tokens=512, d_model=256, d_ff=128, experts=8, top_k=2, steps=60, rate=2.0, max_norm=1.0, seed=0,
          report=None, balance=0.0):
    """Losses of the steps, without the balance loss."""
    gen = torch.Generator("cuda").manual_seed(seed)
    teacher = MoELayer(d_model, d_ff, experts, top_k, seed + 1)
    layer = MoELayer(d_model, d_ff, experts, top_k, seed + 2, balance)
    padding = tokens // 16
    x = torch.randn((tokens, d_model), device="cuda", generator=gen).to(torch.bfloat16)
    target = teacher.forward(x, padding).float()
    losses = []
    for step in range(steps):
        out = layer.forward(x, padding)
        error = out.float() - target
        losses.append(float((error ** 2).sum(1).mean()))
        grads, _ = layer.backward((2.0 / tokens * error).to(torch.bfloat16), seed=step + 1)
        norm = mx.grad_clip(grads, max_norm)
        for p, g in zip(layer.parameters(), grads):
            p -= rate * g
        if report:
            line = "step %3d  loss %9.4f  gradient norm %8.4f" % (step, losses[-1], float(norm))
            if balance:
                line += "  balance %6.4f  fullest expert %d" % (float(layer.balanced[0]), int(layer.balanced[1].max()))
            report(line)
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("d-model", 256), ("d-ff", 128), ("experts", 8), ("top-k", 2), ("steps", 60)):
        parser.add_argument("--" + name, type=int, default=value)
    parser.add_argument("--balance", type=float, default=0.0)
    args = parser.parse_args()
    train(args.tokens, args.d_model, args.d_ff, args.experts, args.top_k, args.steps, report=print,
          balance=args.balance)
