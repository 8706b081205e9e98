"""GPU: the operators together, as the layer of examples/moe_layer.py uses
them.

The layer's outputs are compared with a 64-bit computation over the very
operands that the GEMMs read (decoded codes), step by step along the layer:
each step's own bound is 1e-2 relative (bf16 outputs: 2^-8, and one more
rounding of h, a or y on the way).  Its gradients, whose operands are rounded
stochastically to 4 bits, are compared with those of the unquantized layer in
fp32: E2M1 rounding alone costs 10 to 20% of a tensor's norm (an SNR of 17 to
19 dB), and a product of several such tensors at most the root of the sum of
their squares and the deviation of the forward pass, so 0.6 of the norm and a
cosine above 0.8 are asked for."""
import importlib.util
import os

import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from gpu_util import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


@pytest.fixture(scope="module")
def moe_layer():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def near(got, want, tol):
    got, want = got.double(), want.double()
    assert (got - want).norm() <= tol * want.norm(), float((got - want).norm() / want.norm())


def test_forward_step_by_step(moe_layer):
    tt = torch()
    tokens, d, f, e, k, padding = 300, 96, 64, 8, 2, 13
    layer = moe_layer.MoELayer(d, f, e, k, seed=3)
    x = tt.randn((tokens, d), device="cuda", generator=tt.Generator("cuda").manual_seed(4)).to(tt.bfloat16)
    out = layer.forward(x, padding)
    _, logits, ids, weights, offsets, row_index, slot, up, down, h, a, y = layer.kept
    used = int(offsets[-1])
    assert used == (tokens - padding) * k and (ids[-padding:] == -1).all() and (slot[-padding:] == -1).all()
    s = tt.softmax(logits[:-padding].double(), 1).topk(k, dim=1)
    assert tt.equal(s.indices, ids[:-padding].long())
    near(weights[:-padding], s.values / s.values.sum(1, keepdim=True), 1e-6)
    decode = lambda q, block_rows: mx.dequantize(q[0], q[1], block_rows=block_rows).double()  # noqa: E731
    w_up, w_down = decode(up[:2], 32), decode(down[:2], 32)
    xq, aq = decode(mx.quantize_1d(x), 1), decode(mx.quantize_1d(a), 1)
    want = tt.zeros((tokens, d), dtype=tt.float64, device="cuda")
    for g in range(e):
        b, c = int(offsets[g]), int(offsets[g + 1])
        tok = row_index[b:c].long()
        assert tt.equal(tt.sort(tok).values, tok)          # in token order
        near(h[b:c], xq[tok] @ w_up[g], 1e-2)
        near(y[b:c], aq[b:c] @ w_down[g], 1e-2)
        wt = (weights * (ids == g)).sum(1)[tok].double()
        want[tok] += wt[:, None] * y[b:c].double()
    near(out, want + x.double(), 1e-2)
    assert tt.equal(out[-padding:], x[-padding:])          # padding passes through


def test_gradients_against_the_unquantized_layer(moe_layer):
    tt = torch()
    tokens, d, f, e, k, padding = 512, 128, 64, 4, 2, 9
    layer = moe_layer.MoELayer(d, f, e, k, seed=5)
    gen = tt.Generator("cuda").manual_seed(6)
    x = tt.randn((tokens, d), device="cuda", generator=gen).to(tt.bfloat16)
    dout = tt.randn((tokens, d), device="cuda", generator=gen).to(tt.bfloat16)
    layer.forward(x, padding)
    (drouter, dup, ddown), dx = layer.backward(dout, seed=7)
    ids = layer.kept[2].long()
    p = [v.clone().requires_grad_() for v in layer.parameters()]
    leaf = x.float().requires_grad_()
    weights = tt.softmax((leaf @ p[0]).gather(1, ids.clamp(min=0)), 1) * (ids >= 0)
    out = leaf
    for g in range(e):
        gate, up = (leaf @ p[1][g]).chunk(2, dim=1)
        out = out + (weights * (ids == g)).sum(1, keepdim=True) * ((tt.nn.functional.silu(gate) * up) @ p[2][g])
    want = tt.autograd.grad((out * dout.float()).sum(), p + [leaf])
    for got, ref in zip((drouter, dup, ddown, dx), want):
        got, ref = got.double().flatten(), ref.double().flatten()
        cosine = float(got @ ref / (got.norm() * ref.norm()))
        assert tt.isfinite(got).all() and cosine > 0.8 and (got - ref).norm() < 0.6 * ref.norm(), cosine


def test_training_lowers_the_loss(moe_layer):
    losses = moe_layer.train(tokens=512, d_model=128, d_ff=64, experts=4, top_k=2, steps=40)
    assert all(np.isfinite(losses)) and np.mean(losses[-5:]) < 0.8 * losses[0], losses
