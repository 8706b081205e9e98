"""GPU: the expert layer of examples/moe_layer.py with the balance loss.

The router's gradient is x^T (d + b): d the router's own (taken from the
kernels, which other tests check), b the balance loss's by the logits.  b is
off by (2 experts + 16) 2^-24 of its terms' magnitudes, the sum with d by half a
step, 2^-24, and the product in fp32 by tokens 2^-24 of the sum of its terms'
magnitudes."""
import importlib.util
import os

import numpy as np
import pytest

from gpu_util import torch
from mxfp4_precision_numerics_amd import mx
from oracle import cache as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


@pytest.fixture(scope="module")
def moe_layer():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_router_gradient(moe_layer):
    tt = torch()
    tokens, d, f, e, k, padding, weight = 300, 96, 64, 8, 2, 13, 5.0
    gen = tt.Generator("cuda").manual_seed(4)
    x = tt.randn((tokens, d), device="cuda", generator=gen).to(tt.bfloat16)
    dout = tt.randn((tokens, d), device="cuda", generator=gen).to(tt.bfloat16)
    layer = moe_layer.MoELayer(d, f, e, k, seed=3, balance=weight)
    layer.forward(x, padding)
    (got, _, _), _ = layer.backward(dout, seed=7)
    got = got.double().cpu().numpy()
    _, logits, ids, weights, offsets, _, slot, _, _, _, _, y = layer.kept
    _, dweights = mx.combine_bwd(dout, y, slot, weights, used_rows=offsets[-1:])
    own = mx.route_bwd(logits, ids, dweights).double().cpu().numpy()
    l64, ids64, x64 = logits.double().cpu().numpy(), ids.cpu().numpy(), x.double().cpu().numpy()
    loss, counts, slope = ref.balance(l64, ids64, 0)
    assert abs(float(layer.balanced[0]) - loss) <= (tokens + e + 8) * 2.0 ** -24 * loss
    assert np.array_equal(layer.balanced[1].cpu().numpy(), counts) and counts.sum() == (tokens - padding) * k
    term = ref.balance_bwd(l64, slope, 0, weight)
    s = np.stack([ref.scores_of(r, 0)[0] for r in l64])
    size = weight * s * (slope + (s * slope).sum(1, keepdims=True))
    bound = np.abs(x64.T) @ (np.abs(own) + np.abs(term) + size) * (tokens + 2 * e + 18) * 2.0 ** -24
    assert (np.abs(got - x64.T @ (own + term)) <= bound + 1e-30).all()
    # left out, the term would be an error of its own size: more than the bound and what the rest is off by
    assert np.abs(x64.T @ term).max() > 2 * bound.max()


def test_trains_with_the_balance_loss(moe_layer):
    lines = []
    losses = moe_layer.train(tokens=256, d_model=64, d_ff=64, experts=4, top_k=2, steps=3, report=lines.append,
                             balance=0.01)
    assert len(losses) == 3 and all(np.isfinite(losses)) and all("balance" in v for v in lines)
