"""The bounds of test_gpu_precision.py notice a missing term: with q or p as two
bf16 terms in place of three, everything else in 64 bits, outputs are past them,
with three they are not."""
import numpy as np
import pytest

import oracle
from gpu_util import bf16_bits_to_f64
from test_gpu_precision import U, bounds


def as_terms(x, terms):
    """What a sum of so many bf16, each of what the last ones left, holds of x."""
    held = np.zeros_like(x)
    for _ in range(terms):
        left = (x - held).astype(np.float32)
        held = held + bf16_bits_to_f64(oracle.round_bf16_bits(left.ravel())).reshape(x.shape)
    return held


@pytest.mark.parametrize("q_terms, p_terms, reach, within", [(3, 3, 1, True), (3, 3, 8, True), (2, 3, 8, False), (3, 2, 1, False)])
@pytest.mark.parametrize("rows", [16, 300])
@pytest.mark.parametrize("dim", [32, 256])
def test_two_terms_are_past_the_bounds(dim, rows, q_terms, p_terms, reach, within):
    q = np.random.default_rng(rows).uniform(-reach, reach, size=(rows, dim)).astype(np.float32).astype(np.float64)
    exact = np.exp(q)
    p = np.exp(as_terms(q, q_terms))
    total = p.sum(-1, keepdims=True)
    # (p relative to the row's largest, as fp32)
    top = p.max(-1, keepdims=True)
    out = as_terms((p / top).astype(np.float32).astype(np.float64), p_terms) / (total / top)
    far = np.abs(out / (exact / exact.sum(-1, keepdims=True)) - 1.0).max() / U
    limit = bounds(reach, np.log(exact.sum(-1)))[0]
    assert (far <= limit) == within, (far, limit)
