"""GPU: the global gradient norm and clipping against 64-bit sums.

Tolerances.  Squares are summed in fp64, so the norm is the exact one but for
its rounding to fp32 (2^-24 relative; 2^-23 allows for the sum's own last
bits).  A clipped value is fl32(coef) * g rounded to fp32 (each 2^-24), then to
the tensor's type (2^-9 for bf16); 2^-22 and 2^-8 cover both."""
import math

import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from oracle import moe
from gpu_util import torch

pytestmark = pytest.mark.gpu


def tensors(sizes, types, seed, scale=1e-2):
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(seed)
    return [(scale * tt.randn(n, device="cuda", generator=gen)).to(tt.bfloat16 if b else tt.float32)
            for n, b in zip(sizes, types)]


def norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check_clipped(outs, grads, norm, max_norm):
    tt = torch()
    coef = moe.clip_coef(norm, max_norm)
    for o, g in zip(outs, grads):
        want = g.double() * coef
        tol = want.abs() * (2.0 ** -8 if g.dtype == tt.bfloat16 else 2.0 ** -22) + 1e-38
        assert o.dtype == g.dtype and ((o.double() - want).abs() <= tol).all()


CASES = [
    ([1], [0]), ([1], [1]), ([5, 0, 3], [1, 0, 0]), ([2880, 7, 16385, 1], [1, 1, 0, 0]),
    ([32768, 32769, 65535, 16384, 16383], [1, 1, 1, 0, 0]), ([1_000_003], [0]), ([3_000_001, 9], [1, 0]),
    ([1 + 37 * i for i in range(97)], [i % 2 for i in range(97)]),            # more than one table
    ([0] * 100 + [3] * 200, [i % 3 == 0 for i in range(300)]),
    ([45_000_000], [0]),                                                      # more chunks than workgroups
]


@pytest.mark.parametrize("sizes,types", CASES, ids=lambda v: "%d" % len(v))
def test_norm_and_clip(sizes, types):
    tt = torch()
    grads = tensors(sizes, types, 1)
    kept = [g.clone() for g in grads]
    norm = norm64(grads)
    got = mx.grad_norm(grads)
    assert got.dim() == 0 and got.dtype == tt.float32 and abs(float(got) - norm) <= 2.0 ** -23 * norm
    if sum(sizes) <= 200_000:
        assert abs(moe.grad_norm([g.float().cpu().numpy() for g in grads]) - norm) <= 1e-12 * norm
    for max_norm in (norm / 3, norm * 2, 0.0):
        outs = [tt.full_like(g, 7.0) for g in grads]
        n = mx.grad_clip(grads, max_norm, outs=outs)
        assert tt.equal(n, got) and all(tt.equal(a, b) for a, b in zip(grads, kept))
        check_clipped(outs, grads, norm, max_norm)
        mine = [g.clone() for g in grads]
        assert tt.equal(mx.grad_clip(mine, max_norm), got)
        assert all(tt.equal(a, b) for a, b in zip(mine, outs))
        if max_norm > norm:
            assert all(tt.equal(a, b) for a, b in zip(mine, kept))


def test_no_tensors():
    assert float(mx.grad_norm([])) == 0.0 and float(mx.grad_clip([], 1.0)) == 0.0
    empty = torch().zeros(0, device="cuda")
    assert float(mx.grad_norm([empty])) == 0.0 and float(mx.grad_clip([empty, empty], 1.0)) == 0.0


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-42])
def test_squares_outside_fp32(scale):
    tt = torch()
    grads = [tt.full((1000,), scale, device="cuda"), tt.full((77,), -scale, device="cuda")]
    norm = norm64(grads)
    assert abs(float(mx.grad_norm(grads)) - norm) <= 2.0 ** -23 * norm + 1e-45
    outs = [tt.empty_like(g) for g in grads]
    mx.grad_clip(grads, 1.0, outs=outs)
    coef = moe.clip_coef(norm, 1.0)
    for o, g in zip(outs, grads):
        assert ((o.double() - g.double() * coef).abs() <= 2.0 ** -22 * (g.double() * coef).abs() + 1.5e-45).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    tt = torch()
    grads = tensors([5000, 333, 70_000], [0, 1, 1], 4, scale=10.0)
    grads[1][17] = bad
    kept = [g.clone() for g in grads]
    outs = [tt.zeros_like(g) for g in grads]
    n = float(mx.grad_clip(grads, 0.5, outs=outs))
    assert math.isnan(n) if math.isnan(bad) else n == math.inf
    mx.grad_clip(grads, 0.5)
    for o, g, k in zip(outs, grads, kept):
        assert tt.equal(tt.nan_to_num(o, nan=123.0), tt.nan_to_num(k, nan=123.0))
        assert tt.equal(tt.nan_to_num(g, nan=123.0), tt.nan_to_num(k, nan=123.0))


@pytest.mark.parametrize("count", [2, 9_000_000])
def test_a_norm_past_fp32_leaves_the_values(count):
    """Finite gradients whose norm is not: *norm is infinite, so the values
    stay; the largest norm that fp32 holds still clips."""
    tt = torch()
    grads = [tt.full((count,), -1e34, device="cuda"), tt.tensor([3e38, 3e38], device="cuda"),
             tt.tensor([1.0, 2.0 ** 127], dtype=tt.bfloat16, device="cuda")]
    kept = [g.clone() for g in grads]
    outs = [tt.zeros_like(g) for g in grads]
    for max_norm in (1.0, 1e38):
        assert float(mx.grad_clip(grads, max_norm, outs=outs)) == math.inf == float(mx.grad_norm(grads))
        assert float(mx.grad_clip(grads, max_norm)) == math.inf
        assert all(tt.equal(o, k) and tt.equal(g, k) for o, g, k in zip(outs, grads, kept))
    most = tt.tensor([float(tt.finfo(tt.float32).max)], device="cuda")
    assert float(mx.grad_clip([most], 1.0)) == float(tt.finfo(tt.float32).max)
    assert abs(float(most) - 1.0) <= 2.0 ** -22


def test_offsets_past_32_bits():
    """One tensor of more than 2^32 bytes and 2^31 elements."""
    tt = torch()
    n = 2 ** 31 + 12_345
    g = tt.zeros(n, dtype=tt.bfloat16, device="cuda")
    at = [0, 2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 4097, n - 1]
    for i, a in enumerate(at):
        g[a] = float(i + 1)
    norm = math.sqrt(sum((i + 1) ** 2 for i in range(len(at))))
    out = tt.full_like(g, 7.0)
    assert abs(float(mx.grad_clip([g], norm / 2, outs=[out])) - norm) <= 2.0 ** -23 * norm
    assert int((out != 0).sum()) == len(at)
    for i, a in enumerate(at):
        assert abs(float(out[a]) - (i + 1) * 0.5) <= 2.0 ** -8 * (i + 1)


@pytest.mark.parametrize("bf16", [0, 1])
def test_views_off_their_alignment(bf16):
    tt = torch()
    buf = tensors([200_001], [bf16], 5)[0]
    out = tt.full_like(buf, 7.0)
    for a, b in ((1, 200_001), (3, 40_000), (2, 9), (5, 5)):
        g, o = buf[a:b], out[a:b]
        norm = norm64([g])
        assert abs(float(mx.grad_norm([g])) - norm) <= 2.0 ** -23 * norm
        out.fill_(7.0)
        mx.grad_clip([g], norm / 2, outs=[o])
        check_clipped([o], [g], norm, norm / 2)
        assert (out[:a] == 7.0).all() and (out[b:] == 7.0).all()
    shifted = tt.empty(200_008, dtype=buf.dtype, device="cuda")[3:200_004]
    mx.grad_clip([buf], 0.1, outs=[shifted])               # the two sides aligned differently
    check_clipped([shifted], [buf], norm64([buf]), 0.1)


def test_same_bits_every_time():
    tt = torch()
    grads = tensors([1_234_567, 99, 500_000], [0, 1, 1], 6)
    first = mx.grad_norm(grads)
    for _ in range(5):
        assert tt.equal(mx.grad_norm(grads), first)


def test_other_stream_and_graph():
    tt = torch()
    grads = tensors([30_000, 501, 70_001], [0, 1, 1], 7)
    outs = [tt.empty_like(g) for g in grads]
    tt.cuda.synchronize()
    side = tt.cuda.Stream()
    with tt.cuda.stream(side):
        n = mx.grad_clip(grads, 0.5, outs=outs)
    side.synchronize()
    assert abs(float(n) - norm64(grads)) <= 2.0 ** -23 * norm64(grads)
    check_clipped(outs, grads, norm64(grads), 0.5)
    graph = tt.cuda.CUDAGraph()
    with tt.cuda.graph(graph):
        n = mx.grad_clip(grads, 0.5, outs=outs)
    for i in range(3):
        for j, g in enumerate(grads):
            g.copy_(tensors([g.numel()], [0], 100 + 3 * i + j)[0])
        graph.replay()
        tt.cuda.synchronize()
        assert abs(float(n) - norm64(grads)) <= 2.0 ** -23 * norm64(grads)
        check_clipped(outs, grads, norm64(grads), 0.5)


def test_refusals():
    tt = torch()
    g = tt.zeros(10, device="cuda")
    with pytest.raises(TypeError):
        mx.grad_norm([g.half()])
    with pytest.raises(ValueError):
        mx.grad_norm([g.cpu()])
    with pytest.raises(ValueError):
        mx.grad_norm([tt.zeros((4, 4), device="cuda").t()[:, :2]])
    with pytest.raises(ValueError):
        mx.grad_clip([g], 1.0, outs=[])
    with pytest.raises(ValueError):
        mx.grad_clip([g], 1.0, outs=[g.bfloat16()])
    with pytest.raises(ValueError):
        mx.grad_clip([g], 1.0, outs=[tt.zeros(11, device="cuda")])
    for bad in (-1.0, float("nan")):
        with pytest.raises(mx.MXError):
            mx.grad_clip([g], bad)
    with pytest.raises(ValueError):
        mx.grad_norm([g], workspace=tt.zeros(8, dtype=tt.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mx.grad_norm([g], norm=tt.zeros(1, device="cuda"))
