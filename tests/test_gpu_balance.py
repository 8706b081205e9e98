"""GPU: the balance loss, its counts and its gradient against the 64-bit
definitions of oracle/cache.py.

Tolerances.  A score is an exponential (2 steps of 2^-24) over a sum of
`experts` of them in fp32, at most (experts + 8) 2^-24 relative; the sum over
the tokens adds at most tokens 2^-24 of itself: the loss, a sum of positive
terms, is off by (tokens + experts + 8) 2^-24 relative.  The gradient's
difference slope_e - <slope, s> is off by (2 experts + 16) 2^-24 of the sum of
both magnitudes, and the result is rounded once to the logits' type."""
import numpy as np
import pytest

import oracle
from mxfp4_precision_numerics_amd import mx
from oracle import cache as ref
from gpu_util import bf16_bits_to_f64, dev, torch

pytestmark = pytest.mark.gpu


def logits_of(tokens, experts, kind, seed, pad=0, padding=0, scale=2.0):
    tt = torch()
    x = tt.from_numpy((np.random.default_rng(seed).normal(size=(tokens, experts)) * scale).astype(np.float32))
    x = x.to(tt.bfloat16 if kind == "bf16" else tt.float32)
    if padding:
        x[tokens - padding:] = -float("inf")
    buf = tt.full((tokens, experts + pad), float("nan"), dtype=x.dtype)
    buf[:, :experts] = x
    return x.double().numpy(), buf.cuda()[:, :experts]


def ids_of(tokens, experts, k, seed):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, size=(tokens, k)).astype(np.int32)
    ids[rng.random((tokens, k)) < 0.1] = rng.choice([-1, experts, 2 ** 31 - 1, -2 ** 31])
    return ids


CASES = [
    # tokens, experts, k, type, score, pad, padding tokens
    (1, 1, 1, "f32", 0, 0, 0),
    (1, 32, 4, "bf16", 0, 0, 0),
    (3, 7, 2, "f32", 1, 1, 1),
    (65, 33, 40, "bf16", 1, 3, 7),
    (64, 60, 6, "f32", 0, 4, 0),
    (500, 128, 8, "bf16", 0, 0, 20),
    (1001, 256, 8, "f32", 1, 0, 11),
    (300, 257, 3, "f32", 0, 0, 3),
    (130, 512, 1, "bf16", 1, 8, 0),
    (70, 1000, 2, "bf16", 0, 0, 9),
    (90, 1024, 8, "f32", 0, 0, 0),
    (20000, 16, 2, "f32", 0, 0, 100),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_loss_and_gradient(case):
    tokens, experts, k, kind, score, pad, padding = case
    tt = torch()
    l64, l = logits_of(tokens, experts, kind, 1, pad, padding)
    ids = ids_of(tokens, experts, k, 2)
    loss, counts, slope = mx.balance(l, dev(ids), score=score)
    want = ref.balance(l64, ids, score)
    assert np.array_equal(counts.cpu().numpy(), want[1]) and counts.dtype == tt.int32
    assert np.abs(slope.cpu().numpy() - want[2]).max() <= 2.0 ** -23 * want[2].max()
    assert abs(float(loss) - want[0]) <= (tokens + experts + 8) * 2.0 ** -24 * want[0] + 1e-30
    dloss = tt.tensor(0.37, device="cuda")
    factor = float(np.float32(0.37)) * 1.5
    for add in (None, logits_of(tokens, experts, kind, 3, pad, scale=1e-3)):
        got = mx.balance_bwd(l, slope, score=score, dloss=dloss, scale=1.5, add=None if add is None else add[1])
        g = ref.balance_bwd(l64, want[2], score, factor)
        rows = [ref.scores_of(r, score) for r in l64]
        tol = np.stack([s * rest * (want[2] + (s * want[2]).sum()) for s, rest in rows]) * factor
        tol = tol * (2 * experts + 16) * 2.0 ** -24
        g = g + (0.0 if add is None else add[0])
        tol = tol + 2.0 ** -24 * np.abs(g) + 1e-37
        low, high = g - tol, g + tol
        if kind == "bf16":                                 # rounding keeps the order
            low, high = (bf16_bits_to_f64(oracle.round_bf16_bits(v)) for v in (low, high))
        have = got.double().cpu().numpy()
        assert got.dtype == l.dtype and ((low <= have) & (have <= high)).all()
        if add is not None:
            kept = add[1].clone()
            assert mx.balance_bwd(l, slope, score=score, dloss=dloss, scale=1.5, add=kept, dlogits=kept) is kept
            assert tt.equal(kept, got)


@pytest.mark.parametrize("score", [0, 1])
def test_gradient_against_differences(score):
    """Central differences of the 64-bit loss, the counts held fixed."""
    tt = torch()
    l64, l = logits_of(9, 12, "f32", 5)
    ids = ids_of(9, 12, 3, 6)
    _, _, slope = mx.balance(l, dev(ids), score=score)
    got = mx.balance_bwd(l, slope, score=score).double().cpu().numpy()
    h = 1e-6
    for t in range(9):
        for e in range(12):
            up, down = l64.copy(), l64.copy()
            up[t, e] += h
            down[t, e] -= h
            d = (ref.balance(up, ids, score)[0] - ref.balance(down, ids, score)[0]) / (2 * h)
            assert abs(d - got[t, e]) <= 1e-7


def test_even_and_one_sided():
    tt = torch()
    l = tt.zeros((64, 16), device="cuda")
    even = dev(np.arange(128, dtype=np.int32).reshape(64, 2) % 16)
    assert abs(float(mx.balance(l, even)[0]) - 1.0) < 1e-6
    l[:, 3] = 80.0
    ids = tt.full((64, 2), 3, dtype=tt.int32, device="cuda")
    loss, counts, slope = mx.balance(l, ids)
    assert abs(float(loss) - 16.0) < 1e-5 and int(counts[3]) == 128
    assert float(mx.balance_bwd(l, slope).abs().max()) < 1e-30


def test_masked_experts_and_padding():
    l64, l = logits_of(40, 24, "f32", 7, padding=4)
    l[:, 5] = -float("inf")
    l64[:, 5] = -np.inf
    ids = ids_of(40, 24, 2, 8)
    for score in (0, 1):
        loss, counts, slope = mx.balance(l, dev(ids), score=score)
        assert abs(float(loss) - ref.balance(l64, ids, score)[0]) < 1e-5
        g = mx.balance_bwd(l, slope, score=score)
        assert (g[:, 5] == 0).all() and (g[-4:] == 0).all() and bool(g[:36].abs().sum() > 0)


def test_small_sigmoids_keep_their_proportions():
    l64, l = logits_of(10, 8, "f32", 9)
    ids = ids_of(10, 8, 2, 10)
    want = None
    for shift in (-60.0, -200.0):
        loss, _, slope = mx.balance(l + shift, dev(ids), score=mx.SIGMOID)
        x = (l + shift).double().cpu().numpy()
        assert abs(float(loss) - ref.balance(x, ids, 1)[0]) < 1e-5
        assert np.abs(mx.balance_bwd(l + shift, slope, score=mx.SIGMOID).cpu().numpy() - ref.balance_bwd(x, slope.double().cpu().numpy(), 1)).max() < 1e-6


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite(value):
    """The loss is NaN as the formula says; other rows' gradients are not."""
    tt = torch()
    _, l = logits_of(10, 8, "f32", 11)
    l[4, 2] = value
    ids = ids_of(10, 8, 2, 12)
    loss, counts, slope = mx.balance(l, dev(ids))
    assert tt.isnan(loss) and tt.isfinite(slope).all()
    g = mx.balance_bwd(l, slope)
    assert tt.isnan(g[4]).any() and tt.isfinite(g[tt.arange(10, device="cuda") != 4]).all()


def test_nothing():
    tt = torch()
    none = tt.empty((0, 8), device="cuda")
    loss, counts, slope = mx.balance(none, tt.empty((0, 2), dtype=tt.int32, device="cuda"))
    assert float(loss) == 0 and (counts == 0).all() and (slope == 0).all()
    assert mx.balance_bwd(none, slope).shape == (0, 8)
    # assignments to nobody, tokens with no expert
    _, l = logits_of(5, 8, "f32", 13)
    for x, i in ((l, tt.full((5, 2), -1, dtype=tt.int32, device="cuda")),
                 (tt.full_like(l, -float("inf")), tt.zeros((5, 2), dtype=tt.int32, device="cuda"))):
        loss, counts, slope = mx.balance(x, i)
        assert float(loss) == 0 and (slope == 0).all() and (mx.balance_bwd(x, slope) == 0).all()


def test_with_the_router_and_captured():
    """Router, balance loss and both gradients in one captured graph."""
    tt = torch()
    _, l = logits_of(3000, 64, "bf16", 14, padding=50)
    dw = tt.randn((3000, 4), device="cuda", generator=tt.Generator("cuda").manual_seed(1))

    def step():
        ids, weights = mx.route(l, 4)
        loss, counts, slope = mx.balance(l, ids)
        d = mx.route_bwd(l, ids, dw)
        return loss, counts, mx.balance_bwd(l, slope, scale=0.01, add=d, dlogits=d)

    step()
    tt.cuda.synchronize()
    graph = tt.cuda.CUDAGraph()
    with tt.cuda.graph(graph):
        kept = step()
    for _ in range(3):
        l.mul_(0.9)
        l[-50:] = -float("inf")
        graph.replay()
        tt.cuda.synchronize()
        for a, b in zip(kept, step()):
            assert tt.equal(a, b)


def test_refusals():
    tt = torch()
    _, l = logits_of(5, 8, "f32", 15)
    ids, slope = tt.zeros((5, 2), dtype=tt.int32, device="cuda"), tt.zeros(8, device="cuda")
    for bad in (lambda: mx.balance(l, ids.long()), lambda: mx.balance(l, ids[:4]), lambda: mx.balance(l.half(), ids),
                lambda: mx.balance(l, ids, score=2), lambda: mx.balance(l.cpu(), ids), lambda: mx.balance(l, ids[0]),
                lambda: mx.balance(l, ids, counts=slope), lambda: mx.balance_bwd(l, slope[:7]),
                lambda: mx.balance_bwd(l, slope, add=l.bfloat16()), lambda: mx.balance_bwd(l, slope, scale=float("nan")),
                lambda: mx.balance_bwd(l, slope, dloss=slope), lambda: mx.balance_bwd(l, slope, dlogits=l[:4]),
                lambda: mx.balance(l, ids, workspace=tt.empty(3, dtype=tt.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError, mx.MXError)):
            bad()


@pytest.mark.parametrize("experts", [5, 32, 60, 200, 500, 1024])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rows_with_a_single_expert_left(kind, experts):
    """Token t has a score for expert t alone: each has one, wherever it lies."""
    tt = torch()
    tokens = experts + 3
    l = tt.full((tokens, experts), -float("inf"), dtype=tt.bfloat16 if kind == "bf16" else tt.float32, device="cuda")
    at = tt.arange(experts, device="cuda")
    l[at, at] = 0.5
    ids = tt.full((tokens, 1), -1, dtype=tt.int32, device="cuda")
    ids[:experts, 0] = at.int()
    loss, counts, slope = mx.balance(l, ids)
    want = ref.balance(l.double().cpu().numpy(), ids.cpu().numpy(), 0)
    assert (counts == 1).all()
    assert np.abs(slope.cpu().numpy() - want[2]).max() <= 2.0 ** -23 * want[2].max()
    assert abs(float(loss) - want[0]) <= (tokens + experts + 8) * 2.0 ** -24 * want[0]
    assert (mx.balance_bwd(l, slope) == 0).all()           # the only score of a row is 1 whatever its logit


@pytest.mark.parametrize("experts", [60, 128, 250])
def test_many_tokens(experts):
    """As many tokens as the backward pass takes with fewer lanes a row, and one fewer."""
    tt = torch()
    for tokens in (8191, 8192):
        l64, l = logits_of(tokens, experts, "f32", 21, padding=5)
        ids = ids_of(tokens, experts, 2, 22)
        loss, counts, slope = mx.balance(l, dev(ids), score=mx.SIGMOID)
        want = ref.balance(l64, ids, 1)
        assert np.array_equal(counts.cpu().numpy(), want[1])
        assert abs(float(loss) - want[0]) <= (tokens + experts + 8) * 2.0 ** -24 * want[0]
        got = mx.balance_bwd(l, slope, score=mx.SIGMOID).double().cpu().numpy()
        g = ref.balance_bwd(l64, want[2], 1)
        s = np.where(np.isneginf(l64), 0.0, 1.0 / (1.0 + np.exp(-l64)))
        s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
        tol = s * (want[2] + (s * want[2]).sum(1, keepdims=True)) * (2 * experts + 16) * 2.0 ** -24
        assert (np.abs(got - g) <= tol + 2.0 ** -24 * np.abs(g) + 1e-37).all()


def test_two_streams_at_once():
    tt = torch()
    calls = []
    for seed in (31, 32):
        _, l = logits_of(4000, 100, "bf16", seed)
        calls.append((l, dev(ids_of(4000, 100, 4, seed)), tt.cuda.Stream()))
    want = [mx.balance(l, ids) for l, ids, _ in calls]
    tt.cuda.synchronize()
    got = []
    for _ in range(5):
        for l, ids, stream in calls:
            with tt.cuda.stream(stream):
                got.append(mx.balance(l, ids))
    tt.cuda.synchronize()
    for i, have in enumerate(got):
        assert all(tt.equal(a, b) for a, b in zip(have, want[i % 2]))
