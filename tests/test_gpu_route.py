"""GPU: routing, its gradient and the dispatch plan against the 64-bit
definitions of oracle/moe.py.

Tolerances.  A score is exp or 1 / (1 + exp) of an fp32 difference l - top:
that difference carries half an ulp, which for |l - top| <= 32 is 2e-6
relative in the exponential; exp, the sum of up to 1024 terms (a tree of at
most 20 levels, 1.2e-6), the division and the scale add less than 2e-6.  So
weights are held to 6e-6 relative (plus the smallest normal number, where fp32
rounds coarser).  A logit's gradient is a product of weights with a
difference of terms of size |dw|: 2e-5 of scale * max|dw| * its score.  A bf16
gradient adds its rounding, 2^-8 relative.
Keys with a bias, and sums of two, carry up to 1e-6 absolute: rows whose 64-bit
keys come closer than that may be ordered either way and are checked for a
choice that is right to 1e-6; all others, and every choice between logits
themselves, must be equal."""
import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from oracle import moe
from gpu_util import dev, host, torch

pytestmark = pytest.mark.gpu
INF = float("inf")
W_RTOL, KEY_TOL, D_TOL = 6e-6, 1e-6, 2e-5


def logits_of(t, e, dtype, seed, spread=2.0):
    """fp32 values representable in dtype, with padding rows, masked experts,
    a row of the type's lowest value and ties."""
    tt = torch()
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (t, e)).astype(np.float32)
    if t > 4:
        x[1] = -INF                                        # nothing left
        x[2, rng.permutation(e)[:max(0, e - 2)]] = -INF    # two experts left
        x[3] = float(tt.finfo(dtype).min)                  # masked by the lowest value
        x[4] = 0.5                                         # all equal
    if t > 6:
        x[5, ::2] = float(tt.finfo(dtype).min)
        x[6] = -200.0 - np.arange(e) % 7                   # scores that underflow
    return tt.from_numpy(x).to(dtype)


def placed(x, pad):
    """x on the device, its rows pad elements apart from contiguous, starting
    one element into its buffer when pad is odd."""
    tt = torch()
    t, e = x.shape
    buf = tt.full((t * (e + pad) + 1,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[pad % 2:pad % 2 + t * (e + pad)].view(t, e + pad)[:, :e]
    view.copy_(x)
    return view


CASES = [
    # tokens, experts, k, dtype, score, bias, groups, top_groups, best, renorm, scale, pad
    (1, 32, 4, "bf16", 0, False, 1, 1, 1, True, 1.0, 0),
    (7, 32, 4, "bf16", 0, False, 1, 1, 1, False, 1.0, 0),
    (9, 1, 1, "f32", 0, False, 1, 1, 1, True, 1.0, 0),
    (9, 2, 1, "f32", 1, True, 2, 1, 1, True, 1.0, 1),
    (17, 5, 3, "f32", 1, False, 1, 1, 1, False, 2.5, 3),
    (33, 8, 8, "bf16", 1, True, 1, 1, 1, True, 1.0, 1),
    (65, 31, 6, "f32", 0, True, 1, 1, 1, False, 1.0, 0),
    (67, 33, 9, "bf16", 0, False, 1, 1, 1, True, 1.0, 5),
    (40, 60, 6, "f32", 0, False, 1, 1, 1, False, 1.0, 4),
    (40, 60, 4, "f32", 0, False, 5, 2, 1, True, 1.0, 0),
    (129, 64, 16, "f32", 1, True, 8, 4, 2, True, 2.5, 0),
    (50, 64, 20, "bf16", 1, False, 1, 1, 1, True, 1.0, 0),
    (50, 100, 7, "bf16", 0, False, 10, 3, 2, False, 1.0, 0),
    (31, 128, 8, "f32", 1, False, 1, 1, 1, True, 1.0, 8),
    (31, 129, 2, "f32", 0, True, 3, 2, 2, True, 1.0, 0),
    (257, 256, 8, "f32", 1, True, 8, 4, 2, True, 2.5, 0),
    (70, 256, 8, "bf16", 1, True, 8, 3, 1, True, 2.5, 4),
    (21, 257, 10, "f32", 0, False, 1, 1, 1, False, 1.0, 0),
    (21, 384, 32, "f32", 1, True, 1, 1, 1, True, 1.0, 0),
    (13, 512, 17, "bf16", 0, False, 64, 9, 2, True, 1.0, 0),
    (13, 513, 4, "f32", 0, False, 1, 1, 1, True, 1.0, 1),
    (11, 1000, 32, "f32", 1, True, 4, 2, 2, False, 1.0, 0),
    (11, 1024, 12, "bf16", 0, True, 16, 5, 2, True, 1.0, 0),
    (19, 300, 6, "f32", 1, False, 1, 1, 1, True, 1.0, 0),
    (19, 384, 8, "bf16", 0, True, 8, 3, 2, False, 1.0, 8),
    (19, 512, 4, "f32", 0, False, 1, 1, 1, False, 1.0, 2),
    (10, 1024, 8, "bf16", 1, True, 1, 1, 1, True, 1.0, 0),
    (10, 777, 5, "f32", 0, False, 7, 3, 1, True, 1.0, 0),
    (23, 128, 1, "bf16", 1, False, 1, 1, 1, False, 1.0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_route_and_gradient(case):
    t, e, k, dtype, score, with_bias, groups, top_groups, best, renorm, scale, pad = case
    tt = torch()
    dtype = tt.bfloat16 if dtype == "bf16" else tt.float32
    x = logits_of(t, e, dtype, seed=e * 1000 + t)
    rng = np.random.default_rng(e + t)
    bias = (0.001 * rng.integers(-60, 61, e)).astype(np.float32) if with_bias else None
    l = placed(x, pad)
    kw = dict(score=score, renorm=renorm, scale=scale)
    ids, weights = mx.route(l, k, bias=None if bias is None else dev(bias), groups=groups, top_groups=top_groups,
                            group_best=best, **kw)
    dw = rng.normal(size=(t, k)).astype(np.float32)
    dl = mx.route_bwd(l, ids, dev(dw), **kw)
    assert dl.dtype == dtype and ids.dtype == tt.int32
    ids, weights, dl = host(ids), host(weights), dl.float().cpu().numpy()
    x64 = x.double().numpy()
    by_score = with_bias or (groups > 1 and best > 1)
    for r in range(t):
        want, _, margin = moe.route_row(x64[r], k, score, bias, groups, top_groups, best, renorm, scale)
        if not by_score or margin > KEY_TOL:
            assert ids[r].tolist() == want.tolist(), (r, margin)
        else:
            key = moe.keys(x64[r], bias, score, groups, best)
            held = ids[r][ids[r] >= 0]
            assert len(set(held)) == len(held) and ((want < 0) == (ids[r] < 0)).all()
            assert (np.abs(key[ids[r]] - key[want]) <= KEY_TOL)[want >= 0].all() or groups > 1
        w = moe.weights_of(x64[r], ids[r], score, renorm, scale)
        assert np.allclose(weights[r], w, rtol=W_RTOL, atol=1.2e-38), (r, weights[r], w)
        d = moe.route_bwd_row(x64[r], ids[r], dw[r], score, renorm, scale)
        s = np.zeros(e)
        there = ids[r] >= 0
        s[ids[r][there]] = 1.0
        if score == mx.SOFTMAX and not renorm:
            s = moe.scores(x64[r], score)
        tol = D_TOL * scale * np.abs(dw[r]).max() * s + (2.0 ** -8 * np.abs(d) if dtype == tt.bfloat16 else 0) + 1.2e-38
        assert (np.abs(dl[r] - d) <= tol).all(), (r, np.abs(dl[r] - d).max())


def near_tie_faults(key, ids, groups, top_groups, best, key_tol):
    """Rows [tokens] whose ids are not a choice that errors of key_tol in each
    key explain: distinct, in the order of the keys, from few enough groups,
    none of them clearly behind a group left out, and no expert of a group
    that is clearly kept clearly ahead of a chosen one.  A group's score, the
    sum of two keys below 2, is rounded once more (2^-23).  Two values are
    clearly apart beyond both their errors."""
    t, e = key.shape
    k, size = ids.shape[1], e // groups
    rows = np.arange(t)[:, None]
    chosen = np.zeros((t, e), bool)
    chosen[rows, ids] = True
    bad = (ids < 0).any(1) | (chosen.sum(1) != k)
    mine = key[rows, ids]
    bad |= (mine[:, :-1] < mine[:, 1:] - 2 * key_tol).any(1)
    sure = np.ones((t, groups), bool)
    if top_groups < groups:
        of = np.sort(key.reshape(t, groups, size), axis=2)[:, :, -best:].sum(2)
        far = 2 * (best * key_tol + 2.0 ** -23)
        down = -np.sort(-of, axis=1)
        sure = of > down[:, top_groups, None] + far        # ahead of the first one left out
        used = chosen.reshape(t, groups, size).any(2)
        bad |= (used & (of < down[:, top_groups - 1, None] - far)).any(1)
        bad |= (used | sure).sum(1) > top_groups
    missed = np.where(np.repeat(sure, size, axis=1) & ~chosen, key, -INF).max(1)
    return bad | (missed > mine.min(1) + 2 * key_tol)


def near_tie_logits(tokens, experts, seed):
    """Logits and a bias whose sigmoid keys crowd within 5e-7 around a few
    values, and their 64-bit keys."""
    rng = np.random.default_rng(seed)
    bias = (0.001 * rng.integers(-60, 61, experts)).astype(np.float32)
    key = 0.25 + 0.1 * rng.integers(0, 6, (tokens, experts)) + rng.uniform(-5e-7, 5e-7, (tokens, experts))
    s = key - bias.astype(np.float64)
    x = np.log(s / (1 - s)).astype(np.float32)
    return x, bias, 1 / (1 + np.exp(-x.astype(np.float64))) + bias.astype(np.float64)


# The error of a key s + b, s = 1 / (1 + e^-x): the product x log2(e) and its constant are off by 7.3e-8 |x|, the
# exponential by 1 ulp (2^-23); both reach s by the factor s (1 - s), so at most 0.224 * 7.3e-8 + 2^-25 = 4.7e-8.  The
# sum 1 + e^-x (2^-24), the reciprocal (1 ulp, 2^-23) and the sum with b, below 2 (2^-24), add 2.4e-7.
SIGMOID_KEY_TOL = 3e-7


@pytest.mark.parametrize("tokens", [300, 8200])
@pytest.mark.parametrize("experts,groups,top_groups,best,k", [(64, 8, 4, 2, 8), (64, 8, 4, 1, 6), (256, 8, 4, 2, 8),
                                                              (60, 5, 2, 2, 4), (250, 10, 3, 2, 7), (32, 1, 1, 1, 4),
                                                              (512, 64, 9, 2, 12), (1024, 16, 5, 2, 8)])
def test_near_ties(experts, groups, top_groups, best, k, tokens):
    x, bias, key = near_tie_logits(tokens, experts, experts + tokens)
    ids = host(mx.route(dev(x), k, score=mx.SIGMOID, bias=dev(bias), groups=groups, top_groups=top_groups,
                        group_best=best)[0])
    assert not near_tie_faults(key, ids, groups, top_groups, best, SIGMOID_KEY_TOL).any()


def test_equal_keys_go_to_the_lowest_index():
    tt = torch()
    rng = np.random.default_rng(0)
    x = rng.integers(-2, 3, (64, 96)).astype(np.float32)       # many equal logits, -0 among the zeros
    x[x == 0] *= np.where(rng.random((x == 0).sum()) < 0.5, -1, 1)
    for score in (mx.SOFTMAX, mx.SIGMOID):
        ids, _ = mx.route(tt.from_numpy(x).cuda(), 8, score=score)
        assert host(ids).tolist() == np.argsort(-x, axis=1, kind="stable")[:, :8].tolist()
        # equal scores and equal biases give equal keys
        ids, _ = mx.route(tt.from_numpy(x).cuda(), 8, score=score, bias=tt.zeros(96, device="cuda"))
        assert host(ids).tolist() == np.argsort(-x, axis=1, kind="stable")[:, :8].tolist()
    # equal groups: the lower ones
    same = tt.zeros((3, 32), device="cuda")
    ids, _ = mx.route(same, 6, groups=8, top_groups=2, group_best=2, score=mx.SIGMOID)
    assert host(ids).tolist() == [[0, 1, 2, 3, 4, 5]] * 3


def test_nan_and_infinite_logits():
    tt = torch()
    x = tt.randn((5, 32), device="cuda", generator=tt.Generator("cuda").manual_seed(1))
    x[1, 7] = float("nan")
    x[2, 9] = INF
    x[3, 3] = -INF
    x[4] = float("nan")
    for score in (mx.SOFTMAX, mx.SIGMOID):
        for bias in (None, tt.zeros(32, device="cuda")):
            for renorm in (True, False):
                ids, w = (host(v) for v in mx.route(x, 4, score=score, bias=bias, renorm=renorm))
                for row in ids:
                    assert len(set(row)) == 4 and (row >= 0).all() and (row < 32).all()
                assert 3 not in ids[3] and ids[4].tolist() == [0, 1, 2, 3] and np.isnan(w[4]).all()
                assert np.isfinite(w[0]).all() and np.isfinite(w[3]).all()
                if score == mx.SIGMOID or bias is None:
                    assert 7 not in ids[1] and ids[2][0] == 9
                if score == mx.SIGMOID:
                    assert np.isfinite(w[1]).all() and np.isfinite(w[2]).all()
                elif not renorm:
                    assert np.isnan(w[1]).all() and np.isnan(w[2]).all()
                g = host(mx.route_bwd(x, dev(ids), tt.ones((5, 4), device="cuda"), score=score, renorm=renorm))
                assert np.isfinite(g[0]).all() and np.isfinite(g[3]).all()
    # biases of the lowest value keep experts for last, -inf ones keep them out
    low = tt.zeros(32, device="cuda")
    low[:30] = tt.finfo(tt.float32).min
    x = tt.randn((9, 32), device="cuda", generator=tt.Generator("cuda").manual_seed(2))
    for groups in (1, 8):
        ids = host(mx.route(x, 4, score=mx.SIGMOID, bias=low, groups=groups, top_groups=max(1, groups // 4),
                            group_best=1 + (groups > 1))[0])
        assert (np.sort(ids[:, :2], axis=1) == [30, 31]).all() and (ids >= 0).all()
        out = tt.where(low < 0, -INF, low)
        ids = host(mx.route(x, 4, score=mx.SIGMOID, bias=out, groups=groups, top_groups=max(1, groups // 4),
                            group_best=1 + (groups > 1))[0])
        assert (np.sort(ids[:, :2], axis=1) == [30, 31]).all() and (ids[:, 2:] == -1).all()


@pytest.mark.parametrize("tokens", [40, 8200])
@pytest.mark.parametrize("experts,groups,best", [(64, 8, 2), (64, 16, 2), (60, 5, 2), (250, 10, 2), (256, 8, 2), (256, 8, 1),
                                                 (512, 64, 2), (1024, 8, 2)])
def test_nan_keys_add_nothing_to_their_groups(tokens, experts, groups, best):
    """NaN logits in every place of a group, under sigmoid scores with a bias
    of their own; rows whose 64-bit keys or group sums come closer than fp32
    can order are left out."""
    rng = np.random.default_rng(experts + groups)
    x = rng.normal(size=(tokens, experts)).astype(np.float32)
    x[rng.random(x.shape) < np.array([0.1, 0.5, 0.9])[np.arange(tokens) % 3, None]] = float("nan")
    bias = (0.01 * rng.integers(-9, 10, experts)).astype(np.float32)
    top = max(1, groups // 2)
    k = min(8, top * (experts // groups))
    ids = host(mx.route(dev(x), k, score=mx.SIGMOID, bias=dev(bias), groups=groups, top_groups=top, group_best=best)[0])
    tested = 0
    for r in range(40):
        want, _, margin = moe.route_row(x[r].astype(np.float64), k, mx.SIGMOID, bias, groups, top, best)
        if margin > KEY_TOL:
            tested += 1
            assert ids[r].tolist() == want.tolist(), r
    assert tested >= 30


@pytest.mark.parametrize("tokens", [9, 8200])
@pytest.mark.parametrize("experts,groups,k", [(32, 1, 8), (64, 8, 4), (60, 5, 3), (256, 8, 8), (512, 1, 12)])
def test_a_nan_score_does_not_bring_back_what_the_bias_takes_away(tokens, experts, groups, k):
    """Rows with NaN and +inf logits (whose softmax is NaN throughout) under a
    bias of -inf at a third of the experts: those are never chosen."""
    rng = np.random.default_rng(experts)
    x = rng.normal(size=(tokens, experts)).astype(np.float32)
    x[::3, rng.permutation(experts)[:experts // 2]] = float("nan")
    x[1::3, 5] = INF
    bias = (0.01 * rng.integers(-9, 10, experts)).astype(np.float32)
    gone = np.arange(experts) % 3 == 0
    bias[gone] = -INF
    for score in (mx.SOFTMAX, mx.SIGMOID):
        for best in ((1, 2) if groups > 1 else (1,)):
            kw = dict(score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2), group_best=best)
            ids = host(mx.route(dev(x), k, **dict(kw, bias=dev(bias)))[0])
            assert not gone[ids[ids >= 0]].any()
            for r in range(9):
                want, _, margin = moe.route_row(x[r].astype(np.float64), k, **kw)
                if margin > KEY_TOL:
                    assert ids[r].tolist() == want.tolist()


def test_gradient_ignores_ids_out_of_range():
    tt = torch()
    x = tt.randn((4, 24), device="cuda", generator=tt.Generator("cuda").manual_seed(3))
    ids = np.array([[0, 5], [-1, 2], [24, 3], [2 ** 31 - 1, -2 ** 31]], dtype=np.int32)
    dw = np.ones((4, 2), dtype=np.float32)
    for score in (0, 1):
        for renorm in (False, True):
            got = host(mx.route_bwd(x, dev(ids), dev(dw), score=score, renorm=renorm))
            for r in range(4):
                want = moe.route_bwd_row(x[r].double().cpu().numpy(), ids[r], dw[r], score, renorm)
                assert np.allclose(got[r], want, rtol=0, atol=D_TOL)


@pytest.mark.parametrize("tokens", [40, 8200])
@pytest.mark.parametrize("experts", [24, 60, 128, 256, 500, 1024])
def test_dense_gradient_entries(tokens, experts):
    """Every entry that was not chosen, over that of an expert with the row's
    largest logit, is exp of an integer difference, which fp32 holds exactly:
    the exponential (1 ulp, 2^-23, and the rounding that ends it, 2^-24) and
    the two products of each entry (2^-24 each) remain, 7 * 2^-24; 8 leaves
    room for the products' own squares."""
    rng = np.random.default_rng(experts)
    x = -rng.integers(0, 81, (tokens, experts)).astype(np.float32)
    x[:, :3] = 0.0                                         # two chosen, one to compare with
    ids = np.tile(np.array([[0, 1]], np.int32), (tokens, 1))
    for shift in (0.0, 7.0, -1000.0):
        dl = host(mx.route_bwd(dev(x + np.float32(shift)), dev(ids), dev(np.ones((tokens, 2), np.float32)),
                               renorm=False)).astype(np.float64)
        want = np.exp(x[:, 3:].astype(np.float64))
        assert (np.abs(dl[:, 3:] / dl[:, 2:3] - want) <= 8 * 2.0 ** -24 * want).all()


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """The kernel's gradient against central differences of the 64-bit
    weights: their own error is below 1e-8 at this step."""
    tt = torch()
    rng = np.random.default_rng(11)
    x = rng.normal(0, 1.5, (3, 20)).astype(np.float32)
    dw = rng.normal(size=(3, 5)).astype(np.float32)
    ids, _ = mx.route(dev(x), 5, score=score, renorm=renorm)
    got = host(mx.route_bwd(dev(x), ids, dev(dw), score=score, renorm=renorm))
    ids = host(ids)
    for r in range(3):
        for e in range(20):
            up, down = x[r].astype(np.float64), x[r].astype(np.float64)
            up[e] += 1e-6
            down[e] -= 1e-6
            d = (moe.weights_of(up, ids[r], score, renorm, 1.0) - moe.weights_of(down, ids[r], score, renorm, 1.0)) / 2e-6
            assert abs((d * dw[r]).sum() - got[r, e]) <= D_TOL * np.abs(dw[r]).max() + 1e-8


def test_many_rows():
    """More workgroups than are resident, against a vectorised 64-bit form."""
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(5)
    x = tt.randn((70001, 160), device="cuda", generator=gen)
    ids, w = mx.route(x, 6, scale=2.0)
    s = x.double().sort(dim=1, descending=True, stable=True)
    assert tt.equal(ids.long(), s.indices[:, :6])
    p = tt.softmax(s.values[:, :6], 1) * 2.0
    assert ((w - p).abs() <= W_RTOL * p).all()
    dw = tt.randn((70001, 6), device="cuda", generator=gen)
    dl = mx.route_bwd(x, ids, dw, scale=2.0)
    want = tt.zeros(x.shape, device="cuda", dtype=tt.float64)
    want.scatter_(1, ids.long(), p * (dw - (dw * p / 2.0).sum(1, keepdim=True)))
    assert (dl - want).abs().max() <= D_TOL * 2.0 * dw.abs().max()


@pytest.mark.parametrize("experts,k", [(32, 8), (61, 3), (64, 4), (64, 7), (100, 5), (128, 2), (200, 4), (256, 8), (256, 1),
                                       (300, 5), (512, 8), (512, 2), (516, 4), (1024, 8), (1000, 3)])
@pytest.mark.parametrize("groups,best", [(1, 1), (4, 2)])
def test_many_tokens(experts, k, groups, best):
    """The variants for many tokens, with a bias, groups and masked experts,
    against a vectorised 64-bit form; rows that fp32 cannot order are left
    out, the others must agree."""
    tt = torch()
    if experts % groups:
        groups, best = 1, 1
    gen = tt.Generator("cuda").manual_seed(experts + k)
    x = tt.randn((8200, experts), device="cuda", generator=gen)
    x[::7, ::3] = -INF
    x[5] = -INF
    bias = 0.001 * tt.randint(-60, 61, (experts,), device="cuda", generator=gen)
    top_groups = max(1, groups // 2)
    k = min(k, top_groups * experts // groups)
    ids, w = mx.route(x, k, score=mx.SIGMOID, bias=bias, groups=groups, top_groups=top_groups, group_best=best)
    key = tt.where(x == -INF, -INF, tt.sigmoid(x.double()) + bias.double())
    sure = tt.ones(8200, dtype=tt.bool, device="cuda")

    def apart(v, n):
        v = v.sort(dim=1, descending=True).values[:, :n + 1]
        d = v[:, :-1] - v[:, 1:]
        return ((d > KEY_TOL) | tt.isnan(d) | (v[:, :-1] == -INF)).all(1)

    if groups > 1:
        part = key.view(8200, groups, -1).sort(dim=2, descending=True).values[:, :, :best]
        of = tt.where(part == -INF, 0.0, part).sum(2)
        of = tt.where(part[:, :, 0] == -INF, -INF, of)
        sure &= apart(of, top_groups)
        drop = tt.ones_like(of, dtype=tt.bool)
        drop.scatter_(1, of.sort(dim=1, descending=True, stable=True).indices[:, :top_groups], False)
        key = tt.where(drop[:, :, None], -INF, key.view(8200, groups, -1)).view(8200, experts)
    sure &= apart(key, k)
    best_k = key.sort(dim=1, descending=True, stable=True)
    want = tt.where(best_k.values[:, :k] == -INF, -1, best_k.indices[:, :k])
    assert sure.float().mean() > 0.9 and tt.equal(ids[sure].long(), want[sure])
    s = tt.where(ids < 0, 0.0, tt.sigmoid(x.double()).gather(1, ids.long().clamp(min=0)))
    p = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    assert ((w - p).abs() <= W_RTOL * p).all()
    dw = tt.randn((8200, k), device="cuda", generator=gen)
    dl = mx.route_bwd(x, ids, dw, score=mx.SIGMOID)
    g = tt.where(ids < 0, 0.0, dw.double())
    d = p * (1 - s) * (g - (g * p).sum(1, keepdim=True))
    want = tt.zeros((8200, experts), device="cuda", dtype=tt.float64).scatter_add_(1, ids.long().clamp(min=0), d)
    assert (dl - want).abs().max() <= D_TOL * dw.abs().max()


@pytest.mark.parametrize("experts,groups,top_groups,k", [(192, 64, 20, 8), (255, 51, 7, 6), (250, 50, 50, 3),
                                                         (256, 64, 9, 8), (96, 48, 3, 4), (66, 33, 2, 4),
                                                         (48, 12, 5, 7), (256, 2, 1, 5), (448, 64, 11, 8),
                                                         (512, 64, 30, 3), (960, 64, 5, 8), (1023, 33, 4, 5)])
def test_many_and_few_tokens_agree(experts, groups, top_groups, k):
    """The variants for many and for few tokens choose alike, bit for bit, up
    to the largest number of groups."""
    tt = torch()
    x = tt.randn((8300, experts), device="cuda", generator=tt.Generator("cuda").manual_seed(groups))
    x[::5, ::2] = -INF
    bias = tt.linspace(-0.05, 0.05, experts, device="cuda")
    for best in (1, 2):
        kw = dict(score=mx.SIGMOID, bias=bias, groups=groups, top_groups=top_groups, group_best=best)
        ids, w = mx.route(x, k, **kw)
        parts = [mx.route(part, k, **kw) for part in (x[:4000], x[4000:])]
        assert tt.equal(ids, tt.cat([p[0] for p in parts])) and tt.equal(w, tt.cat([p[1] for p in parts]))
        of = ids.clamp(min=0) // (experts // groups)
        taken = tt.zeros((8300, groups), dtype=tt.bool, device="cuda").scatter_(1, of.long(), ids >= 0)
        assert (taken.sum(1) <= top_groups).all()


@pytest.mark.parametrize("tokens,k", [(0, 2), (1, 1), (1, 4), (9, 7), (63, 1), (16, 4), (65, 1), (341, 3), (1025, 1),
                                      (700, 3), (5000, 4), (40000, 8), (100001, 8)])
@pytest.mark.parametrize("experts", [1, 3, 32, 33, 256, 1024])
def test_plan(tokens, k, experts):
    rng = np.random.default_rng(tokens * 1000 + experts)
    p = np.arange(1, experts + 1) ** -1.1
    ids = rng.choice(experts, size=(tokens, k), p=p / p.sum()).astype(np.int32)
    drop = rng.random(ids.shape) < 0.05
    ids[drop] = rng.choice([-1, -7, experts, 2 ** 31 - 1], size=int(drop.sum()))
    offsets, row_index, slot = (host(v) for v in mx.route_plan(dev(ids), experts))
    flat = ids.reshape(-1)
    none = (flat < 0) | (flat >= experts)
    order = np.argsort(np.where(none, experts, flat), kind="stable")
    assert offsets.tolist() == np.concatenate([[0], np.cumsum(np.bincount(flat[~none], minlength=experts))]).tolist()
    assert np.array_equal(row_index, order // k)
    want = np.empty(flat.size, np.int64)
    want[order] = np.arange(flat.size)
    assert np.array_equal(slot.reshape(-1), np.where(none, -1, want))
    if tokens <= 1000:
        for a, b in zip((offsets, row_index, slot), moe.route_plan(ids, experts)):
            assert np.array_equal(a, b)


def test_no_tokens():
    tt = torch()
    x = tt.zeros((0, 32), device="cuda")
    ids, w = mx.route(x, 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert mx.route_bwd(x, ids, w).shape == (0, 32)


@pytest.mark.parametrize("tokens", [5, 9000])
@pytest.mark.parametrize("experts", [64, 100, 256])
def test_bias_off_its_alignment(tokens, experts):
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(experts)
    x = tt.randn((tokens, experts), device="cuda", generator=gen)
    bias = 0.1 * tt.randn(experts + 3, device="cuda", generator=gen)
    for at in (1, 2, 3):
        part = bias[at:at + experts]
        assert part.data_ptr() % 16
        for score in (0, 1):
            a, b = (mx.route(x, 6, score=score, bias=v) for v in (part, part.clone()))
            assert tt.equal(a[0], b[0]) and tt.equal(a[1], b[1])


def test_plan_of_one_expert_and_of_none():
    for value in (-1, 0, 31):
        ids = np.full((3000, 2), value, dtype=np.int32)
        offsets, row_index, slot = (host(v) for v in mx.route_plan(dev(ids), 32))
        assert np.array_equal(row_index, np.arange(6000) // 2)
        assert np.array_equal(slot.reshape(-1), np.arange(6000) if value >= 0 else np.full(6000, -1))
        assert offsets.tolist() == [6000 if 0 <= value < e else 0 for e in range(33)]


def test_other_stream_and_graph():
    """On a stream of its own, and captured once and replayed with other
    inputs in place."""
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(8)
    x = tt.randn((300, 64), device="cuda", generator=gen)
    dw = tt.randn((300, 4), device="cuda", generator=gen)
    tt.cuda.synchronize()
    side = tt.cuda.Stream()

    def step():
        ids, w = mx.route(x, 4)
        return (ids, w, mx.route_bwd(x, ids, dw)) + mx.route_plan(ids, 64)

    with tt.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(got, step()):
        assert tt.equal(a, b)
    graph = tt.cuda.CUDAGraph()
    with tt.cuda.graph(graph):
        held = step()
    for n in range(3):
        x.copy_(tt.randn((300, 64), device="cuda", generator=gen))
        graph.replay()
        tt.cuda.synchronize()
        for a, b in zip(held, step()):
            assert tt.equal(a, b), n


def test_refusals():
    tt = torch()
    x = tt.zeros((4, 32), device="cuda")
    ids = tt.zeros((4, 2), dtype=tt.int32, device="cuda")
    dw = tt.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError):
        mx.route(x.cpu(), 2)
    with pytest.raises(TypeError):
        mx.route(x.half(), 2)
    with pytest.raises(ValueError):
        mx.route(x.t(), 2)                                 # rows not contiguous
    with pytest.raises(ValueError):
        mx.route(x[:1].expand(4, 32), 2)                   # rows on top of each other
    with pytest.raises(ValueError):
        mx.route(x, 2, bias=tt.zeros(31, device="cuda"))
    with pytest.raises(TypeError):
        mx.route(x, 2, ids=tt.zeros((4, 2), dtype=tt.int64, device="cuda"))
    for bad in (dict(top_k=33), dict(top_k=2, groups=5), dict(top_k=2, groups=4, top_groups=5),
                dict(top_k=9, groups=4, top_groups=1), dict(top_k=2, group_best=3), dict(top_k=2, score=7),
                dict(top_k=2, scale=INF)):
        with pytest.raises(mx.MXError):
            mx.route(x, **bad)
    with pytest.raises(TypeError):
        mx.route_bwd(x, ids.long(), dw)
    with pytest.raises(ValueError):
        mx.route_bwd(x, ids, dw[:, :1].contiguous())
    with pytest.raises(TypeError):
        mx.route_bwd(x, ids, dw, dlogits=tt.zeros((4, 32), dtype=tt.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mx.route_plan(ids.long(), 32)
    with pytest.raises(mx.MXError):
        mx.route_plan(ids, 1025)
    with pytest.raises(ValueError):
        mx.route_plan(tt.zeros((65536, 2), dtype=tt.int32, device="cuda"), 32,
                      workspace=tt.zeros(8, dtype=tt.uint8, device="cuda"))
