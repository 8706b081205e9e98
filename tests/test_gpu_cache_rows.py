"""GPU: the kernel for many rows of a sequence, at sizes that a test can check.
It is chosen for few rows too where the tables hold many tokens, so these are as
wide as that takes (none of their further columns is looked at).  Compared, and
with the tolerances, as in test_gpu_cache.py."""
import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from oracle import cache as ref
from gpu_util import dev, torch
from test_gpu_cache import Setup, layouts, values
from test_gpu_cache_limits import BYTES, fill, same

pytestmark = pytest.mark.gpu

HEADS = [(32, "bf16", False), (32, "bf16", True), (32, "f32", True), (96, "bf16", True), (64, "bf16", True), (64, "f32", False), (96, "bf16", False), (96, "f32", True), (128, "bf16", False),
         (128, "bf16", True), (128, "f32", False), (160, "bf16", True), (192, "f32", True), (224, "bf16", False),
         (256, "bf16", False), (256, "bf16", True), (256, "f32", False)]
IDS = ["%d-%s-%s" % h for h in HEADS]


class Rows(Setup):
    """More than 96 rows of a head in one sequence, tables for 2^23 tokens."""

    def __init__(self, lengths, heads, group, dim, page, kind="bf16", rht=False, queries=None, **kw):
        assert sum(queries) * group > 96 and sum(queries) * heads * group >= 128
        super().__init__(lengths, heads, group, dim, page, kind, rht, queries=queries, extra_columns=2 ** 23 // page, **kw)


@pytest.mark.parametrize("dim, kind, rht", HEADS, ids=IDS)
@pytest.mark.parametrize("window, causal", [(0, True), (33, True), (100, True), (0, False)])
def test_head_sizes(dim, kind, rht, window, causal):
    s = Rows([150, 0, 70, 40], 2, 2, dim, 16, kind, rht, queries=[70, 3, 65, 1], seed=401)
    sinks = np.random.default_rng(6).normal(size=4).astype(np.float32)
    args = dict(sinks=dev(sinks), window=window, causal=causal)
    s.check(s.call(max_queries=70, **args), s.want(sinks=sinks, window=window, causal=causal))
    s.check(s.call(window=window, causal=causal), s.want(window=window, causal=causal))


@pytest.mark.parametrize("group, queries", [(1, [128]), (1, [129, 1]), (3, [70, 40]), (5, [33, 0, 10]), (7, [200]), (17, [9, 9]),
                                            (40, [4, 5]), (128, [3]), (130, [2, 1])])
@pytest.mark.parametrize("window", [0, 50])
def test_groups(group, queries, window):
    """Tiles of 128 rows by groups that do not divide them, and groups past them."""
    lengths = [n + 37 * (i + 1) for i, n in enumerate(queries)]
    s = Rows(lengths, 2, group, 64, 32, queries=queries, seed=402)
    s.check(s.call(window=window), s.want(window=window))


@pytest.mark.parametrize("dim, kind, rht", HEADS, ids=IDS)
@pytest.mark.parametrize("lengths, queries, window", [([6000], [33], 0), ([2500, 1400], [60, 130], 1300), ([1100, 20], [130, 20], 0)])
def test_cut_segments(dim, kind, rht, lengths, queries, window):
    """Joined from many parts, and from few."""
    s = Rows(lengths, 1, 4, dim, 64, kind, rht, queries=queries, seed=403)
    sinks = np.array([0.5, -np.inf, 9.0, -9.0], dtype=np.float32)
    s.check(s.call(window=window, sinks=dev(sinks)), s.want(window=window, sinks=sinks))


def test_more_queries_than_tokens():
    s = Rows([3, 0, 70], 2, 2, 64, 16, queries=[6, 40, 75], seed=404)
    for window in (0, 20, 2 ** 23, 2 ** 31 - 1):
        got = s.call(window=window)
        s.check(got, s.want(window=min(window, 10 ** 6)))
        assert (got[0][:3] == 0).all() and (got[0][6:46] == 0).all() and (got[1][:3] == -np.inf).all()


@pytest.mark.parametrize("step", [-1, 1])
@pytest.mark.parametrize("each", [30, 200])
@pytest.mark.parametrize("dim, kind", [(64, "bf16"), (128, "f32"), (256, "bf16")])
def test_scores_that_grow(dim, kind, step, each):
    s = Rows([1300], 2, 4, dim, 16, kind, queries=[40], seed=405)
    for j, slot in enumerate(ref.token_slots(s.table[0], 1300, 16, len(s.cache_host[0]))):
        shift = (j if step > 0 else 1299 - j) // each
        codes = s.cache_host[1][slot // 16, :, :, slot % 16]
        s.cache_host[1][slot // 16, :, :, slot % 16] = np.clip(codes.astype(int) + min(shift, 6) - 3, 0, 254)
    s.check(s.call(), s.want())


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("dim, kind, rht", HEADS[1::3], ids=IDS[1::3])
def test_pages_that_do_not_exist(bad, dim, kind, rht):
    s = Rows([70, 200, 16], 2, 2, dim, 16, kind, rht, queries=[3, 70, 2], seed=406)
    s.table[0, 1] = s.table[1, 0] = s.table[1, 7] = s.table[2, 0] = bad
    got, want = s.call(), s.want()
    s.check(got, want)
    assert (got[0][-1] == 0).all()


@pytest.mark.parametrize("rht", [False, True])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_are_not_finite(dim, rht, window):
    s = Rows([150, 90], 2, 2, dim, 16, rht=rht, queries=[100, 3], seed=407)
    for which, seq, key, head, block in ((2, 0, 120, 0, 1), (2, 0, 75, 1, 0), (0, 0, 140, 1, 1), (2, 1, 88, 0, 0)):
        slot = int(ref.token_slots(s.table[seq], key + 1, 16, len(s.cache_host[0]))[-1])
        s.cache_host[which + 1][slot // 16, head, block, slot % 16] = 255
    want = s.want(window=window)
    assert np.isnan(want[0]).any() and np.isfinite(want[0]).any()
    s.check(s.call(window=window), want)


@pytest.mark.parametrize("byte, codes", BYTES)
@pytest.mark.parametrize("dim, kind, rht", HEADS[1::3], ids=IDS[1::3])
def test_bytes_that_no_row_sees(dim, kind, rht, byte, codes):
    s = Rows([70, 200, 5], 2, 2, dim, 16, kind, rht, queries=[3, 70, 2], seed=408)
    missing = np.argwhere(s.table == 0)
    for at in [tuple(m) for m in missing] or [(1, 4)]:
        s.table[at] = -1
    want, far = s.call(), s.call(window=20)
    s.check(want, s.want())
    s.check(far, s.want(window=20))
    pages = len(s.cache_host[0])
    kept, kept_far = set(), set()
    for row, n, count in zip(s.table, s.lengths, s.queries):
        slots = ref.token_slots(row, int(n), 16, pages).tolist()
        kept |= set(slots)
        kept_far |= set(slots[max(0, int(n) - count - 19):])
    clean = [a.copy() for a in s.cache_host]
    fill(s, np.setdiff1d(np.arange(pages * 16), list(kept)), byte, codes)
    assert same(s.call(), want)
    s.cache_host = clean
    fill(s, np.setdiff1d(np.arange(pages * 16), list(kept_far)), byte, codes)
    assert same(s.call(window=20), far)


@pytest.mark.parametrize("byte, codes", BYTES)
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("dim, kind", [(32, "bf16"), (64, "bf16"), (96, "f32"), (128, "bf16"), (128, "f32"), (256, "bf16"), (256, "f32")])
def test_values_that_some_rows_see(dim, kind, window, byte, codes):
    """Rows that do not see a block of a value, and the other blocks of those
    that do, keep their bits."""
    s = Rows([100], 2, 2, dim, 16, kind, queries=[90], seed=409)
    key, args = 41, dict(window=window, scale=1e-3)        # (every p about the same)
    slot = int(ref.token_slots(s.table[0], key + 1, 16, len(s.cache_host[0]))[-1])
    block = dim // 32 - 1
    s.cache_host[3][slot // 16, 1, block, slot % 16] = 0
    want = s.call(**args)
    s.cache_host[2][slot // 16, 1, slot % 16, 16 * block:16 * block + 16] = codes
    s.cache_host[3][slot // 16, 1, block, slot % 16] = byte
    got = s.call(**args)
    pos = np.arange(90) + 10
    seen = (pos >= key) & ((pos < key + window) | (window == 0))
    touched = np.zeros(got[0].shape, dtype=bool)
    touched[seen, 2:, 32 * block:] = True
    have, kept = got[0].float().cpu().numpy(), want[0].float().cpu().numpy()
    assert np.array_equal(have[~touched], kept[~touched]) and same(got[1:], want[1:])
    if byte < 255 and codes == 0x11:
        s.check(got, s.want(window=window, scale=1e-3))    # finite: 2^125 and 2^126
    else:
        assert not np.isfinite(have[touched]).any()


@pytest.mark.parametrize("lengths, queries", [([0, 65, 300], [2, 3, 70]), ([2500, 0], [60, 2])])
@pytest.mark.parametrize("kind, rht", [("bf16", True), ("f32", False)])
def test_large_sinks(lengths, queries, kind, rht):
    s = Rows(lengths, 2, 4, 64, 16, kind, rht, queries=queries, seed=410)
    sinks = np.array([np.inf, 3e38, np.finfo(np.float32).min, 2e38, -2e38, -np.inf, 1.0, np.nan], dtype=np.float32)
    out, lse = s.call(sinks=dev(sinks))
    assert (out[:, 0] == 0).all() and (lse[:, 0] == np.inf).all()
    assert bool(out[:, 7].isnan().all()) and bool(lse[:, 7].isnan().all())
    finite = sinks.copy()
    finite[0] = finite[7] = 1.0                            # (checked above)
    want = s.want(sinks=finite)
    for w in want:
        w[:, [0, 7]] = 0.0
    out[:, [0, 7]], lse[:, [0, 7]] = 0.0, 0.0
    s.check((out, lse), want)


def test_queries_that_are_not_finite():
    s = Rows([100, 50], 1, 2, 64, 16, queries=[70, 1], seed=411)
    s.q[0, 1, 3] = float("nan")
    s.q64[0, 1, 3] = np.nan
    s.check(s.call(), s.want())


@pytest.mark.parametrize("layout", ["heads first", "joint"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_layouts_and_rows_in_no_sequence(layout, kind):
    tt = torch()
    s = Rows([100, 70], 2, 3, 96, 16, kind, queries=[60, 2], rht=True, seed=412)
    want = s.call()
    s.check(want, s.want())
    _, q = values((66, 6, 96), s.q.dtype, 413)
    q[1:63] = s.q
    out, lse = layouts(tt.full_like(q, 3.0), layout), tt.full((66, 6), 5.0, device="cuda")
    s.call(q=layouts(q, layout), q_offsets=dev(s.offsets + 1), out=out, lse=lse)
    assert same((out[1:63], lse[1:63]), want)
    assert (out[0] == 3).all() and (out[63:] == 3).all() and (lse[0] == 5).all() and (lse[63:] == 5).all()


def test_same_bits_captured_and_beside_another_stream():
    tt = torch()
    s = Rows([900, 300], 2, 4, 128, 64, queries=[70, 40], rht=True, seed=414)
    args = (s.cache(), s.q.clone(), dev(s.table), dev(s.lengths))
    off = dev(s.offsets)
    call = lambda **kw: mx.cache_attention(*args, q_offsets=off, **kw)[0]  # noqa: E731
    want = call()
    s.check((want, s.call()[1]), s.want())
    stream = tt.cuda.Stream()
    stream.wait_stream(tt.cuda.current_stream())
    with tt.cuda.stream(stream):
        call()
    tt.cuda.current_stream().wait_stream(stream)
    tt.cuda.synchronize()
    graph = tt.cuda.CUDAGraph()
    with tt.cuda.graph(graph):
        out = call()
    for i in range(4):
        args[1].copy_(s.q * (1.0 + 0.25 * i))
        args[3].copy_(dev(s.lengths - 7 * i))
        with tt.cuda.stream(stream):
            stream.wait_stream(tt.cuda.current_stream())
            other = call()
        tt.cuda.current_stream().wait_stream(stream)
        graph.replay()
        tt.cuda.synchronize()
        eager = call()
        assert tt.equal(out, eager) and tt.equal(other, eager)
        assert i > 0 or tt.equal(out, want)
