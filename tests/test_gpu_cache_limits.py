"""GPU: the attention over the MXFP4 cache at the ends of what its arguments
may be: windows up to 2^31 - 1, every scale byte in what a row does not see,
sinks up to infinity.
Compared, and with the tolerances, as in test_gpu_cache.py."""
import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from gpu_util import dev, torch
from oracle import cache as ref
from test_gpu_cache import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 320, 319, 290])
@pytest.mark.parametrize("queries", [None, [3, 40, 75, 2], [200, 40, 75, 2]])
def test_windows_as_long_as_the_cache_and_longer(queries, window):
    """Queries before the first key see nothing then either, and the sequences
    after them get their rows."""
    s = Setup([0, 20, 70, 300], 2, 2, 64, 16, queries=queries, seed=301)
    assert s.table.shape[1] * s.page == 320
    got = s.call(window=window, max_queries=None if queries is None else max(queries))
    s.check(got, s.want(window=min(window, 10 ** 6)))
    if window >= 300:                                      # as many as the longest sequence has: none
        none = s.call(max_queries=None if queries is None else max(queries))
        assert all(np.array_equal(a.float().cpu().numpy(), b.float().cpu().numpy()) for a, b in zip(got, none))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 500])
def test_sequences_without_keys_beside_others(window):
    """Padded sequences: rows, but no tokens."""
    tt = torch()
    s = Setup([0, 0, 400, 0, 65], 1, 4, 128, 64, rht=True, queries=[40, 1, 7, 33, 65], seed=302)
    got = s.call(window=window)
    s.check(got, s.want(window=min(window, 10 ** 6)))
    assert (got[0][:41] == 0).all() and bool(tt.isneginf(got[1][:41]).all())


def same(a, b):
    return all(np.array_equal(x.float().cpu().numpy(), y.float().cpu().numpy(), equal_nan=True) for x, y in zip(a, b))


def fill(s, slots, byte, codes):
    for c, sc in ((0, 1), (2, 3)):
        s.cache_host[c][slots // s.page, :, slots % s.page] = codes
        s.cache_host[sc][slots // s.page, :, :, slots % s.page] = byte


# scale bytes from which on some codes, or all, pass the range of fp32; codes of 6, 4, -2 and 2, 0.5
BYTES = [(253, 0x77), (253, 0x66), (254, 0x77), (254, 0xC4), (254, 0x11), (255, 0x77), (255, 0x00)]


@pytest.mark.parametrize("byte, codes", BYTES)
@pytest.mark.parametrize("queries", [None, [3, 70, 2], [1, 5, 4]])
@pytest.mark.parametrize("dim, kind, rht", [(64, "bf16", False), (96, "f32", True), (128, "bf16", True), (160, "bf16", False),
                                            (256, "f32", False)])
def test_bytes_that_no_row_sees(dim, kind, rht, queries, byte, codes):
    """Behind a sequence's length, before a window, and in the page that stands
    in for one that does not exist."""
    s = Setup([70, 200, 5], 2, 2, dim, 16, kind, rht, queries=queries, seed=303)
    missing = np.argwhere(s.table == 0)
    for at in [tuple(m) for m in missing] or [(1, 4)]:
        s.table[at] = -1
    known = None if queries is None else max(queries)
    want, far = s.call(max_queries=known), s.call(max_queries=known, window=20)
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
    assert same(s.call(max_queries=known), want)
    s.cache_host = clean
    fill(s, np.setdiff1d(np.arange(pages * 16), list(kept_far)), byte, codes)
    assert same(s.call(max_queries=known, window=20), far)


@pytest.mark.parametrize("byte, codes", BYTES)
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("dim, kind, group", [(64, "bf16", 2), (128, "bf16", 2), (128, "f32", 1), (256, "bf16", 2), (32, "bf16", 4)])
@pytest.mark.parametrize("known", [True, False])
def test_values_that_some_rows_see(known, dim, kind, group, window, byte, codes):
    """A block of a value: rows that do not see it, and the other blocks of those
    that do, keep their bits."""
    s = Setup([100], 2, group, dim, 16, kind, queries=[8 if known else 90], seed=304)
    n = s.queries[0]
    key = 96 if known else 41
    args = dict(window=window, scale=1e-3, max_queries=n if known else None)     # (every p about the same)
    slot = int(ref.token_slots(s.table[0], key + 1, 16, len(s.cache_host[0]))[-1])
    block = dim // 32 - 1
    s.cache_host[3][slot // 16, 1, block, slot % 16] = 0
    want = s.call(**args)
    s.cache_host[2][slot // 16, 1, slot % 16, 16 * block:16 * block + 16] = codes
    s.cache_host[3][slot // 16, 1, block, slot % 16] = byte
    got = s.call(**args)
    pos = np.arange(n) + 100 - n
    seen = (pos >= key) & ((pos < key + window) | (window == 0))
    assert seen.any() and not seen.all()
    touched = np.zeros(got[0].shape, dtype=bool)
    touched[seen, group:, 32 * block:] = True
    have, kept = got[0].float().cpu().numpy(), want[0].float().cpu().numpy()
    assert np.array_equal(have[~touched], kept[~touched]) and same(got[1:], want[1:])
    if byte < 255 and codes == 0x11:
        s.check(got, s.want(window=window, scale=1e-3))    # finite: 2^125 and 2^126
    else:
        assert not np.isfinite(have[touched]).any()


@pytest.mark.parametrize("lengths, queries", [([0, 65, 300], None), ([0, 65, 300], [2, 3, 70]), ([2500, 0], [3, 1]),
                                              ([2500, 0], [60, 2])])
@pytest.mark.parametrize("kind, rht", [("bf16", True), ("f32", False)])
def test_large_sinks(lengths, queries, kind, rht):
    """Times log2 e the second and third pass fp32's range."""
    s = Setup(lengths, 2, 4, 64, 16, kind, rht, queries=queries, seed=305)
    sinks = np.array([np.inf, 3e38, np.finfo(np.float32).min, 2e38, -2e38, -np.inf, 1.0, np.nan], dtype=np.float32)
    out, lse = s.call(sinks=dev(sinks))
    assert (out[:, 0] == 0).all() and (lse[:, 0] == np.inf).all()
    assert (out[:, 1] == 0).all() and (lse[:, 1] == float(sinks[1])).all()
    assert bool(out[:, 7].isnan().all()) and bool(lse[:, 7].isnan().all())
    finite = sinks.copy()
    finite[0] = finite[7] = 1.0                            # (checked above)
    want = s.want(sinks=finite)
    for w in want:
        w[:, [0, 7]] = 0.0
    out[:, [0, 7]], lse[:, [0, 7]] = 0.0, 0.0
    s.check((out, lse), want)


@pytest.mark.parametrize("queries", [None, [3, 70, 1]])
def test_tables_for_all_tokens_that_there_can_be(queries):
    """524287 pages of 4096 tokens a sequence, few of them used: more units than
    32 bits count, if all were."""
    tt = torch()
    s = Setup([70, 300, 5], 32, 2, 32, 4096, queries=queries, seed=306, spare=0)
    narrow = s.call()
    s.check(narrow, s.want())
    wide = tt.full((3, 2 ** 19 - 1), -1, dtype=tt.int32, device="cuda")
    wide[:, :s.table.shape[1]] = dev(s.table)
    args = dict(q_offsets=None if queries is None else dev(s.offsets), need_lse=True)
    got = mx.cache_attention(s.cache(), s.q, wide, dev(s.lengths), max_queries=None if queries is None else 70, **args)
    s.check(got, s.want())


@pytest.mark.parametrize("window", [0, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("rows", [1, 130])
def test_as_many_tokens_as_there_can_be(rows, window):
    """A sequence of 2^31 - 4096 tokens, all of its pages the same one: as over
    that page alone.  A lane adds up 2^18 of the p one after the other, each sum
    off by 2^-24 of itself at most."""
    tt = torch()
    pages = 2 ** 19 - 1
    s = Setup([4096], 1, 1, 32, 4096, "f32", queries=[1], seed=307, spare=0)
    q = s.q.expand(rows, 1, 32).contiguous()
    table = tt.full((1, pages), int(s.table[0, 0]), dtype=tt.int32, device="cuda")
    lengths = tt.full((1,), 2 ** 31 - 4096, dtype=tt.int32, device="cuda")
    out, lse = mx.cache_attention(s.cache(), q, table, lengths, q_offsets=dev(np.array([0, rows], dtype=np.int32)),
                                  max_queries=rows, window=window, need_lse=True)
    want = s.want()
    whole = (2 ** 31 - 4096 if window == 0 or window > 2 ** 30 else 2 ** 30) / 4096
    tol = 2.0 ** -6 * want[2][0] + 1e-5
    # the rows before the last see the page without its last tokens, once: less than 130 of 2^30 tokens
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= tol + 130 * 2.0 ** -30 * np.abs(want[0]).max()).all()
    assert (np.abs(lse.double().cpu().numpy() - want[1] - np.log(whole)) <= 2.0 ** -6).all()


@pytest.mark.parametrize("name, value", [("use_rht", True), ("sign_mask", 5), ("k_codes", None), ("v_scales", None), ("pages", 1),
                                         ("head_dim", 32)])
def test_fields_of_a_cache_cannot_be_set(name, value):
    cache = mx.kv_cache(4, 2, 16, 64)
    before = getattr(cache, name)
    with pytest.raises(AttributeError):
        setattr(cache, name, value)
    assert getattr(cache, name) is before


@pytest.mark.parametrize("which", ["k_codes", "k_scales", "v_codes", "v_scales"])
@pytest.mark.parametrize("how", ["data", "set_", "resize_", "storage"])
def test_a_cache_whose_storage_was_replaced_is_refused(which, how):
    """By each call, which would use the freed address."""
    tt = torch()
    cache = mx.kv_cache(4, 2, 16, 64)
    x, ints = tt.ones((3, 2, 64), device="cuda"), tt.zeros(3, dtype=tt.int32, device="cuda")
    t = getattr(cache, which)
    if how == "data":
        t.data = t.clone()
    elif how == "set_":
        t.set_(tt.zeros_like(t))
    elif how == "resize_":
        t.resize_((64,) + tuple(t.shape[1:]))
    else:
        t.untyped_storage().resize_(0)
    for call in (lambda: mx.cache_write(cache, x, x, ints), lambda: mx.cache_read(cache, ints),
                 lambda: mx.cache_attention(cache, x, tt.zeros((3, 1), dtype=tt.int32, device="cuda"), ints + 1)):
        with pytest.raises(ValueError, match="storage"):
            call()


@pytest.mark.parametrize("name, value", [("window", 2 ** 32 + 5), ("window", 2 ** 31), ("window", -2 ** 32), ("max_queries", 2 ** 32 + 1),
                                         ("max_queries", -2 ** 32)])
def test_numbers_past_32_bits_are_refused(name, value):
    """The first was a window of 5, the second was refused with another reason."""
    s = Setup([70], 1, 2, 32, 16, seed=308)
    with pytest.raises((ValueError, mx.MXError), match=name):
        s.call(**{name: value})
