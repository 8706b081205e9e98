"""Pins of oracle/cache.py: hand-worked cases, invariants, differences."""
import numpy as np

import oracle
from oracle import cache as ref


def filled(pages, heads, page, dim, seed):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(2):
        c, s = oracle.quantize_1d(rng.normal(size=(pages * heads * page, dim)).astype(np.float32))
        out += [c.reshape(pages, heads, page, dim // 2), s.reshape(pages, heads, page, dim // 32).swapaxes(2, 3)]
    return out


def test_decode_is_the_quantizers_decode():
    x = np.random.default_rng(0).normal(size=(20, 96)).astype(np.float32)
    c, s = oracle.quantize_1d(x)
    assert np.array_equal(ref.decode(c, s), oracle.dequantize(c, s).astype(np.float64))
    assert np.array_equal(ref.decode(np.array([[0x2F] + [0] * 15]), np.array([[129]]))[0, :2], [-24.0, 4.0])


def test_transform_is_orthogonal_and_the_libraries():
    x = np.random.default_rng(1).normal(size=(5, 64)).astype(np.float32)
    y = ref.rht(x, 0x9A3C61E5)
    assert np.abs(ref.rht(y, 0x9A3C61E5, inverse=True) - x).max() < 1e-14
    assert np.abs(oracle.rht(x, 0x9A3C61E5) - y).max() < 1e-6


def test_attention_of_one_key_is_its_value():
    cache = filled(2, 1, 16, 32, 2)
    q = np.random.default_rng(3).normal(size=(1, 1, 32))
    out, lse, _, _ = ref.attention(cache, q, np.array([[1]]), [1])
    v = ref.held(cache[2], cache[3], np.array([16]), 0)[0]
    k = ref.held(cache[0], cache[1], np.array([16]), 0)[0]
    assert np.array_equal(out[0, 0], v) and abs(lse[0, 0] - k @ q[0, 0] / np.sqrt(32)) < 1e-12


def test_attention_is_the_plain_softmax():
    cache = filled(5, 2, 16, 64, 4)
    table, length, n = np.array([[3, 0, 4]]), 40, 6
    q = np.random.default_rng(5).normal(size=(n, 4, 64))
    out, lse, _, _ = ref.attention(cache, q, table, [length], q_offsets=[0, n])
    slots = ref.token_slots(table[0], length, 16, 5)
    assert slots[0] == 48 and slots[17] == 1 and slots[39] == 71
    for h in range(4):
        k, v = (ref.held(c, s, slots, h // 2) for c, s in ((cache[0], cache[1]), (cache[2], cache[3])))
        z = q[:, h] @ k.T / 8.0
        z[np.arange(length)[None, :] > (length - n + np.arange(n))[:, None]] = -np.inf
        e = np.exp(z - z.max(1, keepdims=True))
        assert np.allclose(out[:, h], e @ v / e.sum(1, keepdims=True), atol=1e-12)


def test_masks():
    cache = filled(3, 1, 16, 32, 6)
    q = np.random.default_rng(7).normal(size=(2, 1, 32))
    out, lse, _, _ = ref.attention(cache, q, np.array([[0, 9]]), [30], q_offsets=[0, 2])
    short, _, _, _ = ref.attention(cache, q[:1], np.array([[0]]), [16])
    assert np.allclose(out[0], short[0])                   # the second page does not exist
    one, _, _, _ = ref.attention(cache, q, np.array([[0, 1]]), [30], q_offsets=[0, 2], window=1)
    v = ref.held(cache[2], cache[3], np.array([28, 29]), 0)
    assert np.array_equal(one[:, 0], v)
    none, lse, _, _ = ref.attention(cache, q, np.array([[0, 1]]), [1], q_offsets=[0, 2])
    assert (none[0] == 0).all() and np.isneginf(lse[0, 0])
    sink, lse, _, _ = ref.attention(cache, q[:1], np.array([[0]]), [0], sinks=np.array([2.0]))
    assert (sink == 0).all() and lse[0, 0] == 2.0


def test_transformed_cache_gives_the_same():
    """Rounding aside, the transform changes nothing."""
    rng = np.random.default_rng(8)
    q, (k, v) = rng.normal(size=(1, 1, 32)), rng.normal(size=(2, 16, 32))
    plain = np.exp(k @ q[0, 0] / np.sqrt(32))
    want = plain @ v / plain.sum()
    cache = []
    for x in (k, v):
        c, s = oracle.quantize_1d(x.astype(np.float32), use_rht=True, sign_mask=77)
        cache += [c.reshape(1, 1, 16, 16), s.reshape(1, 1, 16, 1).swapaxes(2, 3)]
    out, _, _, _ = ref.attention(cache, q, np.array([[0]]), [16], mask=77)
    assert np.linalg.norm(out[0, 0] - want) < 0.3 * np.linalg.norm(want)


def test_balance_by_hand():
    l = np.log(np.array([[3.0, 1.0], [1.0, 1.0], [0.0, 0.0]]) + 0.0, where=[[True, True], [True, True], [False, False]],
               out=np.full((3, 2), -np.inf))
    loss, counts, slope = ref.balance(l, np.array([[0], [1], [0]]))
    assert list(counts) == [2, 1] and np.allclose(slope, [2 * 2 / 6, 2 * 1 / 6])
    assert abs(loss - (4 / 6 * (0.75 + 0.5) + 2 / 6 * (0.25 + 0.5))) < 1e-12


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(9)
    l, ids = rng.normal(size=(6, 5)), rng.integers(-1, 5, size=(6, 2))
    l[2, 3] = -np.inf
    for score in (0, 1):
        _, _, slope = ref.balance(l, ids, score)
        got = ref.balance_bwd(l, slope, score)
        for t in range(6):
            for e in range(5):
                if np.isneginf(l[t, e]):
                    assert got[t, e] == 0
                    continue
                d = []
                for h in (1e-5, -1e-5):
                    x = l.copy()
                    x[t, e] += h
                    d.append(ref.balance(x, ids, score)[0])
                assert abs((d[0] - d[1]) / 2e-5 - got[t, e]) < 1e-8
