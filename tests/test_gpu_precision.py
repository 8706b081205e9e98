"""GPU: what is left of the rounding errors where little is added up, so that a
term of a sum of bf16, or a few tokens, cannot be missing unseen.

Attention of fp32 queries.  Key j is the unit vector e_j, value j too, for as
many keys as the head has elements; all other keys of the sequence lie in pages
that do not exist, and add exact zeros.  So score j is q_j, and output j is
p_j / sum p.  In steps of u = 2^-24 relative, |q| <= R:
  - q as three bf16 terms: what is left of it is u, their sum in the product two
    additions of 2 u: 5 u of |q|, with the constant log2 e 6 u; the subtraction of
    the reference one of u of a difference of up to 2 R: 8 R u in the exponent;
    the exponential 2 u: p is off by (8 R + 2) u, and so is the sum of them
    relative to itself;
  - the sum of the p: eight additions in a lane, two between lanes, four waves,
    four parts joined: 18 u;
  - p as three terms, u, their sum 4 u; waves and parts added up 8 u, each
    scaled by a factor 4 u; the division and the multiplication 3 u.
Together (16 R + 42) u of the output.  (With two terms, 2^-17 of q is missing,
128 R u, or of p, 128 u.)  lse: (8 R + 22) u, its own product and logarithm
4 u of itself and of the sum's.

Balance loss.  A lane adds up its rows' scores, then log2(64 / lanes) exchanges,
16 waves, and workgroups in 64 bits; a score is an exponential (4 u) over a sum of
4 C of them in each of the row's lanes, exchanged log2(lanes) times, u for the
inverse and u for the product.  All terms are positive."""
import numpy as np
import pytest

from mxfp4_precision_numerics_amd import mx
from gpu_util import dev, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bounds(reach, lse):
    """In steps of U: of the outputs, relative, and of lse."""
    return 16 * reach + 42, 8 * reach + 22 + 4 * (np.abs(lse) + reach)


def units(dim, length, seed, width=0):
    """A cache whose pages hold the unit vectors, and a table that has them
    somewhere within `length` tokens (and is for `width`)."""
    tt, rng = torch(), np.random.default_rng(seed)
    pages = dim // 16
    cache = mx.kv_cache(pages, 1, 16, dim)
    codes = np.zeros((pages, 1, 16, dim // 2), dtype=np.uint8)
    for j in range(dim):
        codes[j // 16, 0, j % 16, j // 2] = 2 << (4 * (j % 2))               # (2: the code of 1)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(tt.from_numpy(codes))
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(127)
    table = np.full((1, max(length, width) // 16), -1, dtype=np.int32)
    table[0, np.sort(rng.choice(length // 16, size=pages, replace=False))] = rng.permutation(pages)
    return cache, dev(table)


@pytest.mark.parametrize("reach", [1, 8])
@pytest.mark.parametrize("length", [256, 4096])
@pytest.mark.parametrize("rows", [1, 20, 300])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("width", [0, 2 ** 23])
def test_three_terms(width, dim, rows, length, reach):
    """Few rows and many, in one share and joined from several; a table for many
    tokens chooses the kernel for many rows where there are 300."""
    tt = torch()
    cache, table = units(dim, length, dim + length, width)
    heads = 1 if rows > 1 else 16
    q = np.random.default_rng(rows).uniform(-reach, reach, size=(rows, heads, dim)).astype(np.float32)
    out, lse = mx.cache_attention(cache, dev(q), table, tt.tensor([length], dtype=tt.int32, device="cuda"), scale=1.0,
                                  q_offsets=tt.tensor([0, rows], dtype=tt.int32, device="cuda"), max_queries=rows, causal=False,
                                  need_lse=True)
    p = np.exp(q.astype(np.float64))
    total = p.sum(-1, keepdims=True)
    want = np.log(total[..., 0])
    limit, limit_lse = bounds(reach, want)
    far = np.abs(out.double().cpu().numpy() / (p / total) - 1.0).max() / U
    assert far <= limit, far
    far = (np.abs(lse.double().cpu().numpy() - want) / limit_lse).max() / U
    assert far <= 1.0, far


# tokens, experts, and how many lanes share a row, chunks of four experts each has
SUMS = [(20000, 16, 8, 1), (65536, 64, 16, 1), (65536, 256, 16, 4), (300001, 32, 8, 1), (8192, 1024, 64, 4), (70, 500, 32, 4)]


@pytest.mark.parametrize("case", SUMS, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("score", [0, 1])
def test_no_token_is_missing_in_the_balance_loss(case, score):
    tokens, experts, lanes, chunks = case
    rng = np.random.default_rng(tokens)
    l = (2 * rng.normal(size=(tokens, experts))).astype(np.float32)
    ids = rng.integers(0, experts, size=(tokens, 2)).astype(np.int32)
    loss, counts, slope = mx.balance(dev(l), dev(ids), score=score)
    x = l.astype(np.float64)
    s = np.exp(x - x.max(1, keepdims=True)) if score == 0 else 1.0 / (1.0 + np.exp(-x))
    s /= s.sum(1, keepdims=True)
    c = np.bincount(ids.ravel(), minlength=experts)
    want = float((experts * c / (2.0 * tokens * tokens) * s.sum(0)).sum())
    assert np.array_equal(counts.cpu().numpy(), c)
    rows = -(-tokens // (min(-(-tokens // 64), 256) * (1024 // lanes)))
    depth = rows + np.log2(64 / lanes) + 16
    one = 4 + 4 * chunks + np.log2(lanes) + 2 + (6 if score else 0)          # (a sigmoid: its own sum, inverse, product)
    assert abs(float(loss) - want) <= (depth + 2 * one + 2) * U * want
