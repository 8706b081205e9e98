"""GPU: the attention over the MXFP4 cache at the ends of what its arguments
may be: windows up to 2^31 - 1.  Compared, and with the tolerances, as in
test_gpu_cache.py."""
import numpy as np
import pytest

from gpu_util import torch
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
