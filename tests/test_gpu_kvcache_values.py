"""Attention over the cache where values, keys and weights lie far apart: what a row does not see has no part in it
whatever it holds, and what it sees keeps its bits whatever stands beside it."""
import numpy as np
import pytest

from tests.test_gpu_kvcache import _t, cache_case, check_cache, dev, run_cache

pytestmark = pytest.mark.gpu


# (lens, slots, heads, kv, head_dim): both kernels, and both in one call
SIZES = [([50, 0, 200], 4, 8, 2, 128), ([50, 0, 200], 40, 8, 2, 128), ([9, 300], 65, 10, 2, 64), ([130], 150, 4, 2, 128),
         ([50, 0, 200, 9], 66, 32, 8, 128)]


@pytest.mark.parametrize("lens,slots,heads,kv,hd", SIZES)
@pytest.mark.parametrize("val", [1e10, 1e30, -3.3e38])
def test_unseen_new_tokens_may_hold_any_number(lens, slots, heads, kv, hd, val):
    """Large finite keys and values of new tokens that some rows see, or none."""
    c = cache_case(np.random.RandomState(51), lens, slots, heads, kv, hd, 64, "random")
    c["mask"][:, :, 1] = 0  # seen by nobody
    skip, clean = set(), dict(c, k=c["k"].clone(), v=c["v"].clone())
    for b in range(len(lens)):
        for s, where in ((1, "kv"), (slots // 2, "k"), (slots - 1, "v")):
            for x in where:
                c[x][b, s] = val
            skip |= {(b, a) for a in range(slots) if c["mask"][b, a, s]}
    rows = None if slots * heads < 1000 else [0, 1, 2, 3, slots // 2, *range(slots - 6, slots)]
    check_cache(clean, run_cache(c), rows=rows, skip=skip)
    assert len(skip) < len(lens) * slots
