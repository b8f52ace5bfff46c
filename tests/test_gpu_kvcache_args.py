"""Arguments at the edges of what the cache's bindings take."""
import numpy as np
import pytest

from oracle import kvcache as ok
from tests.test_gpu_kvcache import _t, cache_case, check_append, check_cache, dev, new_cache, pool, run_cache, run_plan, same_plan

pytestmark = pytest.mark.gpu


def test_plan_with_a_path_of_no_width():
    """Every request commits its root only: source rows are the roots' of [n_req, path_rows], and a second new token is a
    path that is too short."""
    rs = np.random.RandomState(91)
    old = rs.randint(0, 60, 5)
    path = np.zeros((5, 0), np.int64)
    table, ring, head, count = pool(rs, old, 6, 16, 9)
    want = ok.plan(old, None, 1, table, ring, head, count, 16, 8, path, 65)
    assert want["status"] == 0 and want["src"][:5].tolist() == [0, 65, 130, 195, 260]
    same_plan(run_plan(old, None, 1, table, ring, head, count, 16, 8, path, 65), want)
    delta = [0, 1, 0, 0, 0]
    want = ok.plan(old, delta, 1, table, ring, head, count, 16, 8, path, 65)
    assert want["status"] == ok.BAD_PATH
    same_plan(run_plan(old, delta, 1, table, ring, head, count, 16, 8, path, 65), want)
