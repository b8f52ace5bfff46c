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


def test_rows_of_single_slots_and_entries():
    """The first slot of every request, heads and rows of one entry with strides of their own: rows are evenly spaced."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import kv_append
    rs = np.random.RandomState(92)
    c = cache_case(rs, [70, 33, 0], 1, 4, 2, 64, 16, "causal")
    wide = torch.randn(3, 5, 4 + 2 + 2, 64, device="cuda").to(torch.bfloat16)
    one = wide[:, :1]
    c["q"], c["k"], c["v"] = one[:, :, :4], one[:, :, 4:6], one[:, :, 6:]
    assert c["q"].stride(0) != c["q"].stride(1)
    check_cache(c, run_cache(c))
    check_append(c["cache"], c["k"], c["v"], [7 * 16, -1, 3 * 16])
    # one request of one slot whose outer strides fit nothing
    c = cache_case(rs, [70], 1, 4, 2, 64, 16, "causal")
    for x, heads in (("q", 4), ("k", 2), ("v", 2)):
        c[x] = c[x].as_strided((1, 1, heads, 64), (3, 5, 64, 1))
    check_cache(c, run_cache(c))
    kv_append(c["cache"], c["k"][0], c["v"][0], dev([16], torch.int64))


def test_keys_of_other_dimensions_are_refused():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import kv_append
    cache = new_cache(np.random.RandomState(93), 4, 2, 16, 64)
    x = torch.zeros(2, 3, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for k in (x, x[0, 0, 0]):
        with pytest.raises(ValueError):
            kv_append(cache, k, k, dev([0], torch.int64))
    torch.cuda.synchronize()


# (rows left over behind two, four and eight pairs of row tiles, which the streaming kernel takes from 8 key/value heads on)
@pytest.mark.parametrize("lens,slots,heads,kv,hd,page,fresh", [
    ([700, 33], 129, 32, 8, 128, 64, "tree"), ([300], 257, 32, 8, 64, 32, "random"), ([0], 513, 32, 8, 128, 64, "tree"),
    ([150, 0, 40], 513, 8, 2, 128, 16, "tree"), ([40], 259, 16, 16, 128, 128, "causal"),
])
def test_rows_left_over_behind_several_pairs(lens, slots, heads, kv, hd, page, fresh):
    c = cache_case(np.random.RandomState(slots + kv), lens, slots, heads, kv, hd, page, fresh)
    check_cache(c, run_cache(c), rows=[0, 31, slots // 2, *range(slots - 4, slots)])
