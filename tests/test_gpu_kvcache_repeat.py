"""The same bits from the same call, many times over, where a kernel hands shared memory from one role to another."""
import numpy as np
import pytest

from tests.test_gpu_kvcache import _t, cache_case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,slots,heads,kv,hd,page,fresh", [
    ([257] * 20, 32, 32, 4, 64, 16, None),
    ([0, 1, 130, 64, 500, 3, 90, 257], 34, 32, 4, 64, 16, "random"),
    ([0, 1, 130, 64, 500, 3, 90, 257], 34, 32, 4, 64, 64, "random"),
    ([0, 1, 130, 64, 500, 3, 90, 257], 34, 32, 4, 64, 128, "random"),
    ([257] * 20, 32, 32, 4, 128, 64, "tree"),
    ([700, 20, 0, 33], 129, 32, 8, 128, 32, "random"),
])
def test_cache_attention_gives_the_same_bits_every_time(lens, slots, heads, kv, hd, page, fresh):
    """Stretches of a full key tile and one that holds a few keys, the unseen ones NaN: a page copied over one that is
    still to be converted shows in the output."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, cache_attention
    c = cache_case(np.random.RandomState(slots + hd + page), lens, slots, heads, kv, hd, page, fresh)
    table, length, work = dev(c["table"], torch.int32), dev(c["lens"], torch.int32), AttentionWorkspace()
    mask = None if c["mask"] is None else dev(c["mask"], torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, first_lse, differ = None, None, torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        lse = torch.full((len(lens), slots, heads), 7.0, device="cuda")
        out = cache_attention(c["cache"], c["q"], table, length, k_new=c["k"], v_new=c["v"], mask=mask, lse=lse, workspace=work,
                              status=status)
        if first is None:
            first, first_lse = out, lse
        differ += (out.view(torch.int16) != first.view(torch.int16)).sum() + (lse.view(torch.int32) != first_lse.view(torch.int32)).sum()
    assert status.item() == 0 and differ.item() == 0
    assert torch.isfinite(first).all()


def test_prompt_attention_gives_the_same_bits_every_time():
    """Short and long sequences in turn, infinities and NaNs among the last keys of some: items follow one another in a
    CTA, and what one notes for its rows is cleared for the next."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import prompt_attention
    rs = np.random.RandomState(71)
    for hd in (64, 128):
        lens = np.concatenate([rs.randint(1, 300, 400), [700, 1500, 0]])
        rs.shuffle(lens)
        at = np.concatenate([[0], np.cumsum(lens)])
        n = int(at[-1])
        q, k, v = (dev(rs.randn(n, x, hd), torch.bfloat16) for x in (8, 2, 2))
        finite = np.ones(n, bool)
        for i in rs.choice(np.nonzero(lens > 1)[0], 150, replace=False):
            row = rs.randint(max(at[i], at[i + 1] - 20), at[i + 1])
            v[row, :, rs.randint(hd)] = float(rs.choice([np.nan, np.inf, -np.inf]))
            finite[row:at[i + 1]] = False
        start = dev(at, torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        first, differ = None, torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(200):
            out = prompt_attention(q, k, v, start, status=status)
            first = out if first is None else first
            differ += (out.isnan() != first.isnan()).sum() + (out.nan_to_num(0) != first.nan_to_num(0)).sum()
        assert status.item() == 0 and differ.item() == 0
        seen = torch.isfinite(first).flatten(1).all(1).cpu().numpy()
        np.testing.assert_array_equal(seen, finite)


@pytest.mark.parametrize("heads,kv,hd", [(6, 2, 128), (7, 1, 64), (40, 8, 128), (6, 1, 64), (100, 2, 128)])
def test_prompt_attention_of_odd_groups_gives_the_same_bits_every_time(heads, kv, hd):
    """Where a group's heads do not divide 128, a tile has rows without a query; and a sequence's last tile has rows of the
    next one's, whose queries are changed in between: neither has a say in a row's bits."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import prompt_attention
    rs = np.random.RandomState(72)
    lens = rs.randint(1, 700, 12)
    at = np.concatenate([[0], np.cumsum(lens)])
    n = int(at[-1])
    q, k, v = (dev(rs.randn(n, x, hd), torch.bfloat16) for x in (heads, kv, kv))
    other = q.clone()
    for i in range(1, 12, 2):  # every other sequence's queries
        other[at[i]:at[i + 1]] *= 30
    loud = [30 * dev(rs.randn(900, x, hd), torch.bfloat16) for x in (8 * kv, kv, kv)]
    start, one = dev(at, torch.int32), dev([0, 900], torch.int32)
    same = torch.cat([torch.arange(at[i], at[i + 1]) for i in range(0, 12, 2)]).cuda()
    first, differ = prompt_attention(q, k, v, start), torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            prompt_attention(*loud, one)
        differ += (prompt_attention(q, k, v, start).view(torch.int16) != first.view(torch.int16)).sum()
        got = prompt_attention(other, k, v, start)
        differ += (got[same].view(torch.int16) != first[same].view(torch.int16)).sum()
    assert differ.item() == 0
