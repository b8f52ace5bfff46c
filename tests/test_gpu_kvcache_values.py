"""Attention over the cache where values, keys and weights lie far apart: what a row does not see has no part in it
whatever it holds, and what it sees keeps its bits whatever stands beside it."""
import numpy as np
import pytest

from oracle import kvcache as ok
from tests.test_gpu_kvcache import _t, cache_case, check_cache, run_cache

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


def check_far(c, got, scale, rows=None):
    """check_cache with what fp16 weights add where values or weights lie far apart.  A cached key's weight times its
    value scale, w, is held in 11 bits, or within 2^-25 of the largest w of its 128 keys where it is 2^-14 of that or
    less (and within 2^-52 of the largest of all); times |code| <= 448, over the sum of the weights."""
    out, lse = got
    cache, page, g = c["cache"], c["page"], c["heads"] // c["kv"]
    codes, vs, kc, ks = (x.float().cpu().numpy().astype(np.float64) for x in (cache.v, cache.v_scale, cache.k, cache.k_scale))
    qf = c["q"].float().cpu().numpy().astype(np.float64)
    fresh = c["k"] is not None
    if fresh:
        kf, vf = (c[x].float().cpu().numpy().astype(np.float64) for x in ("k", "v"))
    for b, ln in enumerate(c["lens"]):
        pages = c["table"][b, :-(-ln // page)]
        for h in range(c["kv"]):
            s = np.repeat(vs[pages, h], page)[:ln]
            code = codes[pages, h].reshape(-1, c["hd"])[:ln]
            k = (kc[pages, h] * ks[pages, h][:, None, None]).reshape(-1, c["hd"])[:ln]
            v, see = code * s[:, None], np.ones((c["slots"], ln), bool)
            if fresh:
                k, v = np.concatenate([k, kf[b, :, h]]), np.concatenate([v, vf[b, :, h]])
                m = np.tril(np.ones((c["slots"],) * 2, bool)) if c["mask"] is None else c["mask"][b] != 0
                see = np.concatenate([see, m], 1)
            for j in range(h * g, (h + 1) * g):
                o, l, to, tl = ok.attend(qf[b, :, j], k, v, see, scale, 2.0 ** -11)
                for a in range(c["slots"]) if rows is None else rows:
                    w = np.exp(scale * (k[:ln] @ qf[b, a, j]) - l[a]) * s
                    extra = sum(2.0 ** -25 * w[t:t + 128].max() * np.abs(code[t:t + 128]).sum(0) for t in range(0, ln, 128))
                    extra = extra + 2.0 ** -52 * w.max(initial=0) * np.abs(code).sum(0)
                    off = np.abs(out[b, a, j] - o[a])
                    assert (off <= to[a] + extra).all(), (b, a, j, off.max(), to[a].max(), np.max(extra))
                    assert abs(lse[b, a, j] - l[a]) <= tl[a]


@pytest.mark.parametrize("slots", [1, 5, 40, 65])
@pytest.mark.parametrize("gap,ratio", [(40, 30), (30, 20), (25, 40), (14, 30), (13, 20), (9, 14)])
def test_pages_of_large_values_without_weight(slots, gap, ratio):
    """Every third page has 2^ratio times the others' value scale, and logits that are some `gap` lower."""
    torch = _t()
    c = cache_case(np.random.RandomState(61), [200, 90, 400], slots, 8, 2, 128, 16, "tree")
    cache = c["cache"]
    c["q"] *= 0.25
    c["q"][..., 0] = 8
    low = torch.tensor(-gap * 32.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).item()
    unit = 2.0 ** -8 if gap <= 14 else 2.0 ** -6
    for b, ln in enumerate(c["lens"]):
        pages = torch.tensor(c["table"][b, :-(-ln // 16)]).cuda()
        cache.k_scale[pages], cache.v_scale[pages] = unit, 2.0 ** -20
        cache.v_scale[pages[::3]] = 2.0 ** (ratio - 20)
        channel = cache.k.view(torch.uint8)[..., 0]
        channel[pages], channel[pages[::3]] = 0, low
        if ln % 16:  # what lies behind the length stays NaN
            for x in (cache.k, cache.v):
                x.view(torch.uint8)[int(pages[-1]), :, int(ln % 16):] = 0x7F
    c["k"][..., 0] = 0
    c["v"] *= 2.0 ** -13
    check_far(c, run_cache(c, scale=1.0), 1.0, rows=None if slots < 10 else [0, 1, slots // 2, slots - 1])


@pytest.mark.parametrize("slots", [1, 40])
def test_a_key_of_nearly_all_weight_and_no_value(slots):
    """A first token that takes most of every row's weight and has zeros for values, before thousands of equal ones: each has
    2^-22 of its weight."""
    torch = _t()
    c = cache_case(np.random.RandomState(62), [3000, 700], slots, 4, 1, 64, 16, None)
    cache = c["cache"]
    c["q"].zero_()
    c["q"][..., 0] = 1
    cache.k_scale.fill_(1)
    cache.v_scale.fill_(2.0 ** -7)
    cache.v.copy_((cache.v.float().nan_to_num(0).abs() + 64).clamp(max=448).to(torch.float8_e4m3fn))
    for b, ln in enumerate(c["lens"]):
        pages = torch.tensor(c["table"][b, :-(-ln // 16)]).cuda()
        cache.k.view(torch.uint8)[..., 0][pages] = 0
        cache.k[int(pages[0]), :, 0, 0] = 15.0
        cache.v.view(torch.uint8)[int(pages[0]), :, 0] = 0
    check_far(c, run_cache(c, scale=1.0), 1.0, rows=[0, slots - 1])


def test_scales_that_are_no_powers_of_two_keep_the_weights_bits():
    """The shape of the repeated calls, whose value scales differ by odd factors."""
    c = cache_case(np.random.RandomState(32 + 64 + 16), [257] * 20, 32, 32, 4, 64, 16, None)
    check_cache(c, run_cache(c), rows=[0, 1, 16, 31])


# ---------------------------------------------------------------------------
# values that are not finite, and lse
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens,slots,heads,kv,hd", SIZES)
def test_lse_has_no_values_in_it(lens, slots, heads, kv, hd):
    """NaN and infinite values among the new tokens and in the cache: the rows that see them are not finite in that
    channel, every row's lse is what it would be without them."""
    torch = _t()
    c = cache_case(np.random.RandomState(55), lens, slots, heads, kv, hd, 64, "random")
    clean = dict(c, v=c["v"].clone())
    want, want_lse = run_cache(clean)
    bad = np.zeros((len(lens), slots), bool)
    for b, (s, val) in enumerate([(0, np.nan), (slots - 1, np.inf), (slots // 2, -np.inf), (1, np.nan)][:len(lens)]):
        c["v"][b, s, :, 5] = float(val)
        bad[b] = c["mask"][b, :, s] != 0
    out, lse = run_cache(c)
    np.testing.assert_array_equal(lse, want_lse)
    assert bad.any() and not bad.all()
    np.testing.assert_array_equal(out[~bad], want[~bad])
    assert not np.isfinite(out[bad][..., 5]).any()
    # a cached value
    b = int(np.argmax(lens))
    cache, page = c["cache"], c["table"][int(np.argmax(lens)), 0]
    cache.v.view(torch.uint8)[int(page), :, 7, 3] = 0x7F
    out, lse = run_cache(clean)
    np.testing.assert_array_equal(lse, want_lse)
    assert not np.isfinite(out[b, :, :, 3]).any()
    keep = np.arange(len(lens)) != b
    np.testing.assert_array_equal(out[keep], want[keep])


@pytest.mark.parametrize("hd", [64, 128])
def test_lse_of_prompts_has_no_values_in_it(hd):
    """The same wherever the value stands in a prompt: in its first key tiles, or among a tile's last keys."""
    torch = _t()
    from tests.test_gpu_kvcache import dev, run_prompt
    rs = np.random.RandomState(56)
    lens = [300, 700, 17]
    q, k, v = (dev(rs.randn(sum(lens), h, hd), torch.bfloat16) for h in (8, 2, 2))
    want, want_lse = run_prompt(q, k, v, lens)
    bad = np.zeros(sum(lens), bool)
    for row, end, val in ((3, 300, np.nan), (299, 300, np.inf), (300 + 650, 1000, -np.inf), (1010, 1017, np.nan)):
        v[row, :, 9] = float(val)
        bad[row:end] = True
    out, lse = run_prompt(q, k, v, lens)
    np.testing.assert_array_equal(lse, want_lse)
    np.testing.assert_array_equal(out[~bad], want[~bad])
    assert not np.isfinite(out[bad][..., 9]).any()
