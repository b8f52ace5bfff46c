"""The key/value cache operators on the GPU against the 64-bit oracle.

Whole numbers, codes and scales are compared exactly; attention within the bounds that
``oracle.kvcache.attend`` derives for each element.
"""
import numpy as np
import pytest

from oracle import kvcache as ok

pytestmark = pytest.mark.gpu


def _t():
    import torch
    torch.cuda.set_device(0)
    return torch


def dev(x, dtype):
    torch = _t()
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def run_plan(old, delta, extra, table, ring, head, count, page, max_rows, path=None, path_rows=0, stream=None):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import kv_plan
    i32 = torch.int32
    n = len(old)
    b = dict(table=dev(table, i32), ring=dev(ring, i32), len=torch.full((n,), -9, dtype=i32, device="cuda"),
             after=torch.full((2,), -9, dtype=i32, device="cuda"),
             row_start=torch.full((n + 1,), -9, dtype=i32, device="cuda"),
             slot=torch.full((max_rows,), -9, dtype=torch.int64, device="cuda"),
             pos=torch.full((max_rows,), -9, dtype=i32, device="cuda"),
             src=torch.full((max_rows,), -9, dtype=i32, device="cuda"),
             status=torch.full((1,), -9, dtype=i32, device="cuda"))
    kv_plan(dev(old, i32), b["len"], b["table"], b["ring"], dev([head, count], i32), b["after"], b["row_start"], b["slot"],
            b["status"], page=page, delta=None if delta is None else dev(delta, i32), extra=extra, positions=b["pos"],
            path=None if path is None else dev(path, i32), path_rows=path_rows, src_rows=b["src"], stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in b.items()}


def same_plan(got, want):
    assert got["status"][0] == want["status"]
    for k in ("len", "row_start", "table", "ring", "slot", "pos", "src"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    assert got["after"].tolist() == [want["head"], want["count"]]


def pool(rs, old, width, page, spare):
    """Tables with distinct pages, and a ring whose free part starts somewhere."""
    held = [min(width, -(-int(o) // page)) for o in old]
    n_pages = sum(held) + spare
    perm = rs.permutation(n_pages)
    table, at = np.full((len(old), width), -1), 0
    for q, h in enumerate(held):
        table[q, :h] = perm[at:at + h]
        at += h
    head = int(rs.randint(n_pages))
    ring = np.roll(np.concatenate([perm[at:], np.full(at, -1)]), head)
    return table, ring, head, n_pages - at


@pytest.mark.parametrize("n,page,seed", [(1, 16, 0), (3, 32, 1), (32, 64, 2), (33, 128, 3), (511, 16, 4), (513, 64, 5), (4096, 16, 6)])
def test_plan_grows_and_shrinks(n, page, seed):
    rs = np.random.RandomState(seed)
    old = rs.randint(0, 5 * page, n)
    old[rs.rand(n) < 0.2] = 0
    delta = rs.randint(-3 * page, 3 * page, n)
    delta[rs.rand(n) < 0.2] = 0
    table, ring, head, count = pool(rs, old, 9, page, 4 * n + 5)
    rows = int(np.maximum(np.maximum(old + delta, 0) - old, 0).sum())
    for extra, cap in ((0, max(1, rows)), (0, rows + 37), (1, rows + n)):
        same_plan(run_plan(old, delta, extra, table, ring, head, count, page, cap),
                  ok.plan(old, delta, extra, table, ring, head, count, page, cap))


def test_plan_without_delta_and_repeated():
    """One token each; a second call with the same inputs gives the same answers."""
    rs = np.random.RandomState(7)
    old = np.array([0, 15, 16, 17, 31, 32])
    table, ring, head, count = pool(rs, old, 4, 16, 8)
    want = ok.plan(old, None, 1, table, ring, head, count, 16, 6)
    got = run_plan(old, None, 1, table, ring, head, count, 16, 6)
    same_plan(got, want)
    same_plan(run_plan(old, None, 1, got["table"], got["ring"], head, count, 16, 6), want)


def test_plan_commits_accepted_paths():
    rs = np.random.RandomState(8)
    n, D, S = 7, 15, 65
    old = rs.randint(0, 200, n)
    acc = np.array([0, 15, 1, 3, 0, 7, 2])
    path = np.full((n, D), -1)
    for q in range(n):
        path[q, :acc[q]] = np.sort(rs.choice(np.arange(1, S), acc[q], replace=False))
    table, ring, head, count = pool(rs, old, 6, 64, 9)
    same_plan(run_plan(old, acc, 1, table, ring, head, count, 64, n * (D + 1), path, S),
              ok.plan(old, acc, 1, table, ring, head, count, 64, n * (D + 1), path, S))


def test_plan_faults_change_nothing():
    rs = np.random.RandomState(9)
    old = np.array([10, 40, 0, 64])
    table, ring, head, count = pool(rs, old, 4, 16, 2)
    path = np.array([[1, 2], [3, 99], [1, -1], [-1, -1]])
    for kw, bit in ((dict(delta=[40, 0, 0, 0]), ok.SHORT_OF_PAGES), (dict(delta=[0, 30, 0, 0]), ok.BAD_LENGTH),
                    (dict(delta=[3, 3, 3, 0], cap=8), ok.SHORT_OF_ROWS),
                    (dict(delta=[2, 2, 0, 0], path=path), ok.BAD_PATH),       # slot 99 of 65
                    (dict(delta=[2, 0, 2, 0], path=path), ok.BAD_PATH),       # a padded entry
                    (dict(delta=[4, 0, 0, 0], path=path), ok.BAD_PATH),       # more tokens than the path has
                    (dict(old=[-1, 40, 0, 64], delta=[3, 0, 0, 0]), ok.BAD_LENGTH),
                    (dict(delta=[0, -40, 0, -64], count=len(ring) - 3), ok.BAD_INDEX)):  # gives back more than is in use
        o, cap, p, cnt = kw.get("old", old), kw.get("cap", 64), kw.get("path"), kw.get("count", count)
        ex = 1 if p is not None else 0
        want = ok.plan(o, kw["delta"], ex, table, ring, head, cnt, 16, cap, p, 65)
        assert want["status"] & bit
        got = run_plan(o, kw["delta"], ex, table, ring, head, cnt, 16, cap, p, 65)
        same_plan(got, want)
        np.testing.assert_array_equal(got["table"], table)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def new_cache(rs, n_pages, kv, page, hd, pow2=True):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import KvCache
    k = (100 * torch.from_numpy(rs.randn(n_pages, kv, page, hd)).float()).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    v = (100 * torch.from_numpy(rs.randn(n_pages, kv, page, hd)).float()).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    s = np.ldexp(1.0, rs.randint(-9, -3, (2, n_pages, kv)))
    if not pow2:
        s *= rs.uniform(1, 2, s.shape)
    return KvCache(k, v, dev(s[0], torch.float32), dev(s[1], torch.float32))


def codes(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_append(cache, k, v, slots, src=None, stream=None, status=None):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import kv_append
    want = []
    for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        cc, ss = codes(c), s.cpu().numpy().astype(np.float64)
        xx = x.float().cpu().numpy().reshape(-1, cache.n_kv, cache.head_dim)
        ok.append(cc, ss, xx, slots, src, cache.page)
        want.append((cc, ss))
    torch.cuda.synchronize()
    kv_append(cache, k, v, dev(slots, torch.int64), src_rows=None if src is None else dev(src, torch.int32), stream=stream,
              status=status)
    torch.cuda.synchronize()
    for (cc, ss), c, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        np.testing.assert_array_equal(s.cpu().numpy(), ss.astype(np.float32))
        np.testing.assert_array_equal(codes(c), cc)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_runs(page, hd):
    """Runs that start and end anywhere: single tokens, whole pages, pages that already hold tokens."""
    torch = _t()
    rs = np.random.RandomState(page + hd)
    kv = 3
    cache = new_cache(rs, 12, kv, page, hd)
    slots = []
    for pg, a, b in ((3, 0, page), (7, 5, page), (0, 0, 7), (9, page - 1, page), (4, 3, 4), (11, 0, 1), (1, 2, page - 2)):
        slots += list(range(pg * page + a, pg * page + b))
        if pg == 0:
            slots += [-1, -1]
    n = len(slots)
    size = 4.0 ** rs.randint(-4, 4, (n, 1, 1))
    k, v = dev(rs.randn(n, kv, hd) * size, torch.bfloat16), dev(rs.randn(n, kv, hd), torch.bfloat16)
    check_append(cache, k, v, slots)


def test_append_many_rows_in_windows():
    """Enough rows that a CTA looks for runs in a window of several rows; ragged requests, then a second
    append that continues their last pages."""
    torch = _t()
    rs = np.random.RandomState(3)
    page, kv, hd = 16, 8, 64
    lens = rs.randint(1, 60, 90)
    more = rs.randint(0, 30, 90)
    held = -(-(lens + more) // page)
    cache = new_cache(rs, int(held.sum()), kv, page, hd)
    perm, table, at = rs.permutation(int(held.sum())), [], 0
    for h in held:
        table.append(perm[at:at + h])
        at += h
    for a, b in ((np.zeros(90, int), lens), (lens, lens + more)):
        slots = [int(table[q][p // page]) * page + p % page for q in range(90) for p in range(a[q], b[q])]
        n = len(slots)
        k, v = dev(rs.randn(n, kv, hd) * 3, torch.bfloat16), dev(rs.randn(n, kv, hd) * 4.0 ** rs.randint(-3, 3, (n, 1, 1)), torch.bfloat16)
        check_append(cache, k, v, slots)


def test_append_gathers_rows_of_strided_tensors_on_another_stream():
    torch = _t()
    rs = np.random.RandomState(4)
    page, kv, hd, n, S = 32, 2, 128, 3, 17
    cache = new_cache(rs, 8, kv, page, hd)
    qkv = dev(rs.randn(n, S, 4 + 2 * kv, hd), torch.bfloat16)
    k, v = qkv[:, :, 4:4 + kv], qkv[:, :, 4 + kv:]
    slots = [40, 41, 42, -1, 64, -1, 127, 128]
    src = [0, 5, 16, -1, 17, -1, 34, 50]
    st = torch.cuda.Stream()
    check_append(cache, k, v, slots, src, stream=st)


def test_append_special_values():
    """Zeros, the smallest and largest bf16, infinities and NaN."""
    torch = _t()
    rs = np.random.RandomState(5)
    cache = new_cache(rs, 8, 1, 16, 64)
    x = np.zeros((8, 1, 64), np.float32)
    x[1, 0, :4] = [1e-40, -9.2e-41, 3e-39, 0]
    x[2, 0, :3] = [3.38e38, -1e30, 1]
    x[3, 0, :4] = [np.inf, -np.inf, np.nan, 2.5]
    x[4, 0] = np.nan
    x[5, 0] = 448
    x[6, 0] = np.linspace(-450, 450, 64)
    x[7, 0] = np.ldexp(1.0, -np.arange(64))
    k = dev(x, torch.bfloat16)
    slots = [0, 17, 33, 48, 64, 95, 96, 112]  # a page each
    check_append(cache, k, k.flip(0).contiguous(), slots)


def test_append_scales_that_are_no_powers_of_two():
    torch = _t()
    rs = np.random.RandomState(6)
    cache = new_cache(rs, 4, 2, 16, 64, pow2=False)
    # values far below the present scale, so that it stays and is divided by; the quotient is rounded
    # once to 32 bits before e4m3, as the oracle's is to 64: inputs stay off the midpoints
    from conditional_draft_tree_lm_gb300 import kv_append
    x = dev(np.full((1, 2, 64), 0.25), torch.bfloat16)
    before = cache.k_scale.clone()
    kv_append(cache, x, x, dev([5], torch.int64))
    assert torch.equal(before, cache.k_scale)
    got = cache.k[0, :, 5].float() * before[0][:, None]
    assert ((got - 0.25).abs() <= 0.25 * 2.0 ** -4 * 1.001).all()


def test_append_bad_indexes_are_reported_and_skipped():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import kv_append
    rs = np.random.RandomState(7)
    cache = new_cache(rs, 4, 1, 16, 64)
    x = dev(rs.randn(3, 1, 64), torch.bfloat16)
    k0 = cache.k.clone().view(torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_append(cache, x, x, dev([64, 1 << 40, -5], torch.int64), status=status)
    assert status.item() == ok.BAD_INDEX and torch.equal(k0, cache.k.view(torch.uint8))
    status.zero_()
    kv_append(cache, x, x, dev([16], torch.int64), src_rows=dev([3], torch.int32), status=status)
    assert status.item() == ok.BAD_INDEX and (cache.k[1, 0, 0].float() == 0).all()
    kv_append(cache, x, x, torch.empty(0, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
def tree_masks(rs, n, slots):
    parent = np.maximum(np.arange(slots) - 1 - rs.randint(0, 8, (n, slots)), 0)
    mask = np.zeros((n, slots, slots), np.uint8)
    mask[:, 0, 0] = 1
    for a in range(1, slots):
        mask[:, a] = mask[np.arange(n), parent[:, a]]
        mask[:, a, a] = 1
    return mask


def cache_case(rs, lens, slots, heads, kv, hd, page, fresh="tree", big=None):
    """Inputs of a call: the pages' unwritten tails hold NaN codes, the pool is scattered."""
    torch = _t()
    n = len(lens)
    held = [-(-int(x) // page) for x in lens]
    n_pages = (big or sum(held)) + 2
    cache = new_cache(rs, sum(held) + 2, kv, page, hd, pow2=rs.rand() < 0.5) if big is None else None
    perm = rs.permutation(sum(held) + 2)
    table, at = np.full((n, max(1, max(held)) + 1), -1), 0
    for q, h in enumerate(held):
        table[q, :h] = perm[at:at + h]
        at += h
        if lens[q] % page:
            for c in (cache.k, cache.v):
                c.view(torch.uint8)[int(table[q, h - 1]), :, int(lens[q] % page):] = 0x7F
    c = dict(cache=cache, table=table, lens=np.array(lens), slots=slots, heads=heads, kv=kv, hd=hd, page=page, n_pages=n_pages)
    c["q"] = dev(rs.randn(n, slots, heads, hd), torch.bfloat16)
    c["k"] = c["v"] = c["mask"] = None
    if fresh:
        c["k"], c["v"] = dev(2 * rs.randn(n, slots, kv, hd), torch.bfloat16), dev(rs.randn(n, slots, kv, hd), torch.bfloat16)
        if fresh == "tree":
            c["mask"] = tree_masks(rs, n, slots)
        elif fresh == "random":  # rows that see nothing among the new tokens included
            c["mask"] = (rs.rand(n, slots, slots) < 0.3).astype(np.uint8) * rs.randint(1, 256, (n, slots, slots)).astype(np.uint8)
            c["mask"][:, ::3] = 0
    return c


def run_cache(c, scale=None, out=None, stream=None, work=None, lse=True, status=None):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, cache_attention
    n = len(c["lens"])
    l = torch.full((n, c["slots"], c["heads"]), 7.0, device="cuda") if lse else None
    out = torch.full((n, c["slots"], c["heads"], c["hd"]), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    args = dict(k_new=c["k"], v_new=c["v"], mask=None if c["mask"] is None else dev(c["mask"], torch.uint8), scale=scale,
                out=out, lse=l, workspace=work or AttentionWorkspace(), stream=stream, status=status)
    table, lens = dev(c["table"], torch.int32), dev(c["lens"], torch.int32)
    torch.cuda.synchronize()
    cache_attention(c["cache"], c["q"], table, lens, **args)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), None if l is None else l.cpu().numpy()


def check_cache(c, got, scale=None, rows=None, skip=()):
    """Against the oracle; rows: only these slots; skip: (request, slot) pairs not compared."""
    out, lse = got
    cache, page = c["cache"], c["page"]
    kc, vc = cache.k.float().cpu().numpy(), cache.v.float().cpu().numpy()
    ks, vs = cache.k_scale.cpu().numpy(), cache.v_scale.cpu().numpy()
    scale = c["hd"] ** -0.5 if scale is None else scale
    g = c["heads"] // c["kv"]
    qf = c["q"].float().cpu().numpy()
    fresh = c["k"] is not None
    if fresh:
        kf, vf = c["k"].float().cpu().numpy(), c["v"].float().cpu().numpy()
    for b, ln in enumerate(c["lens"]):
        pages = c["table"][b, :-(-ln // page)]
        for h in range(c["kv"]):
            k = (kc[pages, h].astype(np.float64) * ks[pages, h][:, None, None]).reshape(-1, c["hd"])[:ln]
            v = (vc[pages, h].astype(np.float64) * vs[pages, h][:, None, None]).reshape(-1, c["hd"])[:ln]
            see = np.ones((c["slots"], ln), bool)
            if fresh:
                k, v = np.concatenate([k, kf[b, :, h]]), np.concatenate([v, vf[b, :, h]])
                m = np.tril(np.ones((c["slots"],) * 2, bool)) if c["mask"] is None else c["mask"][b] != 0
                see = np.concatenate([see, m], 1)
            for j in range(h * g, (h + 1) * g):
                o, l, to, tl = ok.attend(qf[b, :, j], k, v, see, scale, 2.0 ** -11)
                for a in range(c["slots"]) if rows is None else rows:
                    if (b, a) in skip:
                        continue
                    assert (np.abs(out[b, a, j] - o[a]) <= to[a]).all(), (b, a, j, np.abs(out[b, a, j] - o[a]).max(), to[a].max())
                    if lse is not None:
                        if np.isinf(l[a]):
                            assert lse[b, a, j] == l[a] and (out[b, a, j] == 0).all()
                        else:
                            assert abs(lse[b, a, j] - l[a]) <= tl[a], (b, a, j, lse[b, a, j], l[a], tl[a])


CACHE = [
    # lens, slots, heads, kv, hd, page, fresh
    ([1], 1, 1, 1, 64, 16, None),
    ([0, 1, 15, 16, 17], 1, 8, 2, 128, 16, None),
    ([0, 63, 64, 65, 700], 1, 32, 8, 128, 64, "tree"),
    ([129, 0, 1000], 1, 7, 1, 128, 32, None),
    ([300, 5], 1, 6, 2, 64, 128, "tree"),
    ([2000], 1, 16, 1, 128, 64, None),
    ([255, 256, 257], 2, 8, 2, 128, 128, "tree"),
    ([100, 0, 3], 5, 9, 3, 64, 16, "random"),
    ([40, 0], 4, 16, 4, 128, 32, "causal"),
    ([500], 4, 4, 1, 128, 64, None),
    ([0, 1, 64, 200], 17, 8, 2, 128, 16, "tree"),
    ([127, 128, 129], 65, 8, 2, 128, 64, "tree"),
    ([130, 0], 65, 10, 2, 64, 32, "random"),
    ([1500], 33, 4, 4, 128, 128, "causal"),
    ([260], 129, 3, 1, 128, 64, "tree"),
    ([0, 70], 130, 5, 5, 64, 64, "random"),
    ([513], 70, 12, 4, 64, 32, None),
    ([90], 20, 48, 1, 128, 16, "tree"),
]


@pytest.mark.parametrize("lens,slots,heads,kv,hd,page,fresh", CACHE)
def test_cache_attention(lens, slots, heads, kv, hd, page, fresh):
    c = cache_case(np.random.RandomState(len(lens) * 1000 + slots), lens, slots, heads, kv, hd, page, fresh)
    check_cache(c, run_cache(c))


def test_cache_attention_wide_tree():
    c = cache_case(np.random.RandomState(11), [700], 513, 8, 2, 128, 64, "tree")
    check_cache(c, run_cache(c), rows=[0, 1, 31, 32, 63, 64, 127, 128, 300, 511, 512])


@pytest.mark.parametrize("slots", [1, 40])
def test_cache_attention_scales_and_signs(slots):
    """A softmax scale of zero (plain means), a negative and a large one."""
    c = cache_case(np.random.RandomState(12), [77, 300], slots, 4, 2, 128, 32, "tree")
    for scale in (0.0, -0.05, 1.0):
        check_cache(c, run_cache(c, scale=scale), scale=scale)


@pytest.mark.parametrize("slots", [1, 40])
def test_cache_attention_extreme_page_scales(slots):
    """Pages whose scales lie far apart, zero pages among them (scale 2^-126)."""
    torch = _t()
    c = cache_case(np.random.RandomState(13), [200, 130], slots, 8, 2, 128, 16, "tree")
    cache = c["cache"]
    rs = np.random.RandomState(14)
    cache.k_scale.copy_(dev(np.ldexp(1.0, rs.randint(-30, -6, cache.k_scale.shape)), torch.float32))
    cache.v_scale.copy_(dev(np.ldexp(1.0, rs.choice([-126, -60, -20, -8, 0, 40], cache.v_scale.shape)), torch.float32))
    check_cache(c, run_cache(c))


@pytest.mark.parametrize("slots", [1, 5, 65])
def test_cache_attention_repeats_itself(slots):
    """The same bits again and again from one workspace, other sizes between (split requests join in a fixed order)."""
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace
    work = AttentionWorkspace()
    c = cache_case(np.random.RandomState(15), [3000, 10, 0, 900], slots, 8, 2, 128, 64, "tree")
    d = cache_case(np.random.RandomState(16), [50, 1000], slots + 2, 8, 4, 64, 16, "tree")
    first = run_cache(c, work=work)
    check_cache(c, first)
    for _ in range(3):
        check_cache(d, run_cache(d, work=work))
        again = run_cache(c, work=work)
        np.testing.assert_array_equal(first[0], again[0])
        np.testing.assert_array_equal(first[1], again[1])


@pytest.mark.parametrize("slots", [1, 30])
def test_cache_attention_strides_and_stream(slots):
    """q, k and v as slices of one projection, a strided output, another stream, no lse."""
    torch = _t()
    c = cache_case(np.random.RandomState(17), [90, 33], slots, 6, 2, 128, 32, "causal")
    n = 2
    qkv = torch.randn(n, slots, 6 + 2 + 2 + 1, 128, device="cuda").to(torch.bfloat16)
    c["q"], c["k"], c["v"] = qkv[:, :, :6], qkv[:, :, 6:8], qkv[:, :, 8:10]
    # heads of the output lie further apart than rows of it
    out = torch.full((6, n, slots, 128), 7.0, dtype=torch.bfloat16, device="cuda").permute(1, 2, 0, 3)
    st = torch.cuda.Stream()
    got, _ = run_cache(c, out=out, stream=st, lse=False)
    check_cache(c, (got, None))
    assert (qkv[:, :, 10] == qkv[:, :, 10]).all()


@pytest.mark.parametrize("slots", [4, 40])
def test_cache_attention_nan_in_masked_tokens(slots):
    """NaN and infinities in new tokens reach only the rows that see them."""
    torch = _t()
    rs = np.random.RandomState(18)
    c = cache_case(rs, [50, 0, 200], slots, 8, 2, 128, 64, "random")
    bad = {(0, 1): float("nan"), (1, 2): float("inf"), (2, slots - 1): float("-inf")}
    skip = set()
    for (b, s), val in bad.items():
        c["v"][b, s, :, 5] = val
        c["k"][b, s, 0, 7] = val
        skip |= {(b, a) for a in range(slots) if c["mask"][b, a, s]}
    out, lse = run_cache(c)
    clean = dict(c, k=c["k"].nan_to_num(0, 0, 0), v=c["v"].nan_to_num(0, 0, 0))
    check_cache(clean, (out, lse), skip=skip)
    assert skip
    for b, a in skip:
        assert not np.isfinite(out[b, a, :, 5]).any()


# 32 and more key/value heads over all requests, rows behind pairs of full 128-row tiles: up to 16 of them are streamed
REST = [
    ([0, 1, 130, 64, 500, 3, 90, 257], 65, 16, 4, 128, 64, "tree"),     # 4 rows left
    ([0, 1, 130, 64, 500, 3, 90, 257], 34, 32, 4, 64, 16, "random"),    # 16 rows
    ([40, 300, 0, 129], 259, 8, 8, 128, 32, "causal"),                  # 3 rows of single heads
    ([40, 300, 0, 129], 66, 32, 8, 128, 128, None),                     # 8 rows, cached tokens only
    ([700, 20, 0, 33], 69, 32, 8, 128, 64, "random"),                   # 20 rows: a tile of their own
    ([65] * 33, 129, 4, 1, 64, 64, "random"),                           # behind two pairs
]


@pytest.mark.parametrize("lens,slots,heads,kv,hd,page,fresh", REST)
def test_cache_attention_rows_left_over(lens, slots, heads, kv, hd, page, fresh):
    c = cache_case(np.random.RandomState(len(lens) * 2000 + slots), lens, slots, heads, kv, hd, page, fresh)
    check_cache(c, run_cache(c), rows=[0, 1, 31, slots // 2, *range(slots - 6, slots)])


def test_cache_attention_rows_left_over_nan():
    torch = _t()
    rs = np.random.RandomState(41)
    slots = 66
    c = cache_case(rs, [50, 0, 200, 9], slots, 32, 8, 128, 64, "random")
    skip = set()
    for (b, s), val in {(0, 1): float("nan"), (1, 40): float("inf"), (2, slots - 1): float("-inf")}.items():
        c["v"][b, s, :, 5] = val
        c["k"][b, s, 0, 7] = val
        c["mask"][b, slots - 1, s] = b != 2  # the last row sees two of them, the one before it the third
        c["mask"][b, slots - 2, s] = b == 2
        skip |= {(b, a) for a in range(slots) if c["mask"][b, a, s]}
    out, lse = run_cache(c)
    clean = dict(c, k=c["k"].nan_to_num(0, 0, 0), v=c["v"].nan_to_num(0, 0, 0))
    check_cache(clean, (out, lse), skip=skip, rows=[0, 2, slots - 3, slots - 2, slots - 1])
    for b, a in skip:
        assert not np.isfinite(out[b, a, :, 5]).any()


def test_cache_attention_rows_left_over_repeats():
    """Both kernels of a call in one workspace, again and again, next to calls of other kinds."""
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace
    work = AttentionWorkspace()
    rs = np.random.RandomState(42)
    c = cache_case(rs, [3000, 10, 0, 900], 65, 32, 8, 128, 64, "tree")
    d = cache_case(rs, [50, 1000, 7], 1, 8, 4, 64, 16, "tree")
    first = run_cache(c, work=work)
    check_cache(c, first, rows=[0, 63, 64])
    for _ in range(5):
        check_cache(d, run_cache(d, work=work))
        again = run_cache(c, work=work)
        np.testing.assert_array_equal(first[0], again[0])
        np.testing.assert_array_equal(first[1], again[1])


def test_cache_attention_bad_pages_count_as_absent():
    torch = _t()
    for slots in (1, 30):
        c = cache_case(np.random.RandomState(19), [100, 64], slots, 4, 2, 128, 32, "tree")
        want = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
        # request 1's second page is out of range: as if it held its first 32 tokens only
        c["table"][1, 1] = 10 ** 6
        want["lens"] = np.array([100, 32])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_cache(c, status=status)
        assert status.item() == ok.BAD_INDEX
        check_cache(want, got)


def test_cache_attention_behind_32_bits():
    """Pages whose bytes stand beyond 2^32."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import KvCache, kv_append
    n_pages, kv, page, hd = 70000, 8, 64, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    cache = KvCache.empty(n_pages, page, kv, hd)
    rs = np.random.RandomState(20)
    for slots in (1, 20):
        table = np.array([[n_pages - 1, 3, n_pages - 2]])
        ln = 150
        x, y = dev(rs.randn(ln, kv, hd), torch.bfloat16), dev(rs.randn(ln, kv, hd), torch.bfloat16)
        kv_append(cache, x, y, dev([table[0, p // page] * page + p % page for p in range(ln)], torch.int64))
        sub = sorted(set(table[0].tolist()))
        c = cache_case(rs, [ln], slots, 16, kv, hd, page, "tree")
        small = KvCache(cache.k[sub].clone(), cache.v[sub].clone(), cache.k_scale[sub].clone(), cache.v_scale[sub].clone())
        c["cache"], c["table"] = cache, table
        got = run_cache(c)
        check_cache(dict(c, cache=small, table=np.array([[sub.index(t) for t in table[0]]])), got)


def test_cache_attention_refusals():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, DtreeError, KvCache, cache_attention, kv_append
    c = cache_case(np.random.RandomState(21), [20], 3, 4, 2, 64, 16, "tree")
    w = AttentionWorkspace()
    t, ln, m = dev(c["table"], torch.int32), dev(c["lens"], torch.int32), dev(c["mask"], torch.uint8)
    good = dict(k_new=c["k"], v_new=c["v"], mask=m, workspace=w)
    for kw, err in ((dict(q=c["q"].float()), TypeError), (dict(q=c["q"].cpu()), ValueError),
                    (dict(q=c["q"][:, :, :3]), DtreeError),                       # 3 heads over 2
                    (dict(q=c["q"][..., :32]), ValueError),
                    (dict(q=c["q"].transpose(2, 3).contiguous().transpose(2, 3)), ValueError),
                    (dict(v_new=None), ValueError), (dict(k_new=c["k"][:, :2]), ValueError),
                    (dict(k_new=None, v_new=None), DtreeError),                  # a mask without new keys
                    (dict(mask=m.bool()), TypeError), (dict(mask=m[:, :2]), ValueError),
                    (dict(length=ln.long()), TypeError), (dict(scale=float("nan")), DtreeError),
                    (dict(scale=float("inf")), DtreeError), (dict(lse=torch.zeros(3, device="cuda")), ValueError)):
        a = dict(good, q=c["q"], length=ln) | kw
        q, length = a.pop("q"), a.pop("length")
        with pytest.raises(err):
            cache_attention(c["cache"], q, t, length, **a)
    off = torch.empty(1, 3, 4, 72, dtype=torch.bfloat16, device="cuda")[..., 4:68]  # heads 8 bytes off 16
    with pytest.raises(DtreeError):
        cache_attention(c["cache"], off, t, ln, **good)
    with pytest.raises(DtreeError):
        KvBad = KvCache.empty(4, 48, 2, 64)
        kv_append(KvBad, c["k"], c["v"], dev([0], torch.int64))
    with pytest.raises(ValueError):
        kv_append(c["cache"], c["k"], c["v"], dev([0, 1, 2, 3], torch.int64))  # more rows than k has
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------
def run_prompt(q, k, v, lens, scale=None, out=None, stream=None, first=0):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import prompt_attention
    rows, heads, hd = q.shape
    start = dev(first + np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    lse = torch.full((rows, heads), 7.0, device="cuda")
    out = torch.full((rows, heads, hd), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    torch.cuda.synchronize()
    prompt_attention(q, k, v, start, scale=scale, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def check_prompt(q, k, v, lens, got, scale=None, first=0, skip=(), sample=None):
    out, lse = got
    heads, hd = q.shape[1:]
    g = heads // k.shape[1]
    scale = hd ** -0.5 if scale is None else scale
    qf, kf, vf = (x.float().cpu().numpy() for x in (q, k, v))
    a = first
    for ln in lens:
        rows = np.arange(ln) if sample is None else np.unique(np.clip(np.array(sample), 0, max(ln - 1, 0)))[:ln]
        for h in range(heads) if sample is None else (0, heads // 2, heads - 1):
            if len(rows) == 0:
                continue
            see = np.arange(ln) <= rows[:, None]
            o, l, to, tl = ok.attend(qf[a + rows, h], kf[a:a + ln, h // g], vf[a:a + ln, h // g], see, scale, 2.0 ** -8)
            for i, r in enumerate(rows):
                if a + r in skip:
                    continue
                assert (np.abs(out[a + r, h] - o[i]) <= to[i]).all(), (a, r, h, np.abs(out[a + r, h] - o[i]).max(), to[i].max())
                assert abs(lse[a + r, h] - l[i]) <= tl[i], (a, r, h)
        a += ln


PROMPTS = [
    ([1], 1, 1, 64), ([1, 0, 2], 4, 2, 128), ([17], 8, 2, 128), ([0, 5, 0, 31, 32, 33, 0], 4, 1, 128),
    ([64, 65, 63], 2, 2, 64), ([127, 128, 129], 4, 4, 128), ([255, 257], 6, 2, 128), ([300], 32, 8, 128),
    ([130, 7], 10, 2, 64), ([90, 40], 7, 1, 128), ([200], 48, 1, 64), ([33, 1, 1, 1, 70], 24, 8, 128), ([260], 100, 1, 64),
]


@pytest.mark.parametrize("lens,heads,kv,hd", PROMPTS)
def test_prompt_attention(lens, heads, kv, hd):
    torch = _t()
    rs = np.random.RandomState(sum(lens) + heads)
    n = sum(lens)
    q, k, v = (dev(rs.randn(n, x, hd) * s, torch.bfloat16) for x, s in ((heads, 1), (kv, 2), (kv, 1)))
    check_prompt(q, k, v, lens, run_prompt(q, k, v, lens))


def test_prompt_attention_long():
    torch = _t()
    rs = np.random.RandomState(30)
    lens = [3001, 1500]
    q, k, v = (dev(rs.randn(sum(lens), x, 128), torch.bfloat16) for x in (8, 2, 2))
    got = run_prompt(q, k, v, lens)
    check_prompt(q, k, v, lens, got, sample=[0, 1, 127, 128, 129, 255, 256, 1000, 1499, 1535, 2047, 2048, 2999, 3000])


def test_prompt_attention_strides_stream_scale():
    """Slices of one projection, a head-major output, rows before and behind the sequences left alone."""
    torch = _t()
    rs = np.random.RandomState(31)
    lens, first = [100, 37], 5
    n = sum(lens) + 12
    qkv = dev(rs.randn(n, 6 + 2 + 2, 128), torch.bfloat16)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    for scale in (0.0, -0.07, 0.5):
        out = torch.full((6, n, 128), 7.0, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
        got = run_prompt(q, k, v, lens, scale=scale, out=out, stream=torch.cuda.Stream(), first=first)
        check_prompt(q, k, v, lens, got, scale=scale, first=first)
        assert (got[0][:first] == 7).all() and (got[0][first + 137:] == 7).all() and (got[1][first + 137:] == 7).all()


def test_prompt_attention_nan_stays_where_it_is_seen():
    """NaN and infinities of later rows and of other sequences do not reach a row."""
    torch = _t()
    rs = np.random.RandomState(32)
    lens = [50, 140, 60]
    q, k, v = (dev(rs.randn(250, x, 128), torch.bfloat16) for x in (4, 2, 2))
    clean = [x.clone() for x in (q, k, v)]
    skip = set()
    for row, end, val in ((30, 50, float("nan")), (50 + 129, 190, float("inf")), (190 + 59, 250, float("-inf"))):
        v[row, :, 3] = val
        k[row, 0, 9] = val
        skip |= set(range(row, end))
    out, lse = run_prompt(q, k, v, lens)
    check_prompt(*clean, lens, (out, lse), skip=skip)
    for r in skip:
        assert not np.isfinite(out[r, :, 3]).any(), r


def test_prompt_attention_many_short_sequences_again_and_again():
    """Most items have one row tile of two, so that the two softmax groups of a CTA are often items apart; the same
    bits in every pass, and no wait that gives up (it would leave rows unwritten)."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import prompt_attention
    rs = np.random.RandomState(35)
    lens = np.concatenate([rs.randint(1, 33, 3000), [700, 290, 0, 65]])
    rs.shuffle(lens)
    n = int(lens.sum())
    q, k, v = (dev(rs.randn(n, x, 128), torch.bfloat16) for x in (8, 2, 2))
    start = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    first = run_prompt(q, k, v, lens)
    some = np.concatenate([[0], np.cumsum(lens)])
    for i in list(range(0, 3004, 301)) + [int(np.argmax(lens))]:
        part = (first[0][some[i]:some[i + 1]], first[1][some[i]:some[i + 1]])
        check_prompt(q[some[i]:some[i + 1]], k[some[i]:some[i + 1]], v[some[i]:some[i + 1]], [int(lens[i])], part)
    want = torch.from_numpy(first[0]).cuda()
    for _ in range(100):
        out = torch.full((n, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        prompt_attention(q, k, v, start, out=out)
        assert torch.equal(out.float(), want)


def test_prompt_attention_large_logits():
    """Maxima that rise along the keys, so that the running sums are rescaled again and again, and logits in the hundreds."""
    torch = _t()
    rs = np.random.RandomState(33)
    n = 700
    q = dev(np.ones((n, 2, 128)) + 0.1 * rs.randn(n, 2, 128), torch.bfloat16)
    k = dev(np.linspace(-20, 20, n)[:, None, None] * np.ones((1, 1, 128)) + 0.1 * rs.randn(n, 1, 128), torch.bfloat16)
    v = dev(rs.randn(n, 1, 128), torch.bfloat16)
    check_prompt(q, k, v, [n], run_prompt(q, k, v, [n]), sample=list(range(0, n, 23)) + [n - 1])


def test_prompt_attention_behind_32_bits():
    """Rows whose elements stand beyond 2^32 bytes."""
    torch = _t()
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB")
    rs = np.random.RandomState(34)
    n, stride = 300, 1 << 23
    buf = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    view = buf.view(n, stride)[:, :8 * 128].view(n, 8, 128)
    view.copy_(dev(rs.randn(n, 8, 128), torch.bfloat16))
    q, k, v = view[:, :4], view[:, 4:6], view[:, 6:8]
    check_prompt(q, k, v, [n], run_prompt(q, k, v, [n]), sample=[0, 100, 255, 256, 299])


def test_prompt_attention_refusals():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import DtreeError, prompt_attention
    q, k = torch.zeros(10, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(10, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = dev([0, 10], torch.int32)
    for a, err in (((q.float(), k, k, s), TypeError), ((q, k[:9], k, s), ValueError), ((q, k, k, s.long()), TypeError),
                   ((q[:, :3], k, k, s), DtreeError), ((q[..., :48], k[..., :48], k[..., :48], s), DtreeError),
                   ((q, k, k, s[:1]), DtreeError), ((q.cpu(), k, k, s), ValueError)):
        with pytest.raises(err):
            prompt_attention(*a)
    with pytest.raises(DtreeError):
        prompt_attention(q, k, k, s, scale=float("inf"))
    torch.cuda.synchronize()
