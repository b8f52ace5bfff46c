"""Measured cases of the operators around the target model's key/value cache.

Four operators, in the order in which a serving loop calls them: the page plan (block tables and
slot maps from request lengths), the append that holds keys and values in 8 bits with one scale for
each page and head, causal attention over packed prompts, and attention of new tokens (one token, or
a drafted tree under its ancestor-only mask) over that cache.

``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is true, through
``conditional_draft_tree_lm_gb300``.  ``exact`` states each definition once more in 64 bits.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
DEV = "cuda"

# DT_KV_* bits of the plan's status word
SHORT_OF_PAGES, BAD_LENGTH, SHORT_OF_ROWS, BAD_PATH = 1, 2, 4, 8


def listed():
    return [
        # a verification round's commit: 32 requests take the root and 0 to 15 accepted tree slots
        dict(name="plan_commit", op="plan", req=32, page=64, ctx=4096, new=16, tree=65, ends=False),
        # admission of 256 prompts of up to 2048 tokens while other requests end and give pages back
        dict(name="plan_prompts", op="plan", req=256, page=32, ctx=4096, new=2048, tree=0, ends=True),
        # plain decoding, one new token in each of 32 requests, in pages that already hold tokens
        dict(name="append_token", op="append", req=32, new=1, ctx=4000, page=64, kv=8, hd=128, tree=0),
        # the accepted slots of 32 verified 65-slot trees
        dict(name="append_commit", op="append", req=32, new=16, ctx=4000, page=64, kv=8, hd=128, tree=65),
        # 16 prompts of up to 4096 tokens, ragged
        dict(name="append_prompts", op="append", req=16, new=4096, ctx=0, page=64, kv=8, hd=128, tree=0),
        # one user, one token, a short conversation: latency
        dict(name="token_1x2k", op="attend", req=1, slots=1, ctx=2047, heads=32, kv=8, hd=128, page=64, fresh=False),
        # 32 users decoding over ragged contexts of up to 16k tokens: bandwidth
        dict(name="token_32x16k", op="attend", req=32, slots=1, ctx=16384, heads=32, kv=8, hd=128, page=64, fresh=True),
        # verification of 32 trees of 64 nodes and their roots
        dict(name="tree_32x4k", op="attend", req=32, slots=65, ctx=4096, heads=32, kv=8, hd=128, page=64, fresh=True),
        # verification of the wide tree, 512 nodes and the root, over a long context
        dict(name="wide_1x32k", op="attend", req=1, slots=513, ctx=32768, heads=32, kv=8, hd=128, page=64, fresh=True),
        # one short prompt: latency
        dict(name="prompt_1x300", op="prompt", req=1, longest=300, heads=32, kv=8, hd=128),
        # 48 ragged prompts in one packed batch
        dict(name="prompt_48x1k", op="prompt", req=48, longest=1024, heads=32, kv=8, hd=128),
        # one long document
        dict(name="prompt_1x16k", op="prompt", req=1, longest=16384, heads=32, kv=8, hd=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), kv, rng.choice([64, 128, 128])


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        tree = rng.choice([0, 17, 65, 129])
        return dict(op=op, req=_log_int(rng, 1, 512), page=page, ctx=_log_int(rng, 16, 8192),
                    new=rng.randint(1, 16) if tree else _log_int(rng, 1, 2048), tree=tree, ends=rng.random() < 0.5)
    if op == "append":
        _, kv, hd = _heads(rng)
        tree = rng.choice([0, 0, 65, 129])
        return dict(op=op, req=_log_int(rng, 1, 64), new=rng.randint(1, 16) if tree else _log_int(rng, 1, 1024),
                    ctx=rng.choice([0, _log_int(rng, 1, 4096)]), page=page, kv=kv, hd=hd, tree=tree)
    if op == "attend":
        heads, kv, hd = _heads(rng)
        slots = rng.choice([1, 1, 2, 5, 17, 65, 129, 513])
        ctx = _log_int(rng, 1, 32768)
        # at most 2^29 logits in all, so that a drawn case stays below the largest listed ones
        req = max(1, min(_log_int(rng, 1, 64), (1 << 29) // (slots * heads * (ctx + slots)), (1 << 22) // (ctx * kv)))
        return dict(op=op, req=req, slots=slots, ctx=ctx, heads=heads, kv=kv, hd=hd, page=page,
                    fresh=slots > 1 or rng.random() < 0.5)
    heads, kv, hd = _heads(rng)
    longest = _log_int(rng, 1, 8192)
    req = max(1, min(_log_int(rng, 1, 64), (1 << 31) // (heads * longest * longest)))
    return dict(op=op, req=req, longest=longest, heads=heads, kv=kv, hd=hd)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(rs, n, longest, shortest=0):
    """Ragged lengths from a quarter of `longest` to all of it, in an order of the seed's."""
    x = np.linspace(max(shortest, longest // 4), longest, n) if n > 1 else np.array([longest])
    return rs.permutation(np.floor(x).astype(np.int64))


def _blocks(x, page):
    return -(-x // page)


def _tables(rs, held, width, n_pages):
    """Block tables whose pages are scattered over the pool, and the pages that are left."""
    perm = rs.permutation(n_pages).astype(np.int32)
    table = np.full((len(held), width), -1, np.int32)
    at = 0
    for q, h in enumerate(held):
        table[q, :h] = perm[at:at + h]
        at += h
    return table, perm[at:]


def _dev(x, dtype):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).to(DEV)


def _accepted(rs, n, depth, slots, width):
    """Accepted slots of `n` verified trees as the acceptance walk writes them: ascending, padded with -1."""
    lens = np.minimum(rs.geometric(0.25, n) - 1, depth)
    path = np.full((n, width), -1, np.int64)
    for q, a in enumerate(lens):
        path[q, :a] = np.sort(rs.choice(np.arange(1, slots), a, replace=False))
    return lens.astype(np.int64), path


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _keys(g, rows, kv, hd):
    """Keys with a few channels that stand out, as rotary models have them."""
    k = _normal(g, rows, kv, hd)
    k *= 1 + 4 * (torch.rand(1, kv, hd, generator=g, device=DEV) > 0.95)
    return k.to(torch.bfloat16)


def _values(g, rows, kv, hd):
    return (0.5 * _normal(g, rows, kv, hd)).to(torch.bfloat16)


def prepare(case, seed):
    rs = np.random.RandomState(seed & 0x7FFFFFFF)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "plan":
        _prepare_plan(s, case, rs)
    elif case["op"] == "append":
        _prepare_append(s, case, rs, g)
    elif case["op"] == "attend":
        _prepare_attend(s, case, rs, g)
    else:
        _prepare_prompt(s, case, rs, g)
    return s


def _prepare_plan(s, c, rs):
    n, page, tree = c["req"], c["page"], c["tree"]
    old = rs.randint(0, c["ctx"] + 1, n)
    if tree:
        delta, path = _accepted(rs, n, c["new"] - 1, tree, c["new"] - 1 or 1)
        s["path"], extra = _dev(path, torch.int32), 1
    else:
        delta, extra = rs.randint(max(1, c["new"] // 8), c["new"] + 1, n), 0
        if c["new"] > 64:  # prompts come to requests that hold nothing yet
            old = np.where(rs.rand(n) < 0.75, 0, old)
    if c["ends"]:
        delta = np.where((rs.rand(n) < 0.25) & (old > 0), -old, delta)
    width = _blocks(c["ctx"] + c["new"], page) + 1
    # a pool with room for every request at its longest, rounded to whole powers of two as servers size it
    n_pages = 1 << int(np.ceil(np.log2(n * width + 8)))
    table, left = _tables(rs, _blocks(old, page), width, n_pages)
    ring = np.concatenate([left, np.full(n_pages - len(left), -1, np.int32)])
    head = int(rs.randint(n_pages))
    s["max_rows"] = n * c["new"]
    s["page"], s["extra"], s["path_rows"] = page, extra, tree
    s["old"], s["delta"] = _dev(old, torch.int32), _dev(delta, torch.int32)
    s["table"], s["ring"] = _dev(table, torch.int32), _dev(np.roll(ring, head), torch.int32)
    s["ring_in"] = _dev([head, len(left)], torch.int32)
    # what the caller keeps for the answers
    s["len"], s["ring_out"] = torch.zeros_like(s["old"]), torch.zeros_like(s["ring_in"])
    s["row_start"] = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    s["slot_map"] = torch.zeros(s["max_rows"], dtype=torch.int64, device=DEV)
    s["positions"] = torch.zeros(s["max_rows"], dtype=torch.int32, device=DEV)
    s["src_rows"] = torch.zeros(s["max_rows"], dtype=torch.int32, device=DEV) if tree else None
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)


def _handle(s):
    """The cache handle and the workspace that a server keeps between calls."""
    if own:
        from conditional_draft_tree_lm_gb300 import AttentionWorkspace, KvCache
        s["cache"] = KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if s["op"] == "attend":
            s["work"] = AttentionWorkspace()


def _prepare_append(s, c, rs, g):
    n, page, kv, hd = c["req"], c["page"], c["kv"], c["hd"]
    old = _lengths(rs, n, c["ctx"])
    if c["tree"]:
        acc, path = _accepted(rs, n, c["new"] - 1, c["tree"], c["new"] - 1 or 1)
        cnt, rows_in = acc + 1, n * c["tree"]
    else:
        cnt = _lengths(rs, n, c["new"], 1)
        rows_in = int(cnt.sum())
    held = _blocks(old + cnt, page)
    width = _blocks(c["ctx"] + c["new"], page)
    n_pages = n * width + 3
    table, _ = _tables(rs, held, width, n_pages)
    rows = n * c["new"] if c["tree"] else rows_in
    slot, src = np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    at = 0
    for q in range(n):
        p = old[q] + np.arange(cnt[q])
        slot[at:at + cnt[q]] = table[q, p // page].astype(np.int64) * page + p % page
        if c["tree"]:
            src[at:at + cnt[q]] = q * c["tree"] + np.concatenate([[0], path[q, :cnt[q] - 1]])
        at += cnt[q]
    s["page"], s["req"] = page, n
    s["slot_map"] = _dev(slot, torch.int64)
    s["src_rows"] = _dev(src, torch.int32) if c["tree"] else None
    s["k_new"], s["v_new"] = _keys(g, rows_in, kv, hd), _values(g, rows_in, kv, hd)
    # earlier tokens under scales that the new ones exceed in about half of the pages
    s["k"] = (100 * _normal(g, n_pages, kv, page, hd)).clamp(-448, 448).to(F8)
    s["v"] = (100 * _normal(g, n_pages, kv, page, hd)).clamp(-448, 448).to(F8)
    s["k_scale"] = torch.exp2(torch.randint(-8, -3, (n_pages, kv), generator=g, device=DEV).float())
    s["v_scale"] = torch.exp2(torch.randint(-10, -5, (n_pages, kv), generator=g, device=DEV).float())
    _handle(s)


def _prepare_attend(s, c, rs, g):
    n, page, kv, hd, slots, heads = c["req"], c["page"], c["kv"], c["hd"], c["slots"], c["heads"]
    length = _lengths(rs, n, c["ctx"], 0 if c["fresh"] else 1)
    held = _blocks(length, page)
    n_pages = int(held.sum()) + 3
    table, _ = _tables(rs, held, max(1, int(held.max())), n_pages)
    s["page"], s["length"], s["table"] = page, _dev(length, torch.int32), _dev(table, torch.int32)
    # tokens in 8 bits; every value of a page's unwritten tail is a NaN, as memory that was used for something else may be
    k = (110 * _normal(g, n_pages, kv, page, hd)).clamp(-448, 448).to(F8)
    v = (110 * _normal(g, n_pages, kv, page, hd)).clamp(-448, 448).to(F8)
    for q in range(n):
        if length[q] % page:
            for t in (k, v):
                t.view(torch.uint8)[int(table[q, held[q] - 1]), :, int(length[q] % page):] = 0x7F
    s["k"], s["v"] = k, v
    s["k_scale"] = torch.exp2(torch.randint(-8, -5, (n_pages, kv), generator=g, device=DEV).float())
    s["v_scale"] = torch.exp2(torch.randint(-9, -6, (n_pages, kv), generator=g, device=DEV).float())
    s["q"] = _normal(g, n * slots, heads, hd).to(torch.bfloat16).view(n, slots, heads, hd)
    s["scale"] = hd ** -0.5
    s["mask"] = s["k_new"] = s["v_new"] = None
    if c["fresh"]:
        s["k_new"] = _keys(g, n * slots, kv, hd).view(n, slots, kv, hd)
        s["v_new"] = _values(g, n * slots, kv, hd).view(n, slots, kv, hd)
        # a drafted tree: each slot's parent is one of the slots shortly before it
        parent = np.maximum(np.arange(slots) - 1 - rs.randint(0, 8, (n, slots)), 0)
        mask = np.zeros((n, slots, slots), np.uint8)
        mask[:, 0, 0] = 1
        for a in range(1, slots):
            mask[:, a] = mask[np.arange(n), parent[:, a]]
            mask[:, a, a] = 1
        s["mask"] = _dev(mask, torch.uint8)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(n, slots, heads, dtype=torch.float32, device=DEV)
    _handle(s)


def _prepare_prompt(s, c, rs, g):
    n, kv, hd, heads = c["req"], c["kv"], c["hd"], c["heads"]
    length = _lengths(rs, n, c["longest"], 1)
    start = np.concatenate([[0], np.cumsum(length)])
    rows = int(start[-1])
    s["longest"], s["row_start"] = c["longest"], _dev(start, torch.int32)
    s["q"] = _normal(g, rows, heads, hd).to(torch.bfloat16)
    s["k"], s["v"] = _keys(g, rows, kv, hd), _values(g, rows, kv, hd)
    s["scale"] = hd ** -0.5
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(rows, heads, dtype=torch.float32, device=DEV)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"plan": _plan, "append": _append, "attend": _attend, "prompt": _prompt}[s["op"]](s)


def _plan(s):
    if own:
        from conditional_draft_tree_lm_gb300 import kv_plan
        kv_plan(s["old"], s["len"], s["table"], s["ring"], s["ring_in"], s["ring_out"], s["row_start"],
                s["slot_map"], s["status"], page=s["page"], delta=s["delta"], extra=s["extra"],
                positions=s["positions"], path=s.get("path"), path_rows=s["path_rows"], src_rows=s["src_rows"])
        return _plan_answer(s["len"], s["table"], s["ring"], s["ring_out"], s["row_start"], s["slot_map"],
                            s["positions"], s["src_rows"], s["status"])
    page, table, ring, n_pages, cap = s["page"], s["table"], s["ring"], s["ring"].numel(), s["max_rows"]
    old = s["old"].long()
    new = (old + s["delta"] + s["extra"]).clamp(min=0)
    held, want = (old + page - 1).div(page, rounding_mode="floor"), (new + page - 1).div(page, rounding_mode="floor")
    take, give, rows = (want - held).clamp(min=0), (held - want).clamp(min=0), (new - old).clamp(min=0)
    head, count = s["ring_in"][0].long(), s["ring_in"][1].long()
    bad = (take.sum() > count) * SHORT_OF_PAGES + (torch.maximum(held, want) > table.shape[1]).any() * BAD_LENGTH
    bad = bad + (rows.sum() > cap) * SHORT_OF_ROWS
    if s["path_rows"]:
        depth = torch.arange(s["path"].shape[1], device=DEV)
        off = (depth < rows[:, None] - 1) & ((s["path"] < 0) | (s["path"] >= s["path_rows"]))
        bad = bad + (off.any() | (rows - 1 > s["path"].shape[1]).any()) * BAD_PATH
    ok = bad == 0
    new, want = torch.where(ok, new, old), torch.where(ok, want, held)
    take, give, rows = take * ok, give * ok, rows * ok
    # pages leave the ring at its head in the order of requests, and come back behind its last one
    block = torch.arange(table.shape[1], device=DEV)
    nth = (take.cumsum(0) - take)[:, None] + block - held[:, None]
    comes = (block >= held[:, None]) & (block < want[:, None])
    full = torch.where(comes, ring[(head + nth) % n_pages], table)
    nth = (give.cumsum(0) - give)[:, None] + block - want[:, None]
    goes = (block >= want[:, None]) & (block < held[:, None])
    at = torch.where(goes, (head + count + nth) % n_pages, n_pages)
    ring = torch.cat([ring, ring[:1]]).scatter(0, at.view(-1), table.view(-1))[:n_pages]
    # rows of the new tokens, packed in the order of requests
    start = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    row = torch.arange(cap, device=DEV)
    req = torch.searchsorted(start[1:], row, right=True).clamp(max=old.numel() - 1)
    live, nth = row < start[-1], row - start[req]
    pos = torch.where(live, old[req] + nth, -1)
    slot = torch.where(live, full[req, pos.clamp(min=0).div(page, rounding_mode="floor")].long() * page + pos % page, -1)
    src = None
    if s["path_rows"]:
        step = s["path"][req, (nth - 1).clamp(0, s["path"].shape[1] - 1)]
        src = torch.where(live, req * s["path_rows"] + torch.where(nth > 0, step, 0), -1).int()
    after = torch.stack([(head + take.sum()) % n_pages, count - take.sum() + give.sum()])
    return _plan_answer(new.int(), full, ring, after.int(), start.int(), slot, pos.int(), src, bad.int().view(1))


def _plan_answer(length, table, ring, ring_out, row_start, slot_map, positions, src_rows, status):
    return dict(length=length, table=table, ring=ring, ring_out=ring_out, row_start=row_start, slot_map=slot_map,
                positions=positions, src_rows=src_rows, status=status)


def _append(s):
    if own:
        from conditional_draft_tree_lm_gb300 import kv_append
        kv_append(s["cache"], s["k_new"], s["v_new"], s["slot_map"], src_rows=s["src_rows"])
    else:
        _append_plain(s, s["k"], s["k_scale"], s["k_new"])
        _append_plain(s, s["v"], s["v_scale"], s["v_new"])
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _append_plain(s, codes, scale, x):
    page, slot = s["page"], s["slot_map"]
    n_pages, kv, _, hd = codes.shape
    rows = slot.numel()
    x = x.float() if s["src_rows"] is None else x[s["src_rows"].clamp(min=0)].float()
    live = slot >= 0
    pg, off = torch.where(live, slot.div(page, rounding_mode="floor"), n_pages), slot % page
    # the pages touched, one entry for each, of which there are no more than this
    most = rows // page + 2 * s["req"]
    leads = live & torch.cat([live.new_ones(1), pg[1:] != pg[:-1]])
    nth = leads.long().cumsum(0) - 1
    pages = pg.new_full((most + 1,), n_pages).scatter(0, torch.where(leads, nth, most), torch.where(leads, pg, n_pages))[:most]
    first = off.new_zeros(most + 1).scatter(0, torch.where(leads, nth, most), off)[:most]
    nth = torch.where(live, nth, most)
    # the largest finite magnitude of the new tokens gives the smallest power of two that holds it in 448
    size = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    top = size.new_zeros(most + 1, kv).scatter_reduce(0, nth[:, None].expand(rows, kv), size, "amax")[:most]
    part, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (part > 0.875).int(), -126).clamp(-126, 120)
    fit = ((e.int() + 127) << 23).view(torch.float32)
    at = pages.clamp(max=n_pages - 1)
    before = torch.where((first > 0)[:, None], scale[at], 0)
    now = torch.maximum(before, fit)
    # earlier tokens of those pages move to the new scale
    here = codes[at]
    earlier = (torch.arange(page, device=DEV) < first[:, None])[:, None, :, None]
    moved = torch.where(earlier, (here.float() * (before / now)[:, :, None, None]).to(F8).float(), here.float()).to(F8)
    spare = torch.empty(1, kv, page, hd, dtype=F8, device=DEV)
    whole = torch.cat([codes, spare]).view(torch.uint8)
    whole[pages] = moved.view(torch.uint8)
    scale.copy_(torch.cat([scale, scale[:1]]).index_put((pages,), now)[:n_pages])
    # the new tokens
    y = x / torch.cat([now, now[:1]])[nth][:, :, None]
    y = torch.where(x.isfinite(), y, float("nan")).to(F8)
    whole[pg, :, off] = y.view(torch.uint8)
    codes.view(torch.uint8).copy_(whole[:n_pages])


def _softmax_out(logits, v, shape):
    """exp and sums over the last axis, with rows that see nothing giving zeros and -inf."""
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0, top)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1)
    return out, (top + total.log()).squeeze(-1)


def _attend(s):
    if own:
        from conditional_draft_tree_lm_gb300 import cache_attention
        cache_attention(s["cache"], s["q"], s["table"], s["length"], k_new=s["k_new"], v_new=s["v_new"],
                        mask=s["mask"], scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["work"])
        return dict(out=s["out"], lse=s["lse"])
    n, slots, heads, hd = s["q"].shape
    _, kv, page, _ = s["k"].shape
    at = s["table"].clamp(min=0).long()
    # [request, head, cached token, channel], cleared behind each request's length
    held = (torch.arange(at.shape[1] * page, device=DEV) < s["length"][:, None])[:, None, :, None]

    def cached(codes, scale):
        x = codes[at].float() * scale[at][:, :, :, None, None]
        return torch.where(held, x.transpose(1, 2).reshape(n, kv, -1, hd), 0)

    k, v = cached(s["k"], s["k_scale"]), cached(s["v"], s["v_scale"])
    seen = held[:, :, None, :, 0]
    if s["k_new"] is not None:
        k = torch.cat([k, s["k_new"].float().transpose(1, 2)], 2)
        v = torch.cat([v, s["v_new"].float().transpose(1, 2)], 2)
        tree = s["mask"].bool() if s["mask"] is not None else torch.ones(slots, slots, device=DEV).tril().bool().expand(n, -1, -1)
        seen = torch.cat([seen.expand(n, 1, slots, -1), tree[:, None]], -1)
    # the heads that share a key/value head are rows of one product
    q = s["q"].float().view(n, slots, kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(n, kv, -1, hd)
    logits = torch.matmul(q * s["scale"], k.transpose(-1, -2)).view(n, kv, heads // kv, slots, -1)
    logits = logits.masked_fill_(~seen[:, :, None], -math.inf).view(n, kv, -1, k.shape[2])
    out, lse = _softmax_out(logits, v, None)
    out = out.view(n, kv, heads // kv, slots, hd).permute(0, 3, 1, 2, 4).reshape(n, slots, heads, hd)
    lse = lse.view(n, kv, heads // kv, slots).permute(0, 3, 1, 2).reshape(n, slots, heads)
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _prompt(s):
    if own:
        from conditional_draft_tree_lm_gb300 import prompt_attention
        prompt_attention(s["q"], s["k"], s["v"], s["row_start"], scale=s["scale"], out=s["out"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    rows, heads, hd = s["q"].shape
    kv, n, longest = s["k"].shape[1], s["row_start"].numel() - 1, s["longest"]
    start, end = s["row_start"][:-1].long(), s["row_start"][1:].long()
    # padded to the longest prompt
    pos = torch.arange(longest, device=DEV)
    at = (start[:, None] + pos).clamp(max=rows - 1)
    q = s["q"][at].float().view(n, longest, kv, heads // kv, hd).permute(0, 2, 3, 1, 4)
    k = s["k"][at].float().permute(0, 2, 3, 1).unsqueeze(2)
    v = s["v"][at].float().permute(0, 2, 1, 3).unsqueeze(2)
    logits = torch.matmul(q * s["scale"], k)
    logits = logits.masked_fill_(pos > pos[:, None], -math.inf)
    out, lse = _softmax_out(logits, v, None)
    # back to packed rows
    req = torch.searchsorted(end, torch.arange(rows, device=DEV), right=True)
    nth = torch.arange(rows, device=DEV) - start[req]
    out = out[req, :, :, nth].reshape(rows, heads, hd).to(torch.bfloat16)
    return dict(out=out, lse=lse[req, :, :, nth].reshape(rows, heads))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "plan":
        rows = c["req"] * (4 if c["tree"] else 0.56 * c["new"])
        new = rows / c["page"] + c["req"]
        return dict(bytes=int(rows * (16 if c["tree"] else 12) + 8 * new + 16 * c["req"]), flops=0)
    if c["op"] == "append":
        # 4 of the 16 on average are accepted; ragged prompts average 5/8 of the longest
        rows = c["req"] * ((min(4.0, c["new"])) if c["tree"] else (1 if c["new"] == 1 else 0.625 * c["new"]))
        per = c["kv"] * c["hd"]
        return dict(bytes=int(rows * (2 * per * 3 + 8) + 8 * (rows / c["page"] + c["req"]) * c["kv"]), flops=int(2 * rows * per * 2))
    if c["op"] == "attend":
        keys = c["req"] * (0.625 * c["ctx"] if c["req"] > 1 else c["ctx"])
        fresh = c["req"] * c["slots"] if c["fresh"] else 0
        rows = c["slots"] * c["heads"]
        size = keys * c["kv"] * (2 * c["hd"] + 8 / c["page"]) + 4 * fresh * c["kv"] * c["hd"] + fresh * c["slots"]
        size += c["req"] * rows * (4 * c["hd"] + 4)
        pairs = keys * rows + (fresh * min(c["slots"], 16) * c["heads"] if fresh else 0)
        return dict(bytes=int(size), flops=int(4 * c["hd"] * pairs))
    toks = c["req"] * (0.625 * c["longest"] if c["req"] > 1 else c["longest"])
    pairs = c["req"] * ((0.4375 if c["req"] > 1 else 1) * c["longest"] ** 2 / 2 + c["longest"] / 2)
    return dict(bytes=int(toks * (4 * c["hd"] * (c["heads"] + c["kv"]) + 4 * c["heads"])), flops=int(4 * c["hd"] * c["heads"] * pairs))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _plan_exact, "append": _append_exact, "attend": _attend_exact, "prompt": _prompt_exact}[s["op"]](s)


def _plan_exact(s):
    """The plan, request after request, with a queue of free pages."""
    page, n_pages = s["page"], s["ring"].numel()
    old, delta = s["old"].tolist(), s["delta"].tolist()
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, count = s["ring_in"].tolist()
    path = s["path"].cpu().numpy() if s["path_rows"] else None
    slot, pos, src = (np.full(s["max_rows"], -1, np.int64) for _ in range(3))
    start, length, put, took = [0], [], head + count, 0
    for q, (a, d) in enumerate(zip(old, delta)):
        b = max(0, a + d + s["extra"])
        for j in range(-(-a // page), -(-b // page)):
            table[q, j] = ring[(head + took) % n_pages]
            took += 1
        for j in range(-(-b // page), -(-a // page)):
            ring[put % n_pages] = table[q, j]
            put += 1
        p = np.arange(a, max(a, b))
        at = slice(start[-1], start[-1] + len(p))
        pos[at], slot[at] = p, table[q, p // page].astype(np.int64) * page + p % page
        if path is not None and len(p):
            src[at] = q * s["path_rows"] + np.concatenate([[0], path[q, :len(p) - 1]])
        start.append(start[-1] + len(p))
        length.append(b)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)  # noqa: E731
    return _plan_answer(i32(length), i32(table), i32(ring), i32([(head + took) % n_pages, put - head - took]), i32(start),
                        torch.tensor(slot), i32(pos), i32(src) if path is not None else None, i32([0]))


def _power64(e):
    """2 ** e, by the bits: library powers may be a unit off."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest value of 4 exponent and 3 mantissa bits, ties to even, |x| <= 448."""
    unit = _power64((torch.frexp(x)[1] - 1).clamp(min=-6) - 3)
    return torch.round(x / unit) * unit


def _append_exact(s):
    page, slot = s["page"], s["slot_map"].tolist()
    src = list(range(len(slot))) if s["src_rows"] is None else s["src_rows"].tolist()
    runs = {}
    for r, t in zip(src, slot):
        if t >= 0:
            runs.setdefault(t // page, []).append((r, t % page))
    found = {}
    for name in ("k", "v"):
        codes, scale, x = s[name].double(), s[name + "_scale"].double(), s[name + "_new"].double()
        for pg, group in runs.items():
            y = x[[r for r, _ in group]]
            lo = group[0][1]
            part, e = torch.frexp((y.abs().amax((0, 2)) / 448).clamp(min=2.0 ** -126))
            fit = _power64(e - (part == 0.5).int())
            now = torch.maximum(fit, scale[pg]) if lo else fit
            codes[pg, :, :lo] = _round_e4m3(codes[pg, :, :lo] * (scale[pg] / now)[:, None, None])
            codes[pg, :, lo:lo + len(group)] = _round_e4m3((y / now[:, None]).transpose(0, 1))
            scale[pg] = now
        found[name], found[name + "_scale"] = codes, scale
    return found


def _attend_exact(s):
    n, slots, heads, hd = s["q"].shape
    _, kv, page, _ = s["k"].shape
    g = heads // kv
    if n * heads * slots * s["table"].shape[1] * page > 1 << 31:
        return None
    out = torch.zeros(n, slots, heads, hd, dtype=torch.float64, device=DEV)
    lse = torch.full((n, slots, heads), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(n):
        length = int(s["length"][b])
        at = s["table"][b, :-(-length // page)].long()
        for h in range(kv):
            k = (s["k"][at, h].double() * s["k_scale"][at, h].double()[:, None, None]).reshape(-1, hd)[:length]
            v = (s["v"][at, h].double() * s["v_scale"][at, h].double()[:, None, None]).reshape(-1, hd)[:length]
            see = torch.ones(slots, length, dtype=torch.bool, device=DEV)
            if s["k_new"] is not None:
                k, v = torch.cat([k, s["k_new"][b, :, h].double()]), torch.cat([v, s["v_new"][b, :, h].double()])
                see = torch.cat([see, s["mask"][b] != 0], 1)
            for j in range(h * g, h * g + g):
                z = (s["q"][b, :, j].double() @ k.T * s["scale"]).masked_fill(~see, -math.inf)
                lse[b, :, j] = torch.logsumexp(z, -1)
                out[b, :, j] = torch.exp(z - lse[b, :, j, None]).nan_to_num() @ v
    return dict(out=out, lse=lse)


def _prompt_exact(s):
    rows, heads, hd = s["q"].shape
    kv = s["k"].shape[1]
    out = torch.zeros(rows, heads, hd, dtype=torch.float64, device=DEV)
    lse = torch.zeros(rows, heads, dtype=torch.float64, device=DEV)
    bounds = s["row_start"].tolist()
    for a, z in zip(bounds[:-1], bounds[1:]):
        for h in range(heads):
            k, v = s["k"][a:z, h // (heads // kv)].double(), s["v"][a:z, h // (heads // kv)].double()
            for lo in range(a, z, 2048):
                hi = min(z, lo + 2048)
                w = s["q"][lo:hi, h].double() @ k[:hi - a].T * s["scale"]
                w = w.masked_fill(torch.arange(hi - a, device=DEV) > torch.arange(lo - a, hi - a, device=DEV)[:, None], -math.inf)
                lse[lo:hi, h] = torch.logsumexp(w, -1)
                out[lo:hi, h] = torch.softmax(w, -1) @ v[:hi - a]
    return dict(out=out, lse=lse)
