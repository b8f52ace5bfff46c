"""examples/serve_tree.py end to end: what stands in the cache after rounds of drafting, verification and commits."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("requests,follow", [(1, 0.8), (4, 0.6), (3, 0.0)])
def test_serve_tree_example(requests, follow):
    import torch
    from serve_tree import serve
    server, committed, counts = serve(requests=requests, rounds=10, follow=follow, seed=requests)
    lens = server.length[0].tolist()
    # one root a round and the accepted slots
    assert lens == [len(c) for c in committed]
    assert [len(c) for c in committed] == [5 + 23 * q + sum(1 + acc[q] for acc in counts) for q in range(requests)]
    if follow > 0:
        assert max(max(acc) for acc in counts) >= 2
    # pages: every block has one of its own, the ring holds the others
    table, page, cache = server.table.cpu().numpy(), server.page, server.cache
    used = [table[q, :-(-lens[q] // page)] for q in range(requests)]
    head, count = server.ring[0].tolist()
    free = [server.free.tolist()[(head + i) % cache.n_pages] for i in range(count)]
    assert sorted(np.concatenate(used).tolist() + free) == list(range(cache.n_pages))
    # the cached keys and values are the committed tokens', within e4m3's rounding under the page's scale (half a
    # unit of 3 bits, 2^-4 relative, or half of the smallest step 2^-9), twice where a scale grew later
    for q in range(requests):
        _, k, v = server.target.project(torch.tensor(committed[q], device="cuda"))
        pages = torch.tensor(used[q], device="cuda", dtype=torch.long)
        for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
            s = scale[pages][:, :, None, None].expand(-1, -1, page, cache.head_dim)
            have = (codes[pages].float() * s).transpose(1, 2).reshape(-1, cache.n_kv, cache.head_dim)[:lens[q]]
            unit = s.transpose(1, 2).reshape(-1, cache.n_kv, cache.head_dim)[:lens[q]]
            off = (have - x.float()).abs()
            assert (off <= x.float().abs() * 2.0 ** -4 + unit * 2.0 ** -9).all()


def test_prompt_and_cache_attention_agree():
    """A prompt's last token: attended within the prompt, and as a new token over a cache that holds the others."""
    import torch
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, KvCache, cache_attention, kv_append, prompt_attention
    torch.manual_seed(0)
    n, heads, kv, hd, page = 200, 8, 2, 128, 32
    q, k, v = (torch.randn(n, h, hd, device="cuda").to(torch.bfloat16) for h in (heads, kv, kv))
    # keys and values that e4m3 holds exactly, so that both paths see the same numbers
    k, v = (x.to(torch.float8_e4m3fn).to(torch.bfloat16) for x in (k, v))
    full = prompt_attention(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    cache = KvCache.empty(8, page, kv, hd)
    kv_append(cache, k, v, torch.arange(n, device="cuda"))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    work = AttentionWorkspace()
    for slots in (1, 3, 17):
        a = n - slots
        got = cache_attention(cache, q[None, a:], table, torch.tensor([a], dtype=torch.int32, device="cuda"), k_new=k[None, a:],
                              v_new=v[None, a:], workspace=work)
        assert (got[0].float() - full[a:].float()).abs().max() <= 2.0 ** -6
