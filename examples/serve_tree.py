"""One attention layer of a target model served with drafted trees.

Prompts are read (``kv_plan``, ``prompt_attention``, ``kv_append``), then every round drafts a tree
(``DraftTreeBuilder``), scores all its slots in one pass over the 8-bit cache under the ancestor-only mask
(``cache_attention``), walks the tree against the target's logits, and appends the keys and values of the accepted
path only (``kv_plan`` with the walk's path, ``kv_append`` with its source rows).  No length leaves the GPU: the plan,
the append and the attention read what the walk has written.

The drafter and the target have random weights, so few drafted tokens are accepted; ``--follow`` plants a target that
agrees with a drafted child that often.

    python examples/serve_tree.py [--requests 3] [--rounds 8] [--follow 0.7]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class TargetLayer:
    """Embedding, one layer of grouped-head attention, output head: bf16, random."""

    def __init__(self, vocab, width, heads, kv_heads, head_dim, gen):
        import torch

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.emb = normal(vocab, width, scale=1.0)
        self.qkv = normal((heads + 2 * kv_heads) * head_dim, width, scale=width ** -0.5)
        self.out = normal(vocab, heads * head_dim, scale=(heads * head_dim) ** -0.5)

    def project(self, tokens):
        """q, k, v of tokens: slices of one product, used strided as they are."""
        x = self.emb[tokens.long()] @ self.qkv.T
        x = x.view(*tokens.shape, self.heads + 2 * self.kv_heads, self.head_dim)
        return x[..., :self.heads, :], x[..., self.heads:-self.kv_heads, :], x[..., -self.kv_heads:, :]

    def logits(self, attended):
        return (attended.flatten(-2) @ self.out.T).float()


class Server:
    """The cache, its page ring and tables, and the buffers of a round."""

    def __init__(self, cfg, target, max_tokens, page=16):
        import torch
        from conditional_draft_tree_lm_gb300 import AttentionWorkspace, KvCache
        n, i32, dev = cfg.n_req, torch.int32, "cuda"
        blocks = -(-max_tokens // page)
        pages = n * blocks + 2
        self.cfg, self.target, self.page = cfg, target, page
        self.cache = KvCache.empty(pages, page, target.kv_heads, target.head_dim)
        self.work = AttentionWorkspace()
        self.table = torch.full((n, blocks), -1, dtype=i32, device=dev)
        self.free = torch.arange(pages, dtype=i32, device=dev).flip(0).contiguous()
        # lengths and the ring's state alternate between two buffers: a plan reads one and writes the other
        self.length = [torch.zeros(n, dtype=i32, device=dev) for _ in range(2)]
        self.ring = [torch.tensor([0, pages], dtype=i32, device=dev), torch.zeros(2, dtype=i32, device=dev)]
        self.row_start = torch.zeros(n + 1, dtype=i32, device=dev)
        # what any call has reported: a plan writes its own word, the others add theirs
        self.planned = torch.zeros(1, dtype=i32, device=dev)
        self.status = torch.zeros(1, dtype=i32, device=dev)

    def plan(self, max_rows, **kw):
        import torch
        from conditional_draft_tree_lm_gb300 import kv_plan
        slots = torch.empty(max_rows, dtype=torch.int64, device="cuda")
        src = torch.empty(max_rows, dtype=torch.int32, device="cuda")
        kv_plan(self.length[0], self.length[1], self.table, self.free, self.ring[0], self.ring[1], self.row_start, slots,
                self.planned, page=self.page, src_rows=src, **kw)
        self.status |= self.planned
        self.length.reverse()
        self.ring.reverse()
        return slots, src

    def read_prompts(self, prompts):
        """Packed prompts (a list of int tensors) into the cache; the logits behind each one's last token."""
        import torch
        from conditional_draft_tree_lm_gb300 import kv_append, prompt_attention
        tokens = torch.cat(prompts)
        q, k, v = self.target.project(tokens)
        slots, _ = self.plan(tokens.numel(), delta=torch.tensor([p.numel() for p in prompts], dtype=torch.int32, device="cuda"))
        attended = prompt_attention(q, k, v, self.row_start, status=self.status)
        kv_append(self.cache, k, v, slots, status=self.status)
        return self.target.logits(attended[(self.row_start[1:] - 1).long()])

    def score_tree(self, tree):
        """Target logits [n_req, slots, V] of every tree slot, and the slots' keys and values."""
        from conditional_draft_tree_lm_gb300 import cache_attention
        q, k, v = self.target.project(tree["tok"])
        attended = cache_attention(self.cache, q, self.table, self.length[0], k_new=k, v_new=v, mask=tree["mask"],
                                   workspace=self.work, status=self.status)
        return self.target.logits(attended), k, v

    def commit(self, walk, k, v):
        """Root and accepted slots into the cache."""
        from conditional_draft_tree_lm_gb300 import kv_append
        n, slots = k.shape[:2]
        where, src = self.plan(n * (walk["accepted"].shape[1] + 1), delta=walk["accept_len"], extra=1,
                               path=walk["accepted"], path_rows=slots)
        kv_append(self.cache, k, v, where, src_rows=src, status=self.status)


def serve(requests=3, rounds=8, follow=0.7, seed=0):
    """Returns (server, committed token lists, accepted counts per round)."""
    import torch
    from conditional_draft_tree_lm_gb300 import DraftTreeBuilder, bf16_tensor
    from workloads import get_config, make_round_inputs, make_weights
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cfg = get_config("tiny_bf16", n_req=requests)
    target = TargetLayer(cfg.V, cfg.d, 4, 2, 64, gen)
    builder = DraftTreeBuilder(cfg, {k: bf16_tensor(w) for k, w in make_weights(cfg).items()})
    lens = [5 + 23 * q for q in range(requests)]
    server = Server(cfg, target, max(lens) + rounds * cfg.block + 1)
    prompts = [torch.randint(0, cfg.V, (n,), generator=gen, device="cuda", dtype=torch.int32) for n in lens]
    committed = [p.tolist() for p in prompts]
    root = server.read_prompts(prompts).argmax(-1).int()
    counts = []
    for r in range(rounds):
        H, _ = make_round_inputs(cfg, r)
        tree = builder.build_round(bf16_tensor(H), root)
        logits, k, v = server.score_tree(tree)
        if follow > 0:  # raise a child's token above the rest at some slots
            child = torch.arange(1, tree["tok"].shape[1], device="cuda").expand(requests, -1)
            keep = torch.rand(child.shape, generator=gen, device="cuda") < follow
            q, c = keep.nonzero(as_tuple=True)
            logits[q, tree["parent"][q, c + 1].long(), tree["tok"][q, c + 1].long()] += 1e4 - c
        walk = builder.accept_walk(logits, tree["tok"], tree["parent"])
        server.commit(walk, k, v)
        # what follows is only the example's own record of the tokens
        acc, path, tok = walk["accept_len"].tolist(), walk["accepted"].tolist(), tree["tok"].tolist()
        for q in range(requests):
            committed[q] += [tok[q][s] for s in [0] + path[q][:acc[q]]]
        counts.append(acc)
        root = walk["bonus"]
    if server.status.item() != 0 or builder.device_status() != 0:
        raise RuntimeError(f"cache status {server.status.item()}, builder status {builder.device_status()}")
    builder.close()
    return server, committed, counts


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--follow", type=float, default=0.7)
    a = ap.parse_args()
    server, committed, counts = serve(a.requests, a.rounds, a.follow)
    for r, acc in enumerate(counts):
        print(f"round {r}: accepted {acc}")
    print("cached tokens:", server.length[0].tolist(), "free pages:", server.ring[0][1].item())


if __name__ == "__main__":
    main()
