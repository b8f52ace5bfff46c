"""Measured cases of the operators that stand around the attention of a target layer.

Three operators, in the order in which a pass of the target model meets them: the matrix product with its
bias, activation or gate and residual (projections, the gated feed-forward width, the output head), the norms
of queries and keys for each head with the rotation by their positions, and the log probabilities of given
tokens with entropy and the best alternatives.

``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is true, through
``conditional_draft_tree_lm_gb300``.  ``exact`` states each definition once more in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one user's token through the joint query, key and value projection: latency
        dict(name="linear_qkv_1", op="linear", rows=1, inner=2560, outer=6144, gate=False, act="", bias=True, res=False, full=False),
        # 32 users' tokens through the gated feed-forward width: bandwidth
        dict(name="linear_gate_32", op="linear", rows=32, inner=2560, outer=10240, gate=True, act="silu", bias=False, res=False, full=False),
        # the slots of one drafted tree through the output head, logits in 32 bits
        dict(name="linear_head_65", op="linear", rows=65, inner=2560, outer=151936, gate=False, act="", bias=False, res=False, full=True),
        # the slots of 32 trees from the heads back to the residual stream
        dict(name="linear_out_2080", op="linear", rows=2080, inner=4096, outer=2560, gate=False, act="", bias=False, res=True, full=False),
        # packed prompts through the gated feed-forward width: arithmetic
        dict(name="linear_gate_8k", op="linear", rows=8192, inner=2560, outer=10240, gate=True, act="silu", bias=False, res=False, full=False),
        # plain decoding of 32 users at long contexts: latency
        dict(name="rotate_32", op="rotate", req=32, slots=1, heads=32, kv=8, hd=128, rot=128, pairs="halves", norm=True, ctx=131072),
        # the slots of 32 drafted trees, each at its request's length and its own depth
        dict(name="rotate_tree", op="rotate", req=32, slots=65, heads=32, kv=8, hd=128, rot=128, pairs="halves", norm=True, ctx=16384),
        # 32k tokens of packed prompts
        dict(name="rotate_32k", op="rotate", req=1, slots=32768, heads=32, kv=8, hd=128, rot=128, pairs="halves", norm=True, ctx=0),
        # one user's token, with what a client that shows alternatives asks for: latency
        dict(name="logp_1", op="logp", rows=1, vocab=151936, asked=1, top=20, T=1.0, full=True, banned=False),
        # the slots of one tree with the drafted children, at a temperature
        dict(name="logp_tree_65", op="logp", rows=65, vocab=151936, asked=8, top=8, T=0.6, full=True, banned=False),
        # the slots of 32 trees; a grammar leaves some rows few tokens
        dict(name="logp_2080", op="logp", rows=2080, vocab=151936, asked=1, top=5, T=1.0, full=True, banned=True),
        # scoring 8k tokens of prompts from logits in 16 bits
        dict(name="logp_8k", op="logp", rows=8192, vocab=151936, asked=1, top=0, T=1.0, full=False, banned=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rotate", "logp"])
    if op == "linear":
        rows, inner = _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1024)
        gate = rng.random() < 0.4
        # at most 2^37 products in all, so that a drawn case stays below the largest listed one
        most = min(32768, (1 << 37) // (rows * inner * (2 if gate else 1)))
        outer = _log_int(rng, min(16, most), most)
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"] if gate else ["", "", "silu", "gelu", "gelu_tanh", "relu"])
        return dict(op=op, rows=rows, inner=inner, outer=outer, gate=gate, act=act, bias=rng.random() < 0.5,
                    res=rng.random() < 0.4, full=rng.random() < 0.2)
    if op == "rotate":
        kv = rng.choice([1, 2, 4, 8])
        heads, hd = kv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([64, 96, 128, 128, 256])
        slots = rng.choice([1, 1, 2, 17, 65, 129, _log_int(rng, 1, 4096)])
        req = max(1, min(_log_int(rng, 1, 512), (1 << 27) // (slots * (heads + kv) * hd)))
        return dict(op=op, req=req, slots=slots, heads=heads, kv=kv, hd=hd, rot=rng.choice([hd, hd, hd // 2]),
                    pairs=rng.choice(["halves", "halves", "neighbours"]), norm=rng.random() < 0.7, ctx=_log_int(rng, 1, 1 << 20))
    vocab = _log_int(rng, 100, 262144)
    return dict(op=op, rows=max(1, min(_log_int(rng, 1, 16384), (1 << 29) // vocab)), vocab=vocab, asked=rng.choice([1, 1, 2, 8]),
                top=rng.choice([0, 1, 5, 20, 33]), T=rng.choice([1.0, 1.0, 0.6, 1.7]), full=rng.random() < 0.6,
                banned=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _half(g, *shape, scale=1.0):
    """Normal numbers in bf16, made in pieces so that a large weight needs no copy of itself in 32 bits."""
    x = torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(_normal(g, part.numel()) * scale)
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case, op=case["op"])
    {"linear": _prepare_linear, "rotate": _prepare_rotate, "logp": _prepare_logp}[case["op"]](s, case, g, seed)
    return s


def _prepare_linear(s, c, g, seed):
    rows, inner, outer = c["rows"], c["inner"], c["outer"]
    # hidden states with a few channels that stand out, as trained models have them
    loud = 1 + 7 * (torch.rand(1, inner, generator=g, device=DEV) > 0.99)
    s["x"] = (_normal(g, rows, inner) * loud).to(torch.bfloat16)
    s["w"] = _half(g, outer, inner, scale=inner ** -0.5)
    s["gate"] = _half(g, outer, inner, scale=inner ** -0.5) if c["gate"] else None
    s["b"] = _half(g, outer, scale=0.5) if c["bias"] else None
    s["gate_b"] = _half(g, outer, scale=0.5) if c["bias"] and c["gate"] else None
    s["res"] = _half(g, rows, outer) if c["res"] else None
    s["out"] = torch.zeros(rows, outer, dtype=torch.float32 if c["full"] else torch.bfloat16, device=DEV)


def _prepare_rotate(s, c, g, seed):
    rs = np.random.RandomState(seed & 0x7FFFFFFF)
    req, slots, heads, kv, hd, rot = c["req"], c["slots"], c["heads"], c["kv"], c["hd"], c["rot"]
    # queries and keys as they come from a joint projection: slices of its rows
    qkv = _half(g, req, slots, heads + 2 * kv, hd)
    s["q"], s["k"] = qkv[..., :heads, :], qkv[..., heads:heads + kv, :]
    s["q_w"] = (1 + 0.3 * _normal(g, hd)).to(torch.bfloat16) if c["norm"] else None
    s["k_w"] = (1 + 0.3 * _normal(g, hd)).to(torch.bfloat16) if c["norm"] else None
    # one token stands at its request's length, a tree's slots at their depths behind it, a prompt's tokens one after the other
    if 1 < slots <= 513:
        depth = np.zeros((req, slots), np.int64)
        parent = np.maximum(np.arange(slots) - 1 - rs.randint(0, 8, (req, slots)), 0)
        for a in range(1, slots):
            depth[:, a] = depth[np.arange(req), parent[:, a]] + 1
    else:
        depth = np.tile(np.arange(slots), (req, 1))
    s["depth"] = torch.as_tensor(depth, dtype=torch.int32, device=DEV)
    s["length"] = torch.as_tensor(rs.randint(c["ctx"] // 4, c["ctx"] + 1, req), dtype=torch.int32, device=DEV)
    s["theta"], s["eps"] = 1e6, 1e-6
    s["freq"] = s["theta"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    if own:
        from conditional_draft_tree_lm_gb300 import Rotary
        s["rotary"] = Rotary(rot, theta=s["theta"], interleaved=c["pairs"] == "neighbours")
    s["q_out"] = torch.zeros(req, slots, heads, hd, dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.zeros(req, slots, kv, hd, dtype=torch.bfloat16, device=DEV)


def _prepare_logp(s, c, g, seed):
    rows, vocab = c["rows"], c["vocab"]
    x = torch.empty(rows, vocab, dtype=torch.float32 if c["full"] else torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // vocab)
    # flat rows and peaked ones, as confident and unsure models have them
    width = torch.exp(_normal(g, rows, 1) * 0.5) * 2
    for at in range(0, rows, step):
        z = _normal(g, min(step, rows - at), vocab) * width[at:at + step]
        x[at:at + step] = z.to(x.dtype)
    s["tok"] = torch.randint(0, vocab, (rows, c["asked"]), generator=g, device=DEV, dtype=torch.int32)
    if c["banned"]:
        # of a third of the rows a grammar leaves about 80 tokens, the asked ones among them
        few = torch.rand(rows, generator=g, device=DEV) < 0.33
        for r in few.nonzero().view(-1).tolist():
            keep = torch.rand(vocab, generator=g, device=DEV) < 80 / vocab
            keep[s["tok"][r].long()] = True
            x[r].masked_fill_(~keep, -math.inf)
    s["x"] = x


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"linear": _linear, "rotate": _rotate, "logp": _logp}[s["op"]](s)


def _activation(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return z.clamp(min=0)
    return z


def _linear(s):
    c = s["case"]
    if own:
        from conditional_draft_tree_lm_gb300 import linear
        return linear(s["x"], s["w"], bias=s["b"], gate=s["gate"], gate_bias=s["gate_b"], activation=c["act"] or None,
                      residual=s["res"], out=s["out"])
    x = s["x"].float()
    y = torch.matmul(x, s["w"].float().T)
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["gate"] is None:
        y = _activation(y, c["act"])
    else:
        z = torch.matmul(x, s["gate"].float().T)
        if s["gate_b"] is not None:
            z = z + s["gate_b"].float()
        y = _activation(z, c["act"]) * y
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["out"].dtype)


def _rotate(s):
    c = s["case"]
    if own:
        from conditional_draft_tree_lm_gb300 import qk_norm_rope
        return qk_norm_rope(s["q"], s["k"], positions=s["depth"], base=s["length"], rotary=s["rotary"], q_weight=s["q_w"],
                            k_weight=s["k_w"], eps=s["eps"], q_out=s["q_out"], k_out=s["k_out"])
    angle = (s["length"][:, None] + s["depth"]).double()[..., None, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    rot = c["rot"]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        turned, rest = x[..., :rot], x[..., rot:]
        if c["pairs"] == "halves":
            a, b = turned[..., :rot // 2], turned[..., rot // 2:]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([turned, rest], -1).to(torch.bfloat16)

    return one(s["q"], s["q_w"]), one(s["k"], s["k_w"])


def _logp(s):
    c = s["case"]
    if own:
        from conditional_draft_tree_lm_gb300 import token_logprobs
        y = token_logprobs(s["x"], s["tok"], top=c["top"], temperature=c["T"])
        return {k: y[k] for k in ("logp", "lse", "entropy") + (("top_tok", "top_logp") if c["top"] else ())}
    x = s["x"].float() / c["T"]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    mean = torch.where(e > 0, e * (x - top), 0).sum(-1, keepdim=True) / total
    found = dict(logp=x.gather(-1, s["tok"].long()) - lse, lse=lse.squeeze(-1), entropy=(total.log() - mean).squeeze(-1))
    if c["top"]:
        # keys that order by value and, among equals, by the lower token
        bits = s["x"].float().view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = (bits << 32) - torch.arange(x.shape[-1], device=DEV)
        tok = (-torch.topk(key, min(c["top"], x.shape[-1]), -1, sorted=True).values & 0xFFFFFFFF)
        found.update(top_tok=tok.int(), top_logp=x.gather(-1, tok) - lse)
    return found


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        rows, inner, outer, sides = c["rows"], c["inner"], c["outer"], 2 if c["gate"] else 1
        size = 2 * (rows * inner + sides * outer * inner) + (4 if c["full"] else 2) * rows * outer
        size += (2 * rows * outer if c["res"] else 0) + (2 * sides * outer if c["bias"] else 0)
        return dict(bytes=size, flops=2 * rows * inner * outer * sides)
    if c["op"] == "rotate":
        rows, values = c["req"] * c["slots"], (c["heads"] + c["kv"]) * c["hd"]
        return dict(bytes=rows * (4 * values + 4) + 4 * c["req"] + 8 * c["hd"], flops=rows * values * (8 if c["norm"] else 3))
    size = c["rows"] * (c["vocab"] * (4 if c["full"] else 2) + 8 * c["asked"] + 8 * c["top"] + 8)
    return dict(bytes=size, flops=5 * c["rows"] * c["vocab"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _linear_exact, "rotate": _rotate_exact, "logp": _logp_exact}[s["op"]](s)


def _linear_exact(s):
    x, out = s["x"].double(), torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    for lo in range(0, out.shape[1], 16384):
        cols = slice(lo, lo + 16384)
        side = {}
        for w, b in (("w", "b"), ("gate", "gate_b")):
            if s[w] is not None:
                side[w] = torch.einsum("mk,nk->mn", x, s[w][cols].double()) + (0 if s[b] is None else s[b][cols].double())
        z = side.get("gate", side["w"])
        act = s["case"]["act"]
        if act == "silu":
            z = z * torch.special.expit(z)
        elif act == "gelu":
            z = z * torch.special.ndtr(z)
        elif act == "gelu_tanh":
            # (1 + tanh u) / 2 is the logistic function of 2 u
            z = z * torch.special.expit(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        elif act == "relu":
            z = torch.where(z > 0, z, 0)
        out[:, cols] = z * side["w"] if "gate" in side else z
    return out if s["res"] is None else out + s["res"].double()


def _rotate_exact(s):
    rot, halves = s["case"]["rot"], s["case"]["pairs"] == "halves"
    where = s["length"].double()[:, None, None, None] + s["depth"].double()[:, :, None, None]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), where * s["freq"])
    found = []
    for x, w in ((s["q"], s["q_w"]), (s["k"], s["k_w"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        pairs = x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2) if halves else x[..., :rot].unflatten(-1, (-1, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = (z.transpose(-1, -2) if halves else z).flatten(-2)
        found.append(torch.cat([z, x[..., rot:]], -1))
    return tuple(found)


def _logp_exact(s):
    c, rows = s["case"], s["x"].shape[0]
    parts = []
    step = max(1, (1 << 27) // c["vocab"])
    for lo in range(0, rows, step):
        x = s["x"][lo:lo + step].double() / c["T"]
        lse = torch.logsumexp(x, -1, keepdim=True)
        logp = x - lse
        part = dict(logp=logp.gather(-1, s["tok"][lo:lo + step].long()), lse=lse.squeeze(-1),
                    entropy=-torch.special.xlogy(torch.exp(logp), torch.exp(logp)).sum(-1))
        if c["top"]:
            value, tok = torch.sort(s["x"][lo:lo + step].float(), dim=-1, descending=True, stable=True)
            part["top_tok"] = tok[:, :c["top"]].int()
            part["top_logp"] = logp.gather(-1, tok[:, :c["top"]])
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
