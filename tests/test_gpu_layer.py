"""The operators around a target layer's attention on the GPU against their 64-bit definitions.

Tolerances count roundings.  Half a step of bf16 is 2^-8 of a value, of fp32 2^-24.  A sum of K products in fp32 is off by
at most K 2^-23 of the sum of their magnitudes (a rounding or a cut at every addition).  Where outputs are fp32, an accumulator of
the tensor core adds 512 channels, 16 at a time (two cuts each, one of the terms and one of the sum), and the accumulators, or
for one or two tokens the channels of 64 pairs of lanes, are added with a rounding each: (2 * 32 + K / 128 + 16) 2^-23.
"""
import math

import numpy as np
import pytest

from oracle import layer as ol

pytestmark = pytest.mark.gpu

HALF = {"torch.bfloat16": 2.0 ** -8, "torch.float32": 2.0 ** -24}


def _t():
    import torch
    torch.cuda.set_device(0)
    return torch


def bf16(rs, *shape, scale=1.0):
    torch = _t()
    return torch.as_tensor(rs.standard_normal(shape) * scale).to(torch.bfloat16).cuda()


def f64(x):
    return None if x is None else x.double().cpu().numpy()


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------
SLOPE = 1.13  # the largest slope of any of the activations


def linear_case(seed, rows, inner, outer, gate=False, act=None, bias=False, res=False):
    rs = np.random.RandomState(seed)
    c = dict(x=bf16(rs, rows, inner), weight=bf16(rs, outer, inner, scale=inner ** -0.5), activation=act)
    if gate:
        c["gate"] = bf16(rs, outer, inner, scale=inner ** -0.5)
    if bias:
        c["bias"] = bf16(rs, outer)
        if gate:
            c["gate_bias"] = bf16(rs, outer)
    if res:
        c["residual"] = bf16(rs, rows, outer)
    return c


def check_linear(c, out, cols=None):
    """Against NumPy in 64 bits, with the bound of the fp32 sums carried through the activation and the gate."""
    pick = (lambda t: t) if cols is None else (lambda t: t[..., cols] if t.dim() == 1 else t[cols])
    x, w, g = f64(c["x"]), f64(pick(c["weight"])), c.get("gate")
    b, gb, res, act = c.get("bias"), c.get("gate_bias"), c.get("residual"), c["activation"]
    b, gb = (None if t is None else f64(pick(t)) for t in (b, gb))
    g = None if g is None else f64(pick(g))
    res = None if res is None else f64(res if cols is None else res[:, cols])
    got = f64(out if cols is None else out[:, cols])
    want = ol.linear(x, w, b, g, gb, act, res)
    unit = (x.shape[1] + 8) * 2.0 ** -23
    if str(out.dtype) == "torch.float32":
        unit = min(unit, (80 + x.shape[1] / 128) * 2.0 ** -23)
    off = (np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))) * unit
    y = x @ w.T + (0 if b is None else b)
    if g is not None:
        z = x @ g.T + (0 if gb is None else gb)
        off_z = (np.abs(x) @ np.abs(g).T + (0 if gb is None else np.abs(gb))) * unit
        a = ol.activation(z, act)
        off = (np.abs(a) + SLOPE * off_z) * off + SLOPE * off_z * np.abs(y) + np.abs(a * y) * 2.0 ** -20
    elif act:
        off = SLOPE * off + np.abs(ol.activation(y, act)) * 2.0 ** -20
    half = HALF[str(out.dtype)]
    off = off * (1 + half) + np.abs(want) * half + 2.0 ** -126
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], off[bad][:5])


@pytest.mark.parametrize("rows,inner,outer", [
    (1, 8, 1), (1, 2560, 6144), (2, 64, 5), (7, 72, 127), (16, 1032, 128), (17, 512, 129), (33, 2560, 300), (65, 520, 1001),
    (128, 256, 2501), (129, 136, 130), (255, 448, 257), (256, 64, 64), (257, 72, 513), (300, 4096, 1000), (1000, 192, 200),
    (1, 16384, 40), (2, 8, 20000), (513, 8, 3), (3, 8192, 130), (40, 8192, 200), (250, 4096, 129), (20, 256, 10240), (9, 72, 12345),
    (150, 136, 10000), (600, 256, 700), (300, 640, 64)])
@pytest.mark.parametrize("form", ["plain", "all", "gate", "gate32"])
def test_linear_sizes(rows, inner, outer, form):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    kw = dict(plain={}, all=dict(act="gelu_tanh", bias=True, res=True), gate=dict(gate=True, act="silu", bias=True, res=True),
              gate32=dict(gate=True, act="gelu"))[form]
    c = linear_case(rows + inner, rows, inner, outer, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = linear(status=status, out_dtype=torch.float32 if form in ("plain", "gate32") else None, **c)
    check_linear(c, out)
    assert status.item() == 0


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rows", [3, 400])
def test_linear_activations(act, gate, rows):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    c = linear_case(5, rows, 128, 200, gate=gate, act=act, bias=True)
    # arguments far on both sides
    c["gate_bias" if gate else "bias"] = torch.linspace(-30, 30, 200, device="cuda").to(torch.bfloat16)
    for dtype in (torch.float32, torch.bfloat16):
        check_linear(c, linear(out_dtype=dtype, **c))


@pytest.mark.parametrize("rows", [5, 300])
def test_linear_strides_and_what_stands_around(rows):
    """Slices of wider tensors in, columns of a wider one out: nothing beside them is read or written."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    rs = np.random.RandomState(3)
    wide, both = bf16(rs, rows, 3 * 136), bf16(rs, 2 * 259, 200, scale=0.1)
    wide[:, :136] = float("nan")
    wide[:, 272:] = float("nan")
    x, w, g = wide[:, 136:272], both[:259, 64:], both[259:, 64:]
    for off, width in ((8, 300), (7, 301), (1, 267)):
        for dtype in (torch.float32, torch.bfloat16):
            room = torch.full((rows, width), 7.0, dtype=dtype, device="cuda")
            res = bf16(rs, rows, width)[:, off:off + 259]
            c = dict(x=x, weight=w, gate=g, activation="silu", residual=res)
            out = room[:, off:off + 259]
            assert linear(out=out, **c) is out
            check_linear(c, out)
            assert (room[:, :off] == 7).all() and (room[:, off + 259:] == 7).all()
    # in place of the residual, and leading dimensions
    res = bf16(rs, rows, 259)
    c = dict(x=x, weight=w, residual=res.clone(), activation=None)
    assert linear(x, w, residual=res, out=res) is res
    check_linear(c, res)
    y = linear(x.unflatten(0, (rows // 5, 5)), w)
    assert y.shape == (rows // 5, 5, 259) and torch.equal(y.view(rows, 259), linear(x, w))
    one = linear(x[0], w)
    assert one.shape == (259,)
    check_linear(dict(x=x[:1], weight=w, activation=None), one[None])


@pytest.mark.parametrize("rows", [4, 300])
def test_linear_values_that_are_not_finite(rows):
    """They stay in their row and column."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    c = linear_case(11, rows, 264, 140)
    clean = linear(**c)
    c["x"][2, 100] = float("nan")
    c["x"][3, 5] = float("inf")
    c["weight"][7, 30] = float("nan")
    out = linear(**c)
    assert out[2].isnan().all() and out[:, 7].isnan().all() and not out[3].isfinite().any()
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[2:4] = rest[:, 7] = False
    assert torch.equal(out[rest], clean[rest])


def test_linear_of_no_rows():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    c = linear_case(1, 3, 64, 32, gate=True, res=True)
    c["x"], c["residual"] = c["x"][:0], c["residual"][:0]
    assert linear(**c).shape == (0, 32)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,inner,outer", [(257, 512, 96), (300, 520, 256), (700, 1024, 1000), (1000, 2568, 2600), (400, 8192, 77), (5000, 576, 513)])
@pytest.mark.parametrize("gate", [False, True])
def test_linear_of_many_rows_in_32_bits(rows, inner, outer, gate):
    """Several accumulators of 512 channels and one, tiles of all widths, with everything behind the product."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    c = linear_case(rows, rows, inner, outer, gate=gate, act="silu", bias=True, res=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = linear(out_dtype=torch.float32, status=status, **c)
    check_linear(c, out)
    assert status.item() == 0 and torch.equal(out, linear(out_dtype=torch.float32, **c))
    # rows that do not start on 16 bytes, and a residual that does not
    room = torch.full((rows, outer + 3), 7.0, device="cuda")
    c["residual"] = torch.cat([c["residual"], c["residual"][:, :3]], 1)[:, 1:outer + 1]
    linear(out=room[:, 1:outer + 1], **c)
    check_linear(c, room[:, 1:outer + 1])
    assert (room[:, 0] == 7).all() and (room[:, outer + 1:] == 7).all()


@pytest.mark.parametrize("rows", [1, 2, 40, 300])
def test_linear_between_columns_of_one_tensor(rows):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    rs = np.random.RandomState(rows)
    room, w = bf16(rs, rows, 640), bf16(rs, 256, 128, scale=0.1)
    c = dict(x=room[:, :128].clone(), weight=w, residual=room[:, 384:].clone(), activation=None)
    check_linear(c, linear(room[:, :128], w, residual=room[:, 384:], out=room[:, 128:384]))
    assert torch.equal(room[:, :128], c["x"]) and torch.equal(room[:, 384:], c["residual"])
    with pytest.raises(Exception, match="overlaps an input"):
        linear(room[:, :128], w, out=room[:, 127:383])


def test_linear_outputs_behind_32_bits():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    rows, outer = 40, 64
    room = torch.zeros(rows, 1 << 26, dtype=torch.bfloat16, device="cuda")  # rows 2^27 bytes apart, 5 GB in all
    c = linear_case(2, rows, 128, outer, act="silu", bias=True)
    c["residual"] = room[:, 1 << 20:][:, :outer]
    c["residual"].copy_(bf16(np.random.RandomState(4), rows, outer))
    want = linear(**c)
    linear(out=room[:, 77:77 + outer], **c)
    assert torch.equal(room[:, 77:77 + outer], want)
    check_linear(c, want)
    # many rows and columns: the last ones
    many = linear_case(6, 30000, 64, 90000)
    out = linear(**many)
    assert out.numel() > 2 ** 31
    last = dict(x=many["x"][-3:], weight=many["weight"][-200:], activation=None)
    check_linear(last, out[-3:, -200:])


@pytest.mark.parametrize("rows,inner,outer,gate", [(1, 2560, 6144, False), (32, 2560, 1280, True), (700, 512, 600, False), (700, 512, 600, True),
                                                   (64, 1024, 20000, False), (2100, 4096, 2560, False)])
def test_linear_gives_the_same_bits_alone_beside_others_and_replayed(rows, inner, outer, gate):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import linear
    c = linear_case(21, rows, inner, outer, gate=gate, act="silu", res=True)
    d = linear_case(22, 70, 1000, 900, gate=not gate, act="silu")
    want, other = linear(**c), linear(**d)
    side = torch.cuda.Stream()
    out, there = torch.zeros_like(want), torch.zeros_like(other)
    torch.cuda.synchronize()
    for _ in range(100):
        linear(out=there, stream=side, **d)
        linear(out=out, **c)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(there, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linear(out=out, **c)
        linear(out=there, **d)
    c["x"].neg_()
    fresh = linear(**c)
    for _ in range(3):
        out.zero_()
        there.zero_()
        graph.replay()
        assert torch.equal(out, fresh) and torch.equal(there, other)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------
def check_rotated(got, x, position, rotary, weight, eps):
    """fp32 within: the mean of squares, its root and the products (half of head_dim 2^-24, and 2^-20 with the angle) of the
    pair's size, and half a step of bf16."""
    x, w = f64(x), f64(weight)
    rows, heads, dim = x.shape
    rot = rotary.dim if rotary else 0
    amp = rotary.amplitude if rotary else 1.0
    want = ol.qk_norm_rope(x, position, rot, rotary.inv_freq if rotary else [], bool(rotary and rotary.interleaved), w, eps, amp)
    size = np.abs(want)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + rot // 2)
        size[..., a] = size[..., b] = np.hypot(want[..., a], want[..., b])
    off = size * (dim / 2 * 2.0 ** -24 + 2.0 ** -20) * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8 + 2.0 ** -126
    got = f64(got)
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], off[bad][:5])


@pytest.mark.parametrize("rows,heads,kv,dim,rot", [
    (1, 32, 8, 128, 128), (3, 1, 1, 64, 64), (5, 7, 1, 96, 48), (2, 5, 3, 256, 128), (33, 12, 4, 128, 64), (4, 3, 1, 32, 32),
    (2, 9, 9, 80, 16), (700, 4, 2, 64, 32), (3, 64, 1, 176, 176), (9, 6, 2, 48, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["both", "norm", "turn"])
def test_rotate_sizes(rows, heads, kv, dim, rot, interleaved, form):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    rs = np.random.RandomState(rows + dim)
    qkv = bf16(rs, rows, heads + 2 * kv, dim)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
    pos = rs.randint(0, 100000, rows)
    qw, kw = (bf16(rs, dim), bf16(rs, dim)) if form != "turn" else (None, None)
    rotary = Rotary(rot, theta=1e4, interleaved=interleaved, amplitude=1.0 if form == "turn" else 1.25) if form != "norm" else None
    before = qkv.clone()
    qo, ko = qk_norm_rope(q, k, positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary, q_weight=qw, k_weight=kw, eps=1e-5)
    assert torch.equal(qkv, before) and qo.is_contiguous() and ko.is_contiguous()
    check_rotated(qo, q, pos, rotary, qw, 1e-5)
    check_rotated(ko, k, pos, rotary, kw, 1e-5)
    # in place, queries alone, and a norm for one of the two
    qi = qkv.clone()
    a, b = qi[:, :heads], qi[:, heads:heads + kv]
    qk_norm_rope(a, b, positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary, q_weight=qw, k_weight=kw, eps=1e-5, q_out=a, k_out=b)
    assert torch.equal(a, qo) and torch.equal(b, ko) and torch.equal(qi[:, heads + kv:], before[:, heads + kv:])
    alone, none = qk_norm_rope(q, positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary, q_weight=qw, eps=1e-5)
    assert none is None and torch.equal(alone, qo)
    if form == "both":
        _, kt = qk_norm_rope(q, k, positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary, q_weight=qw, eps=1e-5)
        check_rotated(kt, k, pos, rotary, None, 1e-5)


def test_rotate_positions_of_trees_prompts_and_padding():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    rs = np.random.RandomState(8)
    i32 = dict(dtype=torch.int32, device="cuda")
    rotary = Rotary(64, theta=1e6)
    q, k = bf16(rs, 3, 5, 4, 64), bf16(rs, 3, 5, 2, 64)
    base, depth = np.array([0, 2 ** 31 - 1, 77777]), rs.randint(0, 2 ** 20, (3, 5))
    base_t, depth_t = torch.as_tensor(base, **i32), torch.as_tensor(depth, **i32)
    for kw, pos in ((dict(base=base_t, positions=depth_t), base[:, None] + depth), (dict(base=base_t), base[:, None] + np.arange(5)),
                    (dict(), np.zeros((3, 1), int) + np.arange(5)), (dict(positions=depth_t), depth)):
        qo, ko = qk_norm_rope(q, k, rotary=rotary, **kw)
        check_rotated(qo.view(15, 4, 64), q.view(15, 4, 64), pos.reshape(-1), rotary, None, 0)
        check_rotated(ko.view(15, 2, 64), k.view(15, 2, 64), pos.reshape(-1), rotary, None, 0)
    # rows behind the last token are left as they were, whatever the base
    depth_t[1, 2:] = -1
    depth_t[2, 0] = -(2 ** 31)
    room = [torch.full_like(t, 9.0) for t in (q, k)]
    qk_norm_rope(q, k, rotary=rotary, base=base_t, positions=depth_t, q_out=room[0], k_out=room[1])
    full = qk_norm_rope(q, k, rotary=rotary, base=base_t, positions=torch.as_tensor(depth, **i32))
    skipped = (depth_t < 0)
    for r, f in zip(room, full):
        assert (r[skipped] == 9).all() and torch.equal(r[~skipped], f[~skipped])
    # prompts in one row of tokens
    q1, k1 = q.view(15, 4, 64), k.view(15, 2, 64)
    a, b = qk_norm_rope(q1, k1, rotary=rotary, base=torch.as_tensor([40], **i32))
    check_rotated(a, q1, 40 + np.arange(15), rotary, None, 0)


def test_rotate_values_that_are_not_finite_and_empty_calls():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    rs = np.random.RandomState(9)
    q, k, w = bf16(rs, 6, 4, 128), bf16(rs, 6, 2, 128), bf16(rs, 128)
    rotary = Rotary(128)
    clean, kc = qk_norm_rope(q, k, rotary=rotary, q_weight=w, k_weight=w)
    q[3, 2, 17] = float("nan")
    q[4, 1] = 0
    out, ko = qk_norm_rope(q, k, rotary=rotary, q_weight=w, k_weight=w)
    assert out[3, 2].isnan().all() and (out[4, 1] == 0).all() and torch.equal(ko, kc)
    same = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    same[3, 2] = same[4, 1] = False
    assert torch.equal(out[same], clean[same])
    a, b = qk_norm_rope(q[:0], k[:0], rotary=rotary)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
    # far apart rows and heads
    room = torch.zeros(1 << 31, dtype=torch.bfloat16, device="cuda")
    far = room.as_strided((6, 4, 128), (1 << 28, 1 << 26, 1))
    far.copy_(q)
    out2, _ = qk_norm_rope(far, rotary=rotary, q_weight=w, q_out=far)
    assert torch.equal(out2.nan_to_num(), out.nan_to_num())


def test_scaled_frequencies():
    """Given frequencies in place of theta's, zero and negative ones among them."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    rs = np.random.RandomState(10)
    freq = rs.uniform(-3, 7, 32)
    freq[5] = 0
    rotary = Rotary(64, inv_freq=freq)
    q = bf16(rs, 9, 2, 64)
    pos = rs.randint(0, 2 ** 31, 9)
    out, _ = qk_norm_rope(q, positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary)
    check_rotated(out, q, pos, rotary, None, 0)


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------
def check_logp(x, tokens, top, T, found, rows=None):
    """A term 2^d is off by |d| 2^-23 (d, and log2 e / T, to fp32) and 2^-22 (the power), and small where |d| is large; sums
    of n terms in 256 parts by n / 256 + 16 roundings; logarithms and what is added to them by 2^-22 of themselves."""
    x64, tokens = f64(x), tokens.cpu().numpy()
    got = {k: f64(v) for k, v in found.items()}
    n = x64.shape[1]
    unit = (n / 256 + 64) * 2.0 ** -24
    for r in range(x64.shape[0]) if rows is None else rows:
        logp, lse, entropy, ids, best = ol.token_logprobs(x64[r], tokens[r], top, T)

        def near(a, b, off):
            a, b = np.asarray(a), np.asarray(b)
            same = (a == b) | (np.isnan(a) & np.isnan(b))
            with np.errstate(invalid="ignore"):
                assert (same | (np.abs(a - b) <= off)).all(), (r, a, b, off)
        with np.errstate(invalid="ignore"):
            near(got["lse"][r], lse, unit + abs(lse) * 2.0 ** -22)
            near(got["logp"][r], logp, unit + np.abs(logp) * 2.0 ** -22)
            near(got["entropy"][r], entropy, (1 + abs(entropy)) * 2 * unit)
            if top:
                assert got["top_tok"][r].astype(int).tolist() == list(ids), r
                near(got["top_logp"][r], best, unit + np.abs(best) * 2.0 ** -22)


@pytest.mark.parametrize("rows,vocab,n,top", [
    (1, 1, 1, 1), (2, 2, 3, 2), (3, 7, 1, 5), (5, 31, 2, 31), (1, 100, 1, 20), (9, 1000, 4, 33), (4, 4097, 1, 64), (1, 151936, 1, 20),
    (3, 50257, 2, 5), (17, 8191, 1, 32), (40, 2049, 1, 1), (700, 333, 1, 8), (2, 300007, 8, 64), (1, 70001, 0, 7), (6, 129, 3, 0)])
@pytest.mark.parametrize("full", [True, False])
def test_logprobs_sizes(rows, vocab, n, top, full):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(vocab + rows)
    x = torch.as_tensor(rs.standard_normal((rows, vocab)) * 4).to(torch.float32 if full else torch.bfloat16).cuda()
    tokens = torch.as_tensor(rs.randint(0, vocab, (rows, n)), dtype=torch.int32, device="cuda")
    T = [1.0, 0.6, 2.5][rows % 3]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    found = token_logprobs(x, tokens, top=top, temperature=T, status=status)
    check_logp(x, tokens, top, T, found, rows=None if rows < 50 else range(0, rows, 29))
    assert status.item() == 0


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("vocab,rows", [(5001, 3), (40000, 1), (333, 400)])
def test_logprobs_orders_and_ties(full, vocab, rows):
    """Ascending and descending logits, equal ones, blocks of equal ones, zeros of both signs: the lower token first."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(vocab)
    up = np.sort(rs.standard_normal(vocab)) * 5
    zeros = np.where(rs.rand(vocab) < 0.5, 0.0, -0.0)
    zeros[rs.randint(0, vocab, vocab // 3)] = -1.5
    for row in (up, up[::-1], np.zeros(vocab) + 3.25, np.floor(up), -np.abs(np.floor(rs.standard_normal(vocab))), zeros, np.arange(vocab) * 0.001 - 70000):
        x = torch.as_tensor(np.tile(row, (rows, 1))).to(torch.float32 if full else torch.bfloat16).cuda()
        tokens = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
        for top in (1, 20, 64):
            found = token_logprobs(x, tokens, top=top)
            check_logp(x, tokens, top, 1.0, found, rows=[0])
            assert torch.equal(found["top_tok"], found["top_tok"][:1].expand(rows, -1))


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("vocab,rows", [(5001, 7), (333, 400), (90001, 7)])
def test_logprobs_of_masked_rows_and_values_that_are_not_finite(full, vocab, rows):
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(vocab + 1)
    x = rs.standard_normal((rows, vocab)) * 3
    low = float(torch.finfo(torch.float32 if full else torch.bfloat16).min)
    x[0] = -np.inf                                       # nothing is left
    x[1, rs.rand(vocab) < 0.995] = -np.inf               # a few
    x[2] = -np.inf
    x[2, vocab - 2] = 1.0                                # one
    x[3, rs.rand(vocab) < 0.9] = low                     # a mask of the type's lowest value
    x[4, 5] = np.nan
    x[5, vocab - 1] = np.inf
    x[6] = low                                           # all of them equal
    x = torch.as_tensor(x).to(torch.float32 if full else torch.bfloat16).cuda()
    tokens = torch.as_tensor(rs.randint(0, vocab, (rows, 4)), dtype=torch.int32, device="cuda")
    tokens[2, 0] = vocab - 2
    tokens[:, 1] = -1
    for top in (0, 5, 40):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        found = token_logprobs(x, tokens, top=top, status=status)
        check_logp(x, tokens, top, 1.0, found, rows=range(min(rows, 9)))
        assert status.item() == 0
    # a token behind the vocabulary
    from conditional_draft_tree_lm_gb300.kvcache import KV_BAD_INDEX
    tokens[3, 2] = vocab
    tokens[0, 3] = 2 ** 31 - 1
    found = token_logprobs(x, tokens, status=status)
    check_logp(x, tokens, 0, 1.0, found, rows=range(7))
    assert status.item() == KV_BAD_INDEX
    token_logprobs(x, tokens)


@pytest.mark.parametrize("rows,vocab,top,full", [(2000, 5003, 5, True), (2000, 8192, 40, True), (1900, 20000, 5, False), (1900, 20011, 0, False),
                                                 (2000, 2000, 20, False), (400, 1999, 33, True)])
def test_logprobs_of_many_rows_with_and_without_masks(rows, vocab, top, full):
    """Rows that fill all places at once: by turns as they are, with a few logits left, with fewer than are asked for, and
    with logits in one stretch of the row only."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(rows + vocab)
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=gen, device="cuda") * 3
    keep = torch.rand(rows, vocab, generator=gen, device="cuda")
    x[1::4] = x[1::4].masked_fill(keep[1::4] > 60 / vocab, -math.inf)
    x[2::4] = x[2::4].masked_fill(keep[2::4] > 3 / vocab, -math.inf)
    x[3::4, vocab // 3 + 37:] = -math.inf
    x[3::4, :vocab // 3] = -math.inf
    x = x if full else x.to(torch.bfloat16)
    tokens = torch.as_tensor(rs.randint(0, vocab, (rows, 2)), dtype=torch.int32, device="cuda")
    found = token_logprobs(x, tokens, top=top)
    check_logp(x, tokens, top, 1.0, found, rows=[*range(8), *range(rows - 8, rows)])
    # every row as it is alone: read by several CTAs there
    for r in (0, 1, 2, 3, rows - 1):
        alone = token_logprobs(x[r:r + 1], tokens[r:r + 1], top=top)
        if top:
            assert torch.equal(alone["top_tok"][0], found["top_tok"][r])
        check_logp(x[r:r + 1], tokens[r:r + 1], top, 1.0, alone)


def test_logprobs_of_large_logits():
    """Near 10^4, where fp32 holds a thousandth: differences are kept, in rows read by one CTA and by several."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(4)
    x = torch.as_tensor(1e4 + rs.standard_normal((3, 60000)), dtype=torch.float32, device="cuda")
    x[1] -= 2e4
    x[2] = x[2] * 1e30
    tokens = torch.as_tensor(rs.randint(0, 60000, (3, 8)), dtype=torch.int32, device="cuda")
    for x in (x, x.repeat(200, 1)):
        tokens = tokens[:3].repeat(x.shape[0] // 3, 1)
        for T in (1.0, 0.5, 3.0):
            check_logp(x, tokens, 9, T, token_logprobs(x, tokens, top=9, temperature=T), rows=range(3))
    # quotients beyond fp32: what is beyond it in the end is infinite, the largest logit's probability is 1
    x = x[:1].clone()
    x[0, 7] = 1.5e4
    tokens = torch.tensor([[7, 8]], dtype=torch.int32, device="cuda")
    far = token_logprobs(x, tokens, top=1, temperature=2.0 ** -100)
    assert far["lse"].item() == np.float32(1.5e4) * 2.0 ** 100 and far["entropy"].item() == 0 and far["top_tok"].item() == 7
    assert far["logp"][0].tolist()[0] == 0 and far["logp"][0, 1].item() < -1e33
    x[0, 7] = 1e30
    far = token_logprobs(x, tokens, temperature=2.0 ** -100)
    assert far["lse"].item() == math.inf and far["entropy"].item() == 0 and far["logp"][0].tolist() == [0, -math.inf]


def test_logprobs_strides_shapes_and_given_outputs():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(6)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.as_tensor(rs.standard_normal((2, 3, 2100))).to(dtype).cuda()
        tokens = torch.as_tensor(rs.randint(0, 2000, (2, 3)), dtype=torch.int32, device="cuda")
        for off in (0, 1, 3, 8):
            x = wide[..., off:off + 2000]
            found = token_logprobs(x, tokens, top=3)
            assert found["logp"].shape == (2, 3) and found["top_tok"].shape == (2, 3, 3) and found["lse"].shape == (2, 3)
            flat = {k: v.reshape(6, -1) if k[:3] == "top" or k == "logp" else v.reshape(6) for k, v in found.items()}
            check_logp(x.reshape(6, 2000), tokens.view(6, 1), 3, 1.0, flat)
            again = token_logprobs(x, tokens, top=3, out={k: torch.zeros_like(v) for k, v in found.items()})
            assert all(torch.equal(again[k], found[k]) for k in found)
        one = token_logprobs(wide[0, 0], top=2)
        assert one["lse"].shape == () and one["top_tok"].shape == (2,) and "logp" not in one
        same = token_logprobs(wide[0, :1].expand(4, 2100))
        assert (same["lse"] == one["lse"]).all()
        none = token_logprobs(wide[:0], tokens[:0], top=2)
        assert none["logp"].shape == (0, 3) and none["top_tok"].shape == (0, 3, 2)
    # rows behind 32 bits
    x = torch.zeros(9, 1 << 28, device="cuda")[:, 5:3005]
    x.copy_(torch.as_tensor(rs.standard_normal((9, 3000))))
    tokens = torch.as_tensor(rs.randint(0, 3000, (9, 2)), dtype=torch.int32, device="cuda")
    check_logp(x, tokens, 4, 1.0, token_logprobs(x, tokens, top=4))


def test_logprobs_repeat_their_bits_beside_others_and_replayed():
    torch = _t()
    from conditional_draft_tree_lm_gb300 import token_logprobs
    rs = np.random.RandomState(7)
    a = torch.as_tensor(rs.standard_normal((2, 151936)) * 3, dtype=torch.float32, device="cuda")
    b = torch.as_tensor(rs.standard_normal((500, 20001)) * 3).to(torch.bfloat16).cuda()
    ta, tb = (torch.as_tensor(rs.randint(0, x.shape[1], (x.shape[0], 2)), dtype=torch.int32, device="cuda") for x in (a, b))
    wa, wb = token_logprobs(a, ta, top=30), token_logprobs(b, tb, top=5)
    ga, gb = ({k: torch.zeros_like(v) for k, v in w.items()} for w in (wa, wb))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        token_logprobs(b, tb, top=5, out=gb, stream=side)
        token_logprobs(a, ta, top=30, out=ga)
    torch.cuda.synchronize()
    assert all(torch.equal(w[k], g[k]) for w, g in ((wa, ga), (wb, gb)) for k in w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token_logprobs(a, ta, top=30, out=ga)
    a.neg_()
    graph.replay()
    fresh = token_logprobs(a, ta, top=30)
    torch.cuda.synchronize()
    assert all(torch.equal(fresh[k], ga[k]) for k in fresh)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_layer_read_as_a_prompt_and_token_by_token():
    """Two layers of a small target over packed prompts, then the same tokens as drafted chains over the 8-bit cache: the
    new operators between the cache's, each checked against its definition on the inputs that it met."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import (AttentionWorkspace, KvCache, Rotary, cache_attention, kv_append, linear, prompt_attention,
                                                 qk_norm_rope, token_logprobs)
    rs = np.random.RandomState(12)
    d, heads, kv, dim, ffn, vocab = 256, 8, 2, 64, 520, 1000
    rotary, work = Rotary(dim, theta=1e6), AttentionWorkspace()
    emb, head = bf16(rs, vocab, d), bf16(rs, vocab, d, scale=d ** -0.5)
    layers = [dict(qkv=bf16(rs, (heads + 2 * kv) * dim, d, scale=d ** -0.5), b=bf16(rs, (heads + 2 * kv) * dim, scale=0.1), qw=bf16(rs, dim) * 0.1 + 1,
                   kw=bf16(rs, dim) * 0.1 + 1, out=bf16(rs, d, heads * dim, scale=0.05), up=bf16(rs, ffn, d, scale=d ** -0.5),
                   gate=bf16(rs, ffn, d, scale=d ** -0.5), down=bf16(rs, d, ffn, scale=0.05)) for _ in range(2)]
    lens, new = [37, 90], 5
    start = torch.as_tensor([0, 37, 127], dtype=torch.int32, device="cuda")
    tokens = torch.as_tensor(rs.randint(0, vocab, 127), dtype=torch.int32, device="cuda")
    page, blocks = 16, 8
    caches = [KvCache.empty(2 * blocks, page, kv, dim) for _ in layers]
    table = torch.arange(2 * blocks, dtype=torch.int32, device="cuda").view(2, blocks)

    def forward(toks, positions, base, attend):
        x = emb[toks.long()]
        lead = toks.shape
        for i, w in enumerate(layers):
            c = dict(x=x, weight=w["qkv"], bias=w["b"], activation=None)
            qkv = linear(**c)
            check_linear({**c, "x": x.view(-1, d)}, qkv.view(-1, qkv.shape[-1]))
            qkv = qkv.view(*lead, heads + 2 * kv, dim)
            q0, k0, v = qkv[..., :heads, :], qkv[..., heads:heads + kv, :], qkv[..., heads + kv:, :]
            q, k = qk_norm_rope(q0, k0, positions=positions, base=base, rotary=rotary, q_weight=w["qw"], k_weight=w["kw"])
            at = (positions if base is None else positions + base[:, None]).reshape(-1).tolist()
            check_rotated(k.reshape(-1, kv, dim), k0.reshape(-1, kv, dim), at, rotary, w["kw"], 1e-6)
            h = attend(i, q, k, v).reshape(*lead, heads * dim)
            c = dict(x=h, weight=w["out"], residual=x, activation=None)
            x = linear(**c)
            check_linear({**c, "x": h.view(-1, heads * dim), "residual": c["residual"].view(-1, d)}, x.view(-1, d))
            c = dict(x=x, weight=w["up"], gate=w["gate"], activation="silu")
            h = linear(**c)
            check_linear({**c, "x": x.view(-1, d)}, h.view(-1, ffn))
            x = linear(h, w["down"], residual=x, out=x)
        return linear(x, head, out_dtype=torch.float32)

    def prompts(i, q, k, v):
        # all but the last tokens of each go into the cache
        slot = torch.full((127,), -1, dtype=torch.int64, device="cuda")
        for s, n in enumerate(lens):
            r = torch.arange(n - new, device="cuda")
            slot[sum(lens[:s]):][:n - new] = s * blocks * page + r
        kv_append(caches[i], k, v, slot)
        return prompt_attention(q, k, v, start)

    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    logits = forward(tokens, pos, None, prompts)
    want = token_logprobs(logits, tokens.roll(-1), top=4)
    check_logp(logits, tokens.roll(-1)[:, None], 4, 1.0, {**want, "logp": want["logp"][:, None]}, rows=range(0, 127, 9))
    # the last tokens of each, as one drafted chain over what is cached
    last = torch.stack([tokens[37 - new:37], tokens[127 - new:]])
    held = torch.as_tensor([n - new for n in lens], dtype=torch.int32, device="cuda")
    depth = torch.arange(new, dtype=torch.int32, device="cuda").expand(2, new).contiguous()
    tree = forward(last, depth, held, lambda i, q, k, v: cache_attention(caches[i], q, table, held, k_new=k, v_new=v, workspace=work))
    asked = last.roll(-1, 1).contiguous()
    got = token_logprobs(tree, asked, top=4)
    assert got["logp"].shape == (2, new) and got["top_tok"].shape == (2, new, 4)
    check_logp(tree.view(2 * new, vocab), asked.view(-1, 1), 4, 1.0,
               {k: v.reshape(2 * new, -1) if k[:3] == "top" or k == "logp" else v.reshape(-1) for k, v in got.items()})


@pytest.mark.parametrize("rows,inner", [(1, 2048), (2, 2048), (20, 1024), (65, 10240), (300, 512)])
def test_calls_that_follow_one_another_see_what_was_written(rows, inner):
    """A call may begin while the one before it ends: the same bits as with a wait between the calls, behind other kernels, copies and
    fills, in one stream and in a captured graph with branches."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, linear, qk_norm_rope, token_logprobs
    rs = np.random.RandomState(rows)
    source = [bf16(rs, rows, inner) for _ in range(3)]
    w, back = bf16(rs, inner, inner, scale=inner ** -0.5), bf16(rs, inner, inner, scale=inner ** -0.5)
    rotary, norm = Rotary(128), bf16(rs, 128)
    tokens = torch.as_tensor(rs.randint(0, inner, (rows, 2)), dtype=torch.int32, device="cuda")
    x, h, q = (torch.empty_like(source[0]) for _ in range(3))
    logits = torch.empty(rows, inner, device="cuda")
    side = torch.cuda.Stream()

    def chain(n, wait, branch):
        for i in range(n):
            x.copy_(source[i % 3])
            wait()
            if branch:  # a second stream's result joins before the next call
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    h.zero_()
                torch.cuda.current_stream().wait_stream(side)
            linear(x, w, out=h)
            wait()
            qk_norm_rope(h.view(rows, inner // 128, 128), rotary=rotary, q_weight=norm, q_out=q.view(rows, inner // 128, 128))
            wait()
            linear(q, back, gate=w, activation="silu", residual=x, out=x)
            wait()
            x.mul_(0.5)
            linear(x, w, out=logits)
            wait()
            found = token_logprobs(logits, tokens, top=4)
            wait()
        return [t.clone() for t in (x, h, q, logits, *found.values())]

    for n in (1, 2, 3):
        want = chain(n, torch.cuda.synchronize, False)
        for _ in range(5):
            got = chain(n, lambda: None, True)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(n, lambda: None, True)
        for _ in range(5):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,outer", [(1, 1024), (20, 1024), (65, 10240), (300, 1024)])
def test_a_call_behind_another_streams_late_event_waits_for_it(rows, outer):
    """The kernel before the call in its own stream is long done, and is one of the same kind; what the call reads comes late from another."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import Rotary, linear, qk_norm_rope, token_logprobs
    rs = np.random.RandomState(rows)
    x, w = bf16(rs, rows, 1024), bf16(rs, outer, 1024, scale=0.03)
    late, rotary, side = torch.zeros_like(x), Rotary(128), torch.cuda.Stream()
    heads = late.view(rows, 8, 128)
    calls = [lambda: linear(late, w), lambda: qk_norm_rope(heads, rotary=rotary)[0], lambda: token_logprobs(late, top=4)["top_logp"]]

    def run(call):
        late.zero_()
        call()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000)
            late.copy_(x)
        torch.cuda.current_stream().wait_stream(side)
        return call()

    for call in calls:
        late.copy_(x)
        want = call().clone()
        for _ in range(3):
            assert torch.equal(run(call), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(call)
        for _ in range(3):
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
