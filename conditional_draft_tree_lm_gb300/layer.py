"""A target layer around its attention (argument marshalling only).

Binding of ``dt_linear``, ``dt_qk_norm_rope`` and ``dt_token_logprobs`` of
``include/dtree.h``, which states formulas, layouts and errors.  A layer, between
whose calls those of ``kvcache`` stand::

    qkv = linear(x, w_qkv)                                # [rows, heads + 2 kv heads, head_dim], sliced
    q, k = qk_norm_rope(q, k, positions=..., rotary=...)  # norms and rotation
    ...                                                   # prompt_attention, kv_append, cache_attention
    x = linear(attended, w_out, residual=x)
    h = linear(x, w_up, gate=w_gate, activation="silu")
    x = linear(h, w_down, residual=x)
    logits = linear(x, head, out_dtype=torch.float32)     # accept_walk's input
    found = token_logprobs(logits, tokens, top=5)

As for the cache's calls, nothing here computes: tensors become pointers, a refused
call raises ``ValueError``, ``TypeError`` or ``DtreeError``.  Each takes a ``stream``;
``linear`` and ``token_logprobs`` a ``status`` word on the device too (``KV_*`` bits).
"""
from __future__ import annotations

import ctypes
from ctypes import c_float, c_int, c_int64, c_void_p
from fractions import Fraction

from . import kvcache
from .dtree import DtreeError, load_library
from .kvcache import _allocating, _flat, _heads, _on_device, _packer

ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


class _Linear(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("inner", c_int), ("outer", c_int), ("x", c_void_p), ("x_row_stride", c_int64),
                ("weight", c_void_p), ("weight_row_stride", c_int64), ("bias", c_void_p), ("gate", c_void_p),
                ("gate_row_stride", c_int64), ("gate_bias", c_void_p), ("activation", c_int), ("residual", c_void_p),
                ("residual_row_stride", c_int64), ("out", c_void_p), ("out_row_stride", c_int64), ("out_fp32", c_int),
                ("status", c_void_p)]


class _Rotate(ctypes.Structure):
    _fields_ = [(n, c_int) for n in ("n_req", "slots", "n_q", "n_kv", "head_dim", "rot", "interleaved")] + \
        [("eps", c_float), ("amplitude", c_float), ("q", c_void_p), ("k", c_void_p)] + \
        [(n, c_int64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride")] + \
        [(n, c_void_p) for n in ("q_weight", "k_weight", "turns", "positions", "base", "q_out", "k_out")] + \
        [(n, c_int64) for n in ("q_out_row_stride", "q_out_head_stride", "k_out_row_stride", "k_out_head_stride")]


class _Logprobs(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("vocab", c_int), ("n_tokens", c_int), ("n_top", c_int), ("logits_bf16", c_int),
                ("temperature", c_float), ("logits", c_void_p), ("logits_row_stride", c_int64)] + \
        [(n, c_void_p) for n in ("tokens", "logp", "lse", "entropy", "top_tok", "top_logp", "status")]


_pack_linear, _pack_rotate, _pack_logprobs = map(_packer, (_Linear, _Rotate, _Logprobs))

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        for name in ("dt_linear", "dt_qk_norm_rope", "dt_token_logprobs"):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = c_int, [c_void_p] * 2
        _lib = lib
    return _lib


def _refused(status, where):
    return DtreeError(status, where + ": " + _lib.dt_last_error().decode(errors="replace"))


def _rows(t, cols, dtypes, name, index):
    """Pointer, number of rows and row stride of a tensor [..., cols] of one of `dtypes`, whose columns are adjacent and
    whose leading dimensions fold into one row index (the stride of a dimension of one entry is not looked at)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the others on cuda:{index}")
    shape, st = t.shape, t.stride()
    if len(shape) == 2 and shape[1] == cols and (st[1] == 1 or cols == 1):
        return t.data_ptr(), shape[0], st[0] if shape[0] > 1 else cols
    if len(shape) < 1 or shape[-1] != cols:
        raise ValueError(f"{name}: expected [..., {cols}], got {tuple(shape)}")
    rows, stride = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n != 1 and rows not in (0, 1) and s != stride * rows:
            raise ValueError(f"{name}: strides {st}: rows must be evenly spaced")
        stride = s if n != 1 and stride is None else stride
        rows *= n
    if cols > 1 and st[-1] != 1:
        raise ValueError(f"{name}: strides {st}: columns must be adjacent")
    return t.data_ptr(), rows, cols if stride is None else stride


def _status(status, index):
    import torch
    return 0 if status is None else _flat(status, torch.int32, 1, "status", index)


def linear(x, weight, *, bias=None, gate=None, gate_bias=None, activation=None, residual=None, out=None, out_dtype=None,
           status=None, stream=None):
    """Matrix product with its epilogue (``dt_linear``): act(x W^T + bias) + residual, or with ``gate``
    act(x G^T + gate_bias) * (x W^T + bias) + residual.

    x [..., inner], weight and gate [outer, inner], bias and gate_bias [outer], residual [..., outer] bf16; rows may be
    strided (halves of a joint weight).  activation: None, "relu", "silu", "gelu" or "gelu_tanh".  Returns out
    [..., outer] in bf16 or ``out_dtype`` torch.float32; ``out`` may be ``residual`` itself."""
    import torch
    lib = _library()
    bf16 = (torch.bfloat16,)
    dev = _on_device(x, "x")
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError("x: expected [..., inner], weight: [outer, inner]")
    outer, inner = weight.shape
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation: expected one of {list(ACTIVATIONS)}, got {activation!r}")
    xp, rows, xs = _rows(x, inner, bf16, "x", dev)
    wp, _, ws = _rows(weight, inner, bf16, "weight", dev)
    gp = gs = rp = rs = 0
    shape = (*x.shape[:-1], outer)
    if gate is not None:
        if gate.shape != weight.shape:
            raise ValueError(f"gate: expected {tuple(weight.shape)}, got {tuple(gate.shape)}")
        gp, _, gs = _rows(gate, inner, bf16, "gate", dev)
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual: expected {shape}, got {tuple(residual.shape)}")
        rp, _, rs = _rows(residual, outer, bf16, "residual", dev)
    if out is None:
        with _allocating(stream):
            out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=x.device)
    elif out.shape != shape or (out_dtype is not None and out.dtype is not out_dtype):
        raise ValueError(f"out: expected {shape} {out_dtype or ''}, got {tuple(out.shape)} {out.dtype}")
    op, _, os = _rows(out, outer, (torch.bfloat16, torch.float32), "out", dev)
    a = _pack_linear(rows, inner, outer, xp, xs, wp, ws, 0 if bias is None else _flat(bias, torch.bfloat16, outer, "bias", dev), gp, gs,
                     0 if gate_bias is None else _flat(gate_bias, torch.bfloat16, outer, "gate_bias", dev), ACTIVATIONS[activation],
                     rp, rs, op, os, out.dtype is torch.float32, _status(status, dev))
    err = lib.dt_linear(a, kvcache._stream(stream, dev))
    if err:
        raise _refused(err, "dt_linear")
    return out


# 2 pi to 40 digits
_TWO_PI = Fraction(6283185307179586476925286766559005768394, 10 ** 39)


class Rotary:
    """What ``qk_norm_rope`` turns by: ``turns`` [dim / 2], the part of a full turn of one position's step, in units of
    2^-64 (as torch.int64, the upper half as negative numbers).

    Pair i turns by ``inv_freq[i]`` radians a position: theta ** (-2 i / dim), or the values given (of scaled
    variants), in 64 bits.  interleaved: pairs are (2 i, 2 i + 1), not (i, i + dim / 2).  amplitude multiplies what is
    turned."""

    def __init__(self, dim, theta=10000.0, *, inv_freq=None, interleaved=False, amplitude=1.0, device="cuda"):
        import torch
        if dim < 2 or dim % 2:
            raise ValueError(f"dim: expected an even number, got {dim}")
        freq = [float(theta) ** (-2 * i / dim) for i in range(dim // 2)] if inv_freq is None else [float(f) for f in inv_freq]
        if len(freq) != dim // 2:
            raise ValueError(f"inv_freq: expected {dim // 2} values, got {len(freq)}")
        if not all(abs(f) < float("inf") for f in freq):
            raise ValueError("inv_freq: values must be finite")
        turns = [round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64 for f in freq]
        self.dim, self.interleaved, self.amplitude, self.inv_freq = dim, bool(interleaved), float(amplitude), freq
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64).to(device)


def qk_norm_rope(q, k=None, *, positions=None, base=None, rotary=None, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                 k_out=None, stream=None):
    """Norms of queries and keys for each head and their rotation by position (``dt_qk_norm_rope``).

    q [rows, n_q, head_dim] or [n_req, slots, n_q, head_dim] bf16, k likewise with its own heads; rows and heads may be
    strided (slices of a projection's output).  Position of a row: ``positions`` int32 [rows] (or [n_req, slots]; its number
    in its request where not given) plus ``base`` int32 [n_req].  So packed prompts take ``kv_plan``'s positions, a drafted
    tree its depths and the requests' lengths.  Rows whose positions entry is negative are not written.
    q_weight, k_weight [head_dim] bf16: the norms' weights, no norm where not given.  Returns (q_out, k_out), new
    tensors unless given; in place with q_out=q, k_out=k."""
    import torch
    lib = _library()
    dev = _on_device(q, "q")
    if q.dim() not in (3, 4):
        raise ValueError("q: expected [rows, heads, head_dim] or [n_req, slots, heads, head_dim]")
    lead = tuple(q.shape[:-2])
    heads, dim = q.shape[-2:]
    n_req, slots = lead if len(lead) == 2 else (1, lead[0])
    rows = n_req * slots

    def of(t, n, name):
        if t is not None and rows == 0:
            if t.shape != (*lead, n, dim) or t.dtype is not torch.bfloat16:
                raise ValueError(f"{name}: expected {(*lead, n, dim)} torch.bfloat16, got {tuple(t.shape)} {t.dtype}")
            return 0, 0, 0
        return (0, 0, 0) if t is None else _heads(t, lead, n, dim, name, dev)

    kv = 0
    if k is not None:
        if k.dim() != q.dim():
            raise ValueError("k: expected as many dimensions as q")
        kv = k.shape[-2]
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out or k_weight without k")
    if q_out is None or (k is not None and k_out is None):
        with _allocating(stream):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device) if k is not None and k_out is None else k_out
    qp, qr, qh = of(q, heads, "q")
    kp, kr, kh = of(k, kv, "k")
    qop, qor, qoh = of(q_out, heads, "q_out")
    kop, kor, koh = of(k_out, kv, "k_out")
    bf16, i32 = torch.bfloat16, torch.int32
    a = _pack_rotate(n_req, slots, heads, kv, dim, 0 if rotary is None else rotary.dim, rotary is not None and rotary.interleaved,
                     eps, 1.0 if rotary is None else rotary.amplitude, qp, kp, qr, qh, kr, kh,
                     0 if q_weight is None else _flat(q_weight, bf16, dim, "q_weight", dev),
                     0 if k_weight is None else _flat(k_weight, bf16, dim, "k_weight", dev),
                     0 if rotary is None else _flat(rotary.turns, torch.int64, rotary.dim // 2, "rotary.turns", dev),
                     0 if positions is None else _flat(positions, i32, rows, "positions", dev),
                     0 if base is None else _flat(base, i32, n_req, "base", dev), qop, kop, qor, qoh, kor, koh)
    raw = kvcache._stream(stream, dev)
    if rows:
        err = lib.dt_qk_norm_rope(a, raw)
        if err:
            raise _refused(err, "dt_qk_norm_rope")
    return q_out, k_out


def token_logprobs(logits, tokens=None, *, top=0, temperature=1.0, out=None, status=None, stream=None):
    """Log probabilities of given tokens, with entropy and the best alternatives (``dt_token_logprobs``).

    logits [..., vocab] fp32 or bf16, rows may be strided; tokens int32 [..., n] or [...] (one a row).  Returns a dict of
    logp (like tokens), lse and entropy [...] and, with top > 0, top_tok int32 and top_logp [..., top], all fp32 but the
    token ids; tensors of an earlier call's dict given as ``out`` are filled instead."""
    import torch
    lib = _library()
    dev = _on_device(logits, "logits")
    if logits.dim() < 1:
        raise ValueError("logits: expected [..., vocab]")
    vocab, lead = logits.shape[-1], tuple(logits.shape[:-1])
    lp, rows, ls = _rows(logits, vocab, (torch.float32, torch.bfloat16), "logits", dev)
    n = 0
    if tokens is not None:
        if tuple(tokens.shape[:len(lead)]) != lead or tokens.dim() - len(lead) not in (0, 1):
            raise ValueError(f"tokens: expected {lead} or {(*lead, 'n')}, got {tuple(tokens.shape)}")
        n = tokens.shape[-1] if tokens.dim() > len(lead) else 1
    i32, f32 = torch.int32, torch.float32
    want = {"lse": (lead, f32), "entropy": (lead, f32)}
    if tokens is not None:
        want["logp"] = (tuple(tokens.shape), f32)
    if top:
        want["top_tok"], want["top_logp"] = ((*lead, top), i32), ((*lead, top), f32)
    found = {}
    with _allocating(stream):
        for name, (shape, dtype) in want.items():
            t = None if out is None else out.get(name)
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=logits.device)
            elif tuple(t.shape) != shape:
                raise ValueError(f"out[{name!r}]: expected {shape}, got {tuple(t.shape)}")
            found[name] = t
    at = {name: _flat(t, want[name][1], rows * (n if name == "logp" else top if name.startswith("top") else 1), name, dev)
          for name, t in found.items()}
    a = _pack_logprobs(rows, vocab, n, top, logits.dtype is torch.bfloat16, temperature, lp, ls,
                       0 if tokens is None else _flat(tokens, i32, rows * n, "tokens", dev), at.get("logp", 0), at["lse"],
                       at["entropy"], at.get("top_tok", 0), at.get("top_logp", 0), _status(status, dev))
    raw = kvcache._stream(stream, dev)
    if rows:
        err = lib.dt_token_logprobs(a, raw)
        if err:
            raise _refused(err, "dt_token_logprobs")
    return found
