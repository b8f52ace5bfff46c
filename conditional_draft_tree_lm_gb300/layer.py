"""A target layer around its attention (argument marshalling only).

Binding of ``dt_linear``, ``dt_qk_norm_rope`` and ``dt_token_logprobs`` of
``include/dtree.h``, which states formulas, layouts and errors.  A layer, between
whose calls those of ``kvcache`` stand, and with norm() for the norms of the hidden states, which
are the caller's (torch's ``rms_norm``, say)::

    qkv = linear(norm(x), w_qkv)                          # [rows, heads + 2 kv heads, head_dim], sliced
    q, k = qk_norm_rope(q, k, positions=..., rotary=...)  # norms and rotation
    ...                                                   # prompt_attention, kv_append, cache_attention
    x = linear(attended, w_out, residual=x)
    y = norm(x)
    h = linear(y, w_up, gate=w_gate, activation="silu")
    x = linear(h, w_down, residual=x)
    logits = linear(norm(x), head, out_dtype=torch.float32)  # accept_walk's input
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
    shape, st = t.shape, t.stride()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the others on cuda:{index}")
    if len(shape) == 2 and shape[1] == cols and st[1] == 1:
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


def _head_rows(t, shape, dtype, name, index):
    """As ``kvcache._heads``, in a shorter way for the usual strides."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        st = t.stride()
        if len(st) == 4:
            n, slots, heads, _ = shape
            if st[3] == 1 and heads > 1 and n > 1 and (slots == 1 or st[0] == st[1] * slots):
                return t.data_ptr(), st[0] if slots == 1 else st[1], st[2]
        elif st[2] == 1 and shape[0] > 1 and shape[1] > 1:
            return t.data_ptr(), st[0], st[1]
    return _heads(t, tuple(shape[:-2]), shape[-2], shape[-1], name, index)


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
    bf16, i32, shape = torch.bfloat16, torch.int32, q.shape
    if len(shape) == 4:
        n_req, slots, heads, dim = shape
    elif len(shape) == 3:
        n_req, (slots, heads, dim) = 1, shape
    else:
        raise ValueError("q: expected [rows, heads, head_dim] or [n_req, slots, heads, head_dim]")
    rows, kv, k_shape = n_req * slots, 0, None
    if k is not None:
        k_shape = k.shape
        kv = k_shape[-2] if len(k_shape) == len(shape) else 0
        if kv == 0 or k_shape[-1] != dim or k_shape[0] != shape[0] or (len(shape) == 4 and k_shape[1] != slots):
            raise ValueError(f"k: expected {(*shape[:-2], 'heads', dim)}, got {tuple(k.shape)}")
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out or k_weight without k")
    if q_out is None or (k is not None and k_out is None):
        with _allocating(stream):
            q_out = torch.empty(shape, dtype=bf16, device=q.device) if q_out is None else q_out
            k_out = torch.empty(k_shape, dtype=bf16, device=q.device) if k is not None and k_out is None else k_out
    kp = kr = kh = kop = kor = koh = 0
    if rows:
        qp, qr, qh = _head_rows(q, shape, bf16, "q", dev)
        qop, qor, qoh = _head_rows(q_out, shape, bf16, "q_out", dev)
        if k is not None:
            kp, kr, kh = _head_rows(k, k_shape, bf16, "k", dev)
            kop, kor, koh = _head_rows(k_out, k_shape, bf16, "k_out", dev)
    else:
        qp = qr = qh = qop = qor = qoh = 0
        for t, s, name in ((q, shape, "q"), (q_out, shape, "q_out"), (k, k_shape, "k"), (k_out, k_shape, "k_out")):
            if t is not None and (t.shape != s or t.dtype is not bf16):
                raise ValueError(f"{name}: expected {tuple(s)} {bf16}, got {tuple(t.shape)} {t.dtype}")
    if rotary is None:
        rot, inter, amplitude, turns = 0, 0, 1.0, 0
    else:
        rot, inter, amplitude = rotary.dim, rotary.interleaved, rotary.amplitude
        turns = _flat(rotary.turns, torch.int64, rot // 2, "rotary.turns", dev)
    a = _pack_rotate(n_req, slots, heads, kv, dim, rot, inter, eps, amplitude, qp, kp, qr, qh, kr, kh,
                     0 if q_weight is None else _flat(q_weight, bf16, dim, "q_weight", dev),
                     0 if k_weight is None else _flat(k_weight, bf16, dim, "k_weight", dev), turns,
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
    i32, f32, shape, at = torch.int32, torch.float32, logits.shape, logits.device
    if not shape:
        raise ValueError("logits: expected [..., vocab]")
    if top < 0:
        raise ValueError(f"top: {top} is negative")
    vocab, lead = shape[-1], shape[:-1]
    lp, rows, ls = _rows(logits, vocab, (f32, torch.bfloat16), "logits", dev)
    n = tp = 0
    if tokens is not None:
        asked = tokens.shape
        if asked == lead:
            n = 1
        elif len(asked) == len(shape) and asked[:-1] == lead:
            n = asked[-1]
        else:
            raise ValueError(f"tokens: expected {tuple(lead)} or {(*lead, 'n')}, got {tuple(asked)}")
        tp = _flat(tokens, i32, rows * n, "tokens", dev)
    best = (*lead, top)
    with _allocating(stream):
        if out is None:
            empty = torch.empty
            lse, entropy = empty(lead, dtype=f32, device=at), empty(lead, dtype=f32, device=at)
            found = {"lse": lse, "entropy": entropy}
            pointers = [0, lse.data_ptr(), entropy.data_ptr(), 0, 0]
            if tokens is not None:
                found["logp"] = logp = empty(asked, dtype=f32, device=at)
                pointers[0] = logp.data_ptr()
            if top:
                found["top_tok"], found["top_logp"] = ids, values = empty(best, dtype=i32, device=at), empty(best, dtype=f32, device=at)
                pointers[3:] = ids.data_ptr(), values.data_ptr()
        else:
            found, pointers = {}, []
            for name, size, dtype in (("logp", asked if tokens is not None else None, f32), ("lse", lead, f32), ("entropy", lead, f32),
                                      ("top_tok", best if top else None, i32), ("top_logp", best if top else None, f32)):
                if size is None:
                    pointers.append(0)
                    continue
                t = out.get(name)
                if t is None:
                    t = torch.empty(size, dtype=dtype, device=at)
                elif tuple(t.shape) != tuple(size):
                    raise ValueError(f"out[{name!r}]: expected {tuple(size)}, got {tuple(t.shape)}")
                found[name] = t
                pointers.append(_flat(t, dtype, t.numel(), name, dev))
    a = _pack_logprobs(rows, vocab, n, top, logits.dtype is not f32, temperature, lp, ls, tp, *pointers, _status(status, dev))
    raw = kvcache._stream(stream, dev)
    if rows:
        err = lib.dt_token_logprobs(a, raw)
        if err:
            raise _refused(err, "dt_token_logprobs")
    return found
