"""The layer's calls on the host: what they refuse before anything is launched (CPU, no GPU call)."""
import ctypes

import pytest

from conditional_draft_tree_lm_gb300 import kvcache as kc
from conditional_draft_tree_lm_gb300 import layer as ly

INVALID, SHAPE = 1, 2


@pytest.fixture(scope="module")
def lib():
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    dtbuild.build_library()
    return ly._library()


def call(lib, name, a):
    return getattr(lib, name)(ctypes.byref(a), None), lib.dt_last_error().decode()


def linear_args(**kw):
    a = ly._Linear(rows=4, inner=64, outer=48, x=256, x_row_stride=64, weight=512, weight_row_stride=64, out=1024, out_row_stride=48)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code,text", [
    (dict(rows=-1), SHAPE, "rows"), (dict(rows=2 ** 31), SHAPE, "rows"), (dict(outer=0), SHAPE, "outer"),
    (dict(inner=0), SHAPE, "inner"), (dict(inner=60), SHAPE, "multiple of 8"), (dict(activation=5), INVALID, "activation"),
    (dict(activation=-1), INVALID, "activation"), (dict(gate_bias=256), INVALID, "without a gate"), (dict(x=0), INVALID, "null"),
    (dict(x=264), INVALID, "misaligned"), (dict(weight=0), INVALID, "null"), (dict(x_row_stride=56), INVALID, "overlap"),
    (dict(x_row_stride=68), INVALID, "multiples of 8"), (dict(weight_row_stride=0), INVALID, "overlap"),
    (dict(gate=256, gate_row_stride=8), INVALID, "overlap"), (dict(out=0), INVALID, "out"), (dict(out=1025), INVALID, "out"),
    (dict(out=1026, out_fp32=1), INVALID, "out"), (dict(out_row_stride=47), INVALID, "overlap"), (dict(residual=257), INVALID, "residual"),
    (dict(bias=1), INVALID, "bias")])
def test_linear_refuses(lib, kw, code, text):
    err, msg = call(lib, "dt_linear", linear_args(**kw))
    assert err == code and text in msg and "dt_linear" in msg


def test_null_arguments_are_refused(lib):
    for name in ("dt_linear", "dt_qk_norm_rope", "dt_token_logprobs"):
        assert getattr(lib, name)(None, None) == INVALID


def rotate_args(**kw):
    a = ly._Rotate(n_req=2, slots=3, n_q=4, n_kv=2, head_dim=64, rot=64, eps=1e-6, amplitude=1.0, q=256, k=512, q_row_stride=256, q_head_stride=64,
                   k_row_stride=128, k_head_stride=64, turns=256, q_out=1024, k_out=2048, q_out_row_stride=256, q_out_head_stride=64,
                   k_out_row_stride=128, k_out_head_stride=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INF = float("inf")


@pytest.mark.parametrize("kw,code,text", [
    (dict(n_req=-1), INVALID, "n_req"), (dict(n_q=0), INVALID, "n_q"), (dict(n_kv=0), INVALID, "n_kv"), (dict(n_q=5000), SHAPE, "4096"),
    (dict(n_req=2 ** 20, slots=2 ** 12), SHAPE, "rows"), (dict(head_dim=16), SHAPE, "head_dim"), (dict(head_dim=72), SHAPE, "head_dim"),
    (dict(head_dim=272), SHAPE, "head_dim"), (dict(rot=72), SHAPE, "rot"), (dict(rot=8), SHAPE, "rot"), (dict(rot=80), SHAPE, "rot"),
    (dict(rot=0), SHAPE, "rot"), (dict(turns=0), SHAPE, "rot"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=INF), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(amplitude=INF), INVALID, "amplitude"), (dict(turns=0, rot=0), INVALID, "neither"),
    (dict(q=0), INVALID, "null"), (dict(q=264), INVALID, "misaligned"), (dict(q_row_stride=4), INVALID, "misaligned"), (dict(k_out=0), INVALID, "null"),
    (dict(q_weight=8), INVALID, "weights"), (dict(turns=4), INVALID, "turns"), (dict(q_out_row_stride=128), INVALID, "overlap"),
    (dict(k_out_head_stride=0), INVALID, "overlap")])
def test_qk_norm_rope_refuses(lib, kw, code, text):
    err, msg = call(lib, "dt_qk_norm_rope", rotate_args(**kw))
    assert err == code and text in msg and "dt_qk_norm_rope" in msg


def logp_args(**kw):
    a = ly._Logprobs(rows=2, vocab=100, n_tokens=1, n_top=2, temperature=1.0, logits=256, logits_row_stride=100, tokens=256, logp=256,
                     top_tok=256, top_logp=256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code,text", [
    (dict(rows=-1), SHAPE, "rows"), (dict(rows=2 ** 26 + 1), SHAPE, "rows"), (dict(vocab=0), SHAPE, "vocab"), (dict(vocab=2 ** 30 + 1), SHAPE, "vocab"),
    (dict(n_tokens=-1), SHAPE, "n_tokens"), (dict(n_tokens=65537), SHAPE, "n_tokens"), (dict(n_top=65), SHAPE, "n_top"), (dict(n_top=-1), SHAPE, "n_top"),
    (dict(vocab=1), SHAPE, "n_top"), (dict(temperature=0.0), INVALID, "temperature"), (dict(temperature=-1.0), INVALID, "temperature"),
    (dict(temperature=INF), INVALID, "temperature"), (dict(temperature=float("nan")), INVALID, "temperature"), (dict(temperature=1e-31), INVALID, "temperature"),
    (dict(logits=0), INVALID, "logits"), (dict(logits=258), INVALID, "misaligned"), (dict(logits=257, logits_bf16=1), INVALID, "misaligned"),
    (dict(tokens=0), INVALID, "null"), (dict(logp=0), INVALID, "null"), (dict(top_tok=0), INVALID, "null"), (dict(top_logp=0), INVALID, "null")])
def test_token_logprobs_refuses(lib, kw, code, text):
    err, msg = call(lib, "dt_token_logprobs", logp_args(**kw))
    assert err == code and text in msg and "dt_token_logprobs" in msg


def test_calls_without_rows_do_nothing(lib):
    assert call(lib, "dt_linear", linear_args(rows=0, x=0, out=0, weight=0))[0] == 0
    assert call(lib, "dt_qk_norm_rope", rotate_args(n_req=0, q=0, k_out=0))[0] == 0
    assert call(lib, "dt_token_logprobs", logp_args(rows=0, logits=0, logp=0))[0] == 0


def test_mirrors_have_the_headers_sizes(lib, tmp_path):
    import shutil
    import subprocess
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "dtree.h"\nint main(void) { printf("%zu %zu %zu", sizeof(dt_linear_args), '
                   "sizeof(dt_qk_norm_rope_args), sizeof(dt_token_logprobs_args)); return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run([cc, "-I", dtbuild.INCLUDE, str(src), "-o", str(exe)], check=True)
    sizes = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [ctypes.sizeof(c) for c in (ly._Linear, ly._Rotate, ly._Logprobs)]


class Tensor:
    """Stands in for a tensor on cuda:1."""
    is_cuda, device = True, "cuda:1"

    def __init__(self, dtype, *shape, stride=None):
        import torch
        self.dtype, self.shape = dtype, torch.Size(shape)
        self.st = stride or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def stride(self):
        return self.st


def bindings(torch):
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    rotary = ly.Rotary(64, device="cpu")
    rotary.turns = Tensor(torch.int64, 32)
    x, w, out = Tensor(bf16, 3, 64), Tensor(bf16, 48, 64), Tensor(bf16, 3, 48)
    q, k = Tensor(bf16, 3, 4, 64), Tensor(bf16, 3, 2, 64)
    logits = Tensor(f32, 3, 100)
    one = dict(lse=Tensor(f32, 3), entropy=Tensor(f32, 3), logp=Tensor(f32, 3), top_tok=Tensor(i32, 3, 2), top_logp=Tensor(f32, 3, 2))
    return dict(dt_linear=lambda **kw: ly.linear(**{**dict(x=x, weight=w, out=out), **kw}),
                dt_qk_norm_rope=lambda **kw: ly.qk_norm_rope(**{**dict(q=q, k=k, rotary=rotary, q_out=q, k_out=k), **kw}),
                dt_token_logprobs=lambda **kw: ly.token_logprobs(**{**dict(logits=logits, tokens=Tensor(i32, 3), top=2, out=one), **kw}))


class Library:
    calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


def test_every_binding_asks_for_its_device_before_it_launches(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(ly, "_library", Library)
    Library.calls = []
    monkeypatch.setattr(kc, "_current_device", lambda: 0)
    for f in bindings(torch).values():
        with pytest.raises(ValueError, match="cuda:1"):
            f()
    assert Library.calls == []
    monkeypatch.setattr(kc, "_current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    for f in bindings(torch).values():
        f()
    assert Library.calls == ["dt_linear", "dt_qk_norm_rope", "dt_token_logprobs"]


def test_bindings_refuse_tensors_that_do_not_fit(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(ly, "_library", Library)
    monkeypatch.setattr(kc, "_current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    Library.calls = []
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    b = bindings(torch)
    for name, kw in (
            ("dt_linear", dict(x=Tensor(f32, 3, 64))), ("dt_linear", dict(x=Tensor(bf16, 3, 56))), ("dt_linear", dict(weight=Tensor(bf16, 48))),
            ("dt_linear", dict(weight=Tensor(bf16, 48, 64, stride=(64, 2)))), ("dt_linear", dict(gate=Tensor(bf16, 47, 64))),
            ("dt_linear", dict(gate_bias=Tensor(bf16, 47))), ("dt_linear", dict(bias=Tensor(f32, 48))), ("dt_linear", dict(residual=Tensor(bf16, 48))),
            ("dt_linear", dict(activation="swish")), ("dt_linear", dict(out=Tensor(torch.float16, 3, 48))), ("dt_linear", dict(out=Tensor(bf16, 3, 49))),
            ("dt_linear", dict(out_dtype=f32)), ("dt_linear", dict(status=Tensor(i32, 2))),
            ("dt_linear", dict(x=Tensor(bf16, 2, 3, 64, stride=(200, 64, 1)), out=Tensor(bf16, 2, 3, 48))),
            ("dt_qk_norm_rope", dict(q=Tensor(bf16, 4, 64))), ("dt_qk_norm_rope", dict(k=Tensor(bf16, 1, 3, 2, 64))), ("dt_qk_norm_rope", dict(k=None)),
            ("dt_qk_norm_rope", dict(k=Tensor(bf16, 2, 2, 64))), ("dt_qk_norm_rope", dict(positions=Tensor(i32, 4))), ("dt_qk_norm_rope", dict(base=Tensor(i32, 2))),
            ("dt_qk_norm_rope", dict(q_weight=Tensor(bf16, 63))), ("dt_qk_norm_rope", dict(q_out=Tensor(bf16, 3, 4, 63))),
            ("dt_token_logprobs", dict(logits=Tensor(torch.float16, 3, 100))), ("dt_token_logprobs", dict(tokens=Tensor(i32, 2))),
            ("dt_token_logprobs", dict(tokens=Tensor(torch.int64, 3))), ("dt_token_logprobs", dict(logits=Tensor(f32, 3, 100, stride=(1, 3)))),
            ("dt_token_logprobs", dict(top=3)), ("dt_token_logprobs", dict(tokens=Tensor(i32, 3, 1, 1))), ("dt_token_logprobs", dict(status=Tensor(f32, 1)))):
        with pytest.raises((ValueError, TypeError)):
            b[name](**kw)
    assert Library.calls == []


def test_rotary_turns():
    """Units of 2^-64 of a turn: what a position's step is, and what far positions make of it."""
    import math
    from fractions import Fraction
    r = ly.Rotary(8, theta=100.0, device="cpu")
    assert r.turns.tolist()[0] == round(2 ** 64 / Fraction(2 * math.pi)) or abs(r.turns.tolist()[0] / 2 ** 64 - 1 / (2 * math.pi)) < 1e-16
    assert all(abs(t / 2 ** 64 * 2 * math.pi - f) < 1e-15 for t, f in zip(r.turns.tolist(), r.inv_freq))
    half = ly.Rotary(4, inv_freq=[math.pi, -1.0], device="cpu")
    assert abs(abs(half.turns.tolist()[0]) - 2 ** 63) < 2 ** 12 and half.turns.tolist()[1] < 0
    for bad in (dict(dim=7), dict(dim=0), dict(dim=4, inv_freq=[1.0]), dict(dim=4, inv_freq=[1.0, INF])):
        with pytest.raises(ValueError):
            ly.Rotary(device="cpu", **bad)


@pytest.mark.parametrize("kw", [
    dict(out=8192), dict(out=8192 + 3 * 128), dict(out=8192 - 3 * 96), dict(out=65536 + 32, out_row_stride=64), dict(out=65536 + 6144 - 16),
    dict(residual=131072 + 2, residual_row_stride=48), dict(residual=131072, residual_row_stride=56), dict(residual=131072, residual_row_stride=0),
    dict(residual=131072, residual_row_stride=48, out_fp32=1), dict(bias=131072 + 94), dict(rows=1, out=8192 + 126),
    dict(x_row_stride=128, out_row_stride=128, out=8192 + 256 - 64), dict(x_row_stride=128, out_row_stride=128, out=8192 + 126)])
def test_linear_refuses_an_output_over_an_input(lib, kw):
    a = dict(x=8192, weight=65536, out=131072)
    err, msg = call(lib, "dt_linear", linear_args(**{**a, **kw}))
    assert err == INVALID and "overlaps an input" in msg


@pytest.mark.parametrize("kw", [
    dict(q_out=8192 + 512), dict(q_out=8192, q_out_row_stride=264), dict(q_out=16384 + 128, q_out_row_stride=384, k_row_stride=384),
    dict(k_out=8192 + 6 * 512 - 16), dict(k_out=65536 + 64, k_out_row_stride=256), dict(q_out=8192, q_row_stride=384, k=8192 + 512, k_row_stride=384,
                                                                                      q_out_row_stride=384, q_out_head_stride=72)])
def test_qk_norm_rope_refuses_outputs_over_other_tensors(lib, kw):
    a = dict(q=8192, k=16384, q_out=65536, k_out=131072)
    err, msg = call(lib, "dt_qk_norm_rope", rotate_args(**{**a, **kw}))
    assert err == INVALID and "overlaps another tensor" in msg
