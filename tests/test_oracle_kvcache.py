"""Pins of the key/value cache oracle (CPU) and the refusals of its entry points that need no GPU."""
import ctypes

import numpy as np
import pytest

from oracle import kvcache as ok


def test_round_e4m3_against_every_code():
    """The 126 positive values are fixed points; midpoints go to the even code."""
    codes = np.arange(0, 0x7F)
    vals = np.where(codes < 8, codes * 2.0 ** -9, (1 + (codes & 7) / 8) * 2.0 ** ((codes >> 3) - 7.0))
    assert vals[-1] == 448
    np.testing.assert_array_equal(ok.round_e4m3(vals), vals)
    np.testing.assert_array_equal(ok.round_e4m3(-vals), -vals)
    mid = (vals[1:] + vals[:-1]) / 2
    even = np.where(codes[:-1] % 2 == 0, vals[:-1], vals[1:])
    np.testing.assert_array_equal(ok.round_e4m3(mid), even)
    np.testing.assert_array_equal(ok.round_e4m3(mid * (1 + 1e-12)), vals[1:])


def test_round_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    x = np.random.RandomState(0).uniform(-448, 448, 4000).astype(np.float32) * np.exp2(np.arange(4000) % 20 - 19.0).astype(np.float32)
    np.testing.assert_array_equal(torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy(), ok.round_e4m3(x))


@pytest.mark.parametrize("amax,s", [(448.0, 1.0), (448.0000001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                    (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -126), (1e-45, 2.0 ** -126), (3.3e38, 2.0 ** 120)])
def test_pow2_scale(amax, s):
    assert ok.pow2_scale(amax) == s


def test_plan_by_hand():
    """Two requests of a page of 16: one goes from 15 to 18 tokens, one ends and gives two pages back."""
    table = np.array([[7, -1, -1], [3, 5, -1]])
    ring = np.array([9, 8, 1, 0, 2, 4, 6, -1, -1, -1])
    r = ok.plan([15, 20], [3, -20], 0, table, ring, 1, 6, 16, 5)
    assert r["status"] == 0 and r["len"] == [18, 0] and r["row_start"] == [0, 3, 3]
    assert r["table"].tolist() == [[7, 8, -1], [3, 5, -1]]
    assert r["slot"].tolist() == [7 * 16 + 15, 8 * 16, 8 * 16 + 1, -1, -1] and r["pos"].tolist() == [15, 16, 17, -1, -1]
    assert (r["head"], r["count"]) == (2, 7) and r["ring"].tolist() == [9, 8, 1, 0, 2, 4, 6, 3, 5, -1]


def test_rounding_units_of_the_attention_bounds():
    """The largest relative rounding error of bf16 is 2^-8 / (1 + 2^-8), of fp16 2^-11 / (1 + 2^-11)."""
    torch = pytest.importorskip("torch")
    x = 1 + torch.arange(1 << 16, dtype=torch.float64) / (1 << 16)
    for dtype, unit in ((torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)):
        worst = ((x.to(dtype).double() - x).abs() / x).max().item()
        assert 0.99 * unit / (1 + unit) < worst <= unit


def test_attend_against_brute_force():
    rs = np.random.RandomState(1)
    q, k, v = rs.randn(3, 8), rs.randn(5, 8), rs.randn(5, 8)
    see = np.array([[1, 1, 0, 1, 0], [0, 0, 0, 0, 0], [0, 0, 0, 0, 1]], bool)
    out, lse, _, _ = ok.attend(q, k, v, see, 0.5, 2.0 ** -8)
    w = [np.exp(0.5 * q[0] @ k[t]) for t in (0, 1, 3)]
    np.testing.assert_allclose(out[0], sum(a * v[t] for a, t in zip(w, (0, 1, 3))) / sum(w), rtol=1e-12)
    np.testing.assert_allclose(lse[0], np.log(sum(w)), rtol=1e-12)
    assert (out[1] == 0).all() and lse[1] == -np.inf
    np.testing.assert_allclose(out[2], v[4])


def test_null_arguments_are_refused():
    """Refused before any CUDA call, with a message."""
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    dtbuild.build_library()
    from conditional_draft_tree_lm_gb300 import kvcache as kc
    lib = kc._library()
    assert lib.dt_kv_plan(None, None) == 1 and b"dt_kv_plan" in lib.dt_last_error()
    assert lib.dt_kv_append(None, None, None) == 1
    assert lib.dt_cache_attention(None, None, None) == 1
    assert lib.dt_prompt_attention(None, None) == 1
    c = kc._Cache(16, 16, 16, 16, 4, 48, 2, 128)
    assert lib.dt_kv_append(ctypes.byref(c), ctypes.byref(kc._Append()), None) == 2 and b"page 48" in lib.dt_last_error()
    c = kc._Cache(16, 16, 16, 16, 4, 64, 2, 96)
    assert lib.dt_kv_append(ctypes.byref(c), ctypes.byref(kc._Append()), None) == 2 and b"head_dim 96" in lib.dt_last_error()
    c = kc._Cache(16, 24, 16, 16, 4, 64, 2, 128)
    assert lib.dt_kv_append(ctypes.byref(c), ctypes.byref(kc._Append()), None) == 1 and b"aligned" in lib.dt_last_error()
    assert lib.dt_cache_attention_workspace(1, 1, 6, 4, 128) == 0   # 6 heads over 4
    assert lib.dt_cache_attention_workspace(1, 1, 8, 4, 80) == 0
    assert lib.dt_cache_attention_workspace(3, 65, 32, 8, 128) > 0


def test_struct_sizes_match_the_header(tmp_path):
    """The ctypes mirrors have the C structs' sizes."""
    import shutil
    import subprocess
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    from conditional_draft_tree_lm_gb300 import kvcache as kc
    if not shutil.which("gcc"):
        pytest.skip("no C compiler")
    names = ["dt_kv_cache", "dt_kv_plan_args", "dt_kv_append_args", "dt_cache_attention_args", "dt_prompt_attention_args"]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "dtree.h"\nint main(void){' +
                   "".join(f'printf("%zu ", sizeof({n}));' for n in names) + "return 0;}\n")
    subprocess.run(["gcc", "-I", dtbuild.INCLUDE, str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(s) for s in (kc._Cache, kc._Plan, kc._Append, kc._Attend, kc._Prompt)]
