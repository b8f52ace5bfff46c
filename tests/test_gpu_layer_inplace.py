"""qk_norm_rope over its own inputs where the heads of a row are shared by several CTAs, whose shares are not whole warps.

In place a head that two CTAs take is normed and turned twice; with outputs of their own the same call writes it twice alike.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,dim", [(64, 4, 128), (128, 8, 128), (64, 2, 128), (32, 1, 256), (128, 1, 64), (63, 3, 112), (255, 7, 32)])
@pytest.mark.parametrize("rows", [3, 2080])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_in_place_is_that_into_new_tensors(heads, kv, dim, rows, interleaved):
    import torch
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(heads + dim)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    qkv, qw, kw = normal(rows, heads + 2 * kv, dim), normal(dim), normal(dim)
    rot = dim // 32 * 16  # (some channels stay)
    pos = torch.as_tensor(np.random.RandomState(rows).randint(0, 100000, rows), dtype=torch.int32, device="cuda")
    args = dict(positions=pos, rotary=Rotary(rot, interleaved=interleaved), q_weight=qw, k_weight=kw)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
    want_q, want_k = qk_norm_rope(q, k, **args)
    for _ in range(3):
        mine = qkv.clone()
        a, b = mine[:, :heads], mine[:, heads:heads + kv]
        qk_norm_rope(a, b, q_out=a, k_out=b, **args)
        assert torch.equal(a, want_q) and torch.equal(b, want_k) and torch.equal(mine[:, heads + kv:], qkv[:, heads + kv:])
