"""The layer that README.md shows runs as it stands there, and ends in accept_walk's input."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu


def test_the_layer_of_the_readme_runs():
    import torch
    torch.cuda.set_device(0)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        shown = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "qk_norm_rope(" in b]
    assert len(shown) == 1
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)
    requests, slots, d, ffn, vocab = 3, 17, 256, 520, 1000
    depth = torch.arange(slots, dtype=torch.int32, device="cuda").expand(requests, slots).contiguous()
    names = dict(torch=torch, x=normal(requests, slots, d), w_in=normal(d), w_post=normal(d), w_last=normal(d), w_qkv=normal(48 * 128, d, scale=d ** -0.5),
                 b_qkv=normal(48 * 128), w_qn=normal(128), w_kn=normal(128), tree=dict(depth=depth),
                 len_new=torch.full((requests,), 40, dtype=torch.int32, device="cuda"), attended=normal(requests, slots, 32, 128),
                 w_out=normal(d, 32 * 128, scale=1 / 64), w_up=normal(ffn, d, scale=d ** -0.5), w_gate=normal(ffn, d, scale=d ** -0.5),
                 w_down=normal(d, ffn, scale=ffn ** -0.5), head=normal(vocab, d, scale=d ** -0.5),
                 tokens=torch.randint(0, vocab, (requests, slots), generator=gen, device="cuda", dtype=torch.int32))
    stream = names["x"].clone()
    exec(shown[0], names)
    assert names["q"].shape == (requests, slots, 32, 128) and names["k"].shape == names["v"].shape == (requests, slots, 8, 128)
    logits, found = names["logits"], names["found"]
    assert logits.shape == (requests, slots, vocab) and logits.dtype is torch.float32 and logits.isfinite().all()
    assert (found["top_logp"][..., 0] <= 0).all() and torch.equal(found["top_tok"][..., 0].long(), logits.argmax(-1))
    assert not torch.equal(names["x"], stream)
