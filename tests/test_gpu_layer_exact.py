"""linear over small whole numbers, whose products and sums have no rounding but the last: every bit of the outputs is known.

Operands are -1, 0 and 1, so that sums stay below 2^24 by far (they are at most inner, and their products at most inner^2, near
200 and 2^16 as they fall) and fp32 holds every partial sum in whatever order; a channel that is lost, read twice or taken from another
row shows in half of the outputs, at any inner dimension.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,inner,outer", [
    (1, 8192, 300), (1, 2560, 6144), (2, 10248, 70), (2, 1032, 5000), (3, 8200, 130), (20, 10240, 2560), (65, 4096, 2560), (40, 2568, 20000),
    (100, 2560, 12000), (200, 2560, 6144), (256, 8192, 200), (300, 8192, 520), (513, 1032, 777), (700, 2568, 9600), (1024, 2560, 2990), (2080, 4096, 2560),
    (5000, 576, 513)])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("full", [False, True])
def test_linear_of_whole_numbers_is_exact(rows, inner, outer, gate, full):
    import torch
    from conditional_draft_tree_lm_gb300 import linear
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(rows + inner)

    def whole(*shape, most=1):
        return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)
    x, w, bias, res = whole(rows, inner), whole(outer, inner), whole(outer, most=9), whole(rows, outer, most=100)
    y = x.double() @ w.double().T + bias.double()
    if gate:
        g, gate_bias = whole(outer, inner), whole(outer, most=9)
        want = y * (x.double() @ g.double().T + gate_bias.double()).clamp(min=0) + res.double()
        kw = dict(gate=g, gate_bias=gate_bias)
    else:
        want, kw = y.clamp(min=0) + res.double(), {}
    assert want.abs().max() < 2 ** 24
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dtype = torch.float32 if full else torch.bfloat16
    out = linear(x, w, bias=bias, activation="relu", residual=res, out_dtype=dtype, status=status, **kw)
    assert torch.equal(out, want.to(dtype)) and status.item() == 0
