"""qk_norm_rope of heads whose squares leave fp32, above and below: the norm does not depend on a head's unit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale,eps", [(1e19, 1e-6), (1e25, 1e-6), (3e37, 1e-6), (3e37, 0.0), (1e-20, 0.0), (1e-25, 0.0), (1e-38, 0.0), (1e-25, 1e-6), (1e-20, 1e-40),
                                       (1e-13, 1e-27)])
@pytest.mark.parametrize("dim,rows", [(128, 40), (256, 3), (32, 700), (96, 9)])
def test_norms_of_heads_far_from_one(scale, eps, dim, rows):
    """Against the definition in 64 bits, with the tolerance of heads near 1 (scaling by a power of two has no rounding)."""
    from tests.test_gpu_layer import bf16, check_rotated
    import torch
    torch.cuda.set_device(0)
    from conditional_draft_tree_lm_gb300 import Rotary, qk_norm_rope
    rs = np.random.RandomState(dim)
    eps = float(np.float32(eps))
    q, k, qw, kw = bf16(rs, rows, 6, dim), bf16(rs, rows, 2, dim), bf16(rs, dim), bf16(rs, dim)
    rotary, pos = Rotary(32, theta=1e4), rs.randint(0, 100000, rows)
    args = dict(positions=torch.as_tensor(pos, dtype=torch.int32, device="cuda"), rotary=rotary, q_weight=qw, k_weight=kw, eps=eps)
    clean_q, clean_k = qk_norm_rope(q, k, **args)
    near_q, near_k = q.clone(), k.clone()
    q[:, 1::2] = bf16(rs, rows, 3, dim, scale=scale)
    k[:, 1] = bf16(rs, rows, dim, scale=scale)
    q[0, 3, :dim - 3] = 0  # (a few channels of a head)
    out_q, out_k = qk_norm_rope(q, k, **args)
    check_rotated(out_q, q, pos, rotary, qw, eps)
    check_rotated(out_k, k, pos, rotary, kw, eps)
    assert torch.equal(out_q[:, ::2], clean_q[:, ::2]) and torch.equal(out_k[:, 0], clean_k[:, 0])
    check_rotated(clean_q, near_q, pos, rotary, qw, eps)
    check_rotated(clean_k, near_k, pos, rotary, kw, eps)


def test_a_head_of_zeros_without_eps_is_nan_and_an_infinite_one_too():
    """As the formula says: 0 / 0, and inf / inf."""
    import torch
    torch.cuda.set_device(0)
    from conditional_draft_tree_lm_gb300 import qk_norm_rope
    q = torch.ones(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1], q[1, 2, 5] = 0, float("inf")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out, _ = qk_norm_rope(q, q_weight=w, eps=0.0)
    assert out[0, 1].isnan().all() and out[1, 2, 5].isnan() and (out[1, 2].nan_to_num() == 0).all()
    assert (out[0, 0] == 1).all() and (out[0, 2] == 1).all() and (out[1, :2] == 1).all()
