"""More of what the layer's calls refuse on the host (CPU, no GPU call): outputs over what a call reads besides q, k and logits."""
import pytest

from tests.test_layer_host import INVALID, call, lib, logp_args, rotate_args  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(turns=65536), dict(turns=65536 + 8), dict(turns=65536 - 248), dict(positions=131072 + 4), dict(positions=131072 - 20), dict(base=65536 + 3068),
    dict(base=65536 - 4), dict(q_weight=131072 + 16), dict(k_weight=65536 - 112), dict(positions=8192, q_out=8192), dict(k_weight=16384 + 16, k_out=16384)])
def test_qk_norm_rope_refuses_outputs_over_what_else_it_reads(lib, kw):  # noqa: F811
    a = dict(q=8192, k=16384, turns=32768, q_out=65536, k_out=131072)
    err, msg = call(lib, "dt_qk_norm_rope", rotate_args(**{**a, **kw}))
    assert err == INVALID and "overlaps another tensor" in msg
