"""More of what the layer's calls refuse on the host (CPU, no GPU call): outputs over what a call reads besides q, k and logits."""
import pytest

from tests.test_layer_host import INVALID, call, lib, linear_args, logp_args, rotate_args  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(turns=65536), dict(turns=65536 + 8), dict(turns=65536 - 248), dict(positions=131072 + 4), dict(positions=131072 - 20), dict(base=65536 + 3068),
    dict(base=65536 - 4), dict(q_weight=131072 + 16), dict(k_weight=65536 - 112), dict(positions=8192, q_out=8192), dict(k_weight=16384 + 16, k_out=16384)])
def test_qk_norm_rope_refuses_outputs_over_what_else_it_reads(lib, kw):  # noqa: F811
    a = dict(q=8192, k=16384, turns=32768, q_out=65536, k_out=131072)
    err, msg = call(lib, "dt_qk_norm_rope", rotate_args(**{**a, **kw}))
    assert err == INVALID and "overlaps another tensor" in msg


OUTPUTS = dict(logp=65536, lse=66048, entropy=66560, top_tok=67072, top_logp=67584)


@pytest.mark.parametrize("kw", [
    dict(lse=8192), dict(entropy=8192 + 796), dict(logp=8192 - 4), dict(top_tok=8192 + 400), dict(top_logp=8192 + 784), dict(logp=32768), dict(lse=32768 + 4),
    dict(lse=66560), dict(entropy=66048 + 4), dict(top_tok=65536), dict(top_logp=67072 + 12), dict(status=66048), dict(status=8192 + 4),
    dict(logits_row_stride=200, lse=8192 + 396), dict(logits_row_stride=0, entropy=8192 + 4)])
def test_token_logprobs_refuses_outputs_over_its_inputs_or_one_another(lib, kw):  # noqa: F811
    err, msg = call(lib, "dt_token_logprobs", logp_args(**{**dict(logits=8192, tokens=32768), **OUTPUTS, **kw}))
    assert err == INVALID and "overlaps" in msg


@pytest.mark.parametrize("name,kw", [
    ("dt_linear", dict(status=131072 + 2)), ("dt_qk_norm_rope", dict(positions=32770)), ("dt_qk_norm_rope", dict(base=32769)),
    ("dt_token_logprobs", dict(tokens=32770)), ("dt_token_logprobs", dict(logp=65538)), ("dt_token_logprobs", dict(lse=66050)),
    ("dt_token_logprobs", dict(entropy=66561)), ("dt_token_logprobs", dict(top_tok=67073)), ("dt_token_logprobs", dict(top_logp=67586)),
    ("dt_token_logprobs", dict(status=131074))])
def test_addresses_that_are_not_aligned_to_their_elements_are_refused(lib, name, kw):  # noqa: F811
    args = dict(dt_linear=lambda: linear_args(**{**dict(x=8192, weight=16384, out=65536), **kw}),
                dt_qk_norm_rope=lambda: rotate_args(**{**dict(q=8192, k=16384, turns=24576, q_out=65536, k_out=98304), **kw}),
                dt_token_logprobs=lambda: logp_args(**{**dict(logits=8192, tokens=32768), **OUTPUTS, **kw}))[name]()
    err, msg = call(lib, name, args)
    assert err == INVALID and "misaligned" in msg and name in msg


def test_linear_refuses_an_output_over_its_status(lib):  # noqa: F811
    err, msg = call(lib, "dt_linear", linear_args(x=8192, weight=16384, out=65536, status=65536 + 16))
    assert err == INVALID and "overlaps" in msg
