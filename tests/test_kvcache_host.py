"""The cache's bindings on the host: what they refuse before anything is launched (CPU, no GPU call)."""
import pytest

from conditional_draft_tree_lm_gb300 import kvcache as kc


class _Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    monkeypatch.setattr(kc, "_current_device", lambda: 0)
    assert kc._stream(_Stream(0), 0) == 77
    for stream, index in ((None, 1), (_Stream(1), 1), (_Stream(1), 0)):
        with pytest.raises(ValueError, match="cuda:1"):
            kc._stream(stream, index)


def test_every_binding_asks_for_its_stream_before_it_launches(monkeypatch):
    """With a stand-in for the library and for tensors on cuda:1: the call is refused and never made."""
    torch = pytest.importorskip("torch")

    class Tensor:
        is_cuda = True

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

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

        def stride(self, i=None):
            st = torch.empty(self.shape, device="meta").stride()
            return st if i is None else st[i]

    class Work:
        sizes = None

        def reserve(self, *sizes):
            return Tensor(torch.uint8, 1 << 20)

    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(kc, "_library", Library)
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    cache = kc.KvCache(*(Tensor(torch.float8_e4m3fn, 4, 2, 16, 64) for _ in range(2)), *(Tensor(f32, 4, 2) for _ in range(2)))
    rows, one = Tensor(torch.int64, 3), Tensor(i32, 1)
    k = Tensor(bf16, 3, 2, 64)

    def all_calls():
        yield lambda: kc.kv_plan(one, one, Tensor(i32, 1, 2), Tensor(i32, 4), Tensor(i32, 2), Tensor(i32, 2), Tensor(i32, 2), rows, one, page=16)
        yield lambda: kc.kv_append(cache, k, k, rows)
        yield lambda: kc.cache_attention(cache, Tensor(bf16, 1, 3, 2, 64), Tensor(i32, 1, 2), one, out=Tensor(bf16, 1, 3, 2, 64), workspace=Work())
        yield lambda: kc.prompt_attention(k, k, k, Tensor(i32, 2), out=Tensor(bf16, 3, 2, 64))

    monkeypatch.setattr(kc, "_current_device", lambda: 0)
    for call in all_calls():
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert calls == []
    # on the current device the same arguments reach the library
    monkeypatch.setattr(kc, "_current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    for call in all_calls():
        call()
    assert calls == ["dt_kv_plan", "dt_kv_append", "dt_cache_attention", "dt_prompt_attention"]


def test_sizes_that_32_bit_counts_would_pass_are_refused():
    """Lengths and rows up to 2^31-4097 may be asked for; behind that a count some tiles ahead would turn negative."""
    import ctypes
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    dtbuild.build_library()
    lib = kc._library()

    def refused(**kw):
        c = kc._Cache(256, 256, 256, 256, 4, kw.pop("page", 128), 1, 128)
        a = kc._Attend(n_req=1, slots=1, n_q=1, max_blocks=1, scale=1.0, q=256, block_table=256, length=256, out=256, out_row_stride=128,
                       workspace=256, workspace_bytes=0)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.dt_cache_attention(ctypes.byref(c), ctypes.byref(a), None), lib.dt_last_error().decode()

    # (the workspace of no bytes refuses what the sizes let through, before any CUDA call)
    for kw, msg in ((dict(max_blocks=2 ** 24 - 32), "workspace"), (dict(max_blocks=2 ** 24 - 31), "2^31-4096"),
                    (dict(max_blocks=2 ** 27 - 1, page=16), "2^31-4096"), (dict(max_blocks=2 ** 27 - 256, page=16), "workspace"),
                    (dict(slots=2 ** 31 - 4096), "workspace"), (dict(slots=2 ** 31 - 4095), "2^31-4096"),
                    (dict(slots=2 ** 30, n_req=2), "2^31-4096")):
        err, text = refused(**kw)
        assert err != 0 and msg in text, (kw, text)
    assert lib.dt_cache_attention_workspace(1, 2 ** 31 - 1, 1, 1, 128) == 0


@pytest.mark.parametrize("row,head,overlaps", [(0, 128, True), (512, 0, True), (512, 64, True), (504, 128, True), (128, 128, True),
                                               (512, 128, False), (640, 128, False), (128, 768, False), (128, 640, True), (1024, 256, False)])
def test_outputs_whose_rows_overlap_are_refused(row, head, overlaps):
    """Six rows of four heads of 128, by their strides; what passes is refused for its workspace of no bytes."""
    import ctypes
    from conditional_draft_tree_lm_gb300 import build as dtbuild
    dtbuild.build_library()
    lib = kc._library()
    c = kc._Cache(256, 256, 256, 256, 4, 64, 2, 128)
    a = kc._Attend(n_req=2, slots=3, n_q=4, max_blocks=1, scale=1.0, q=256, block_table=256, length=256, out=256, out_row_stride=row,
                   out_head_stride=head, workspace=256, workspace_bytes=0)
    assert lib.dt_cache_attention(ctypes.byref(c), ctypes.byref(a), None) != 0
    assert (b"overlap" in lib.dt_last_error()) == overlaps
    p = kc._Prompt(n_seq=1, n_q=4, n_kv=2, head_dim=128, n_rows=6, scale=1.0, q=256, k=256, v=256, out=256, out_row_stride=row,
                   out_head_stride=head, row_start=256)
    if overlaps:
        assert lib.dt_prompt_attention(ctypes.byref(p), None) != 0 and b"overlap" in lib.dt_last_error()
