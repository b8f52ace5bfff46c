"""The bindings' memory next to streams, captured graphs and devices."""
import numpy as np
import pytest

from tests.test_gpu_kvcache import _t, cache_case, check_cache, check_prompt, dev

pytestmark = pytest.mark.gpu

LATE = 400_000_000  # cycles: some 0.2 s


@pytest.mark.parametrize("slots", [1, 40])
def test_a_call_on_another_stream_does_not_wait_for_the_current_ones_memory(slots):
    """The current stream is busy for a while; a call on another stream has its workspace zeroed and its output written in
    that stream's order, and nothing that the current stream still has to do falls on them."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, cache_attention, prompt_attention
    c = cache_case(np.random.RandomState(81), [3000, 10, 0, 900], slots, 8, 2, 128, 64, "tree")
    table, length, mask = dev(c["table"], torch.int32), dev(c["lens"], torch.int32), dev(c["mask"], torch.uint8)
    lse = torch.zeros(4, slots, 8, device="cuda")
    q, k, v = (torch.randn(300, h, 128, device="cuda").to(torch.bfloat16) for h in (8, 2, 2))
    start = dev([0, 300], torch.int32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory of the outputs' and the workspace's sizes, which the current stream has yet to overwrite when it is free again
    sizes = [c["q"].numel() * 2, q.numel() * 2] + [s << 20 for s in (2, 8, 16, 32, 48, 64)]
    spare = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]

    def call():
        out = cache_attention(c["cache"], c["q"], table, length, k_new=c["k"], v_new=c["v"], mask=mask, lse=lse,
                              workspace=AttentionWorkspace(), stream=side)
        return out, prompt_attention(q, k, v, start, stream=side)
    call()  # (loading kernels and getting memory from the driver wait for the device: done here)
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    for x in spare:
        x.fill_(0xFF)
    del spare, x
    busy = torch.cuda.Event()
    busy.record()
    out, full = call()
    side.synchronize()
    assert not busy.query()  # (the test holds only while the current stream is still busy)
    with torch.cuda.stream(side):
        out_then, full_then = out.clone(), full.clone()
    torch.cuda.synchronize()
    assert torch.equal(out, out_then) and torch.equal(full, full_then)
    check_cache(c, (out.float().cpu().numpy(), lse.cpu().numpy()))
    full_lse = torch.zeros(300, 8, device="cuda")
    assert torch.equal(full, prompt_attention(q, k, v, start, lse=full_lse))
    check_prompt(q, k, v, [300], (full.float().cpu().numpy(), full_lse.cpu().numpy()), sample=[0, 150, 299])


def test_a_workspace_outlives_the_streams_that_use_it():
    """Dropped while another stream still works in it, its memory is not given out again before that work is done."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, cache_attention
    c = cache_case(np.random.RandomState(82), [3000, 900], 1, 8, 2, 128, 64, None)
    table, length = dev(c["table"], torch.int32), dev(c["lens"], torch.int32)
    side = torch.cuda.Stream()
    work = AttentionWorkspace()
    first = cache_attention(c["cache"], c["q"], table, length, workspace=work)
    torch.cuda.synchronize()
    at = work.buffer.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    out = cache_attention(c["cache"], c["q"], table, length, workspace=work, stream=side)
    n = work.buffer.numel()
    del work
    again = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [x.data_ptr() for x in again]
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_captured_calls_keep_their_workspace_when_it_grows():
    """A single-token step is captured, then larger calls grow the workspace; the graph's memory is still there, and its
    replays give what the call gave.  A call that needs more inside a capture has the graph's own memory."""
    torch = _t()
    from conditional_draft_tree_lm_gb300 import AttentionWorkspace, cache_attention
    work = AttentionWorkspace()
    c = cache_case(np.random.RandomState(83), [3000, 900, 0], 1, 8, 2, 128, 64, "tree")
    d = cache_case(np.random.RandomState(84), [500, 40], 70, 8, 2, 128, 64, "tree")
    args = [(x["cache"], x["q"], dev(x["table"], torch.int32), dev(x["lens"], torch.int32)) for x in (c, d)]
    new = [dict(k_new=x["k"], v_new=x["v"], mask=dev(x["mask"], torch.uint8), workspace=work) for x in (c, d)]
    want = cache_attention(*args[0], **new[0])
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache_attention(*args[0], out=out, **new[0])
    small = work.buffer
    at, size = small.data_ptr(), small.numel()
    del small
    inside, twice, third = torch.cuda.CUDAGraph(), torch.zeros_like(d["q"]), torch.zeros_like(d["q"])
    with torch.cuda.graph(inside):
        cache_attention(*args[1], out=twice, **new[1])
        cache_attention(*args[0], out=out, **new[0])
        cache_attention(*args[1], out=third, **new[1])
    assert work.buffer.data_ptr() == at
    fresh = torch.cuda.CUDAGraph()
    with torch.cuda.graph(fresh):
        cache_attention(*args[0], out=out, **dict(new[0], workspace=AttentionWorkspace()))
    torch.cuda.synchronize()
    assert torch.equal(cache_attention(*args[0], **new[0]), want)  # (before any replay)
    large = cache_attention(*args[1], **new[1])
    for _ in range(3):
        for x in (out, twice, third):
            x.fill_(7)
        inside.replay()
        assert torch.equal(twice, large) and torch.equal(third, large) and torch.equal(out, want)
        out.fill_(7)
        fresh.replay()
        assert torch.equal(out, want)
    assert work.buffer.data_ptr() != at and work.buffer.numel() >= 2 * size
    other = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in [x.data_ptr() for x in other]
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(large, cache_attention(*args[1], **new[1]))
    torch.cuda.synchronize()
    assert all((x == 0xFF).all() for x in other)
    # grown, it is captured too
    out = torch.zeros_like(large)
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        cache_attention(*args[1], out=out, **new[1])
    second.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, large)
    check_cache(d, (large.float().cpu().numpy(), None), rows=[0, 30, 69])
