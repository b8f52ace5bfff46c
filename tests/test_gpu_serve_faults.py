"""examples/serve_tree.py keeps what any of its calls has reported."""
import os
import sys

import pytest

from oracle import kvcache as ok

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_a_fault_stays_noted_when_later_plans_go_well():
    import torch
    from serve_tree import Server, TargetLayer
    from workloads import get_config
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    cfg = get_config("tiny_bf16", n_req=2)
    server = Server(cfg, TargetLayer(cfg.V, cfg.d, 4, 2, 64, gen), max_tokens=40)
    grow = lambda *d: torch.tensor(d, dtype=torch.int32, device="cuda")  # noqa: E731
    server.plan(64, delta=grow(3, 60))  # the second is longer than its table
    assert server.length[0].tolist() == [0, 0]
    server.plan(64, delta=grow(3, 4))
    assert server.length[0].tolist() == [3, 4]
    assert server.status.item() == ok.BAD_LENGTH
