"""A CTA of a cluster whose wait gives up tells the others behind the cluster's barrier (dt_linear's clusters then write nothing of the
tile): an mbarrier phase that nothing completes, in a wait of its own with the wait limit, recorded by another CTA of the cluster."""
import time

import pytest

from tests.parity import check_round, to_np, upload_round, upload_weights
from workloads import get_config, make_round_inputs, make_weights

pytestmark = pytest.mark.gpu

DT_ERR_TIMEOUT = 5


def test_the_cluster_learns_of_a_wait_that_gave_up():
    import torch
    from conditional_draft_tree_lm_gb300 import DraftTreeBuilder
    from oracle.dartree import Oracle
    torch.cuda.set_device(0)
    cfg = get_config("tiny_bf16")
    w = make_weights(cfg)
    b = DraftTreeBuilder(cfg, upload_weights(w))
    assert b.device_status() == 0
    began = time.time()
    b.check_bounded_waits(2)
    assert b.device_status() == DT_ERR_TIMEOUT and 1.0 < time.time() - began < 30.0
    H, root = make_round_inputs(cfg, 3)
    out = to_np(b.build_round(*upload_round(H, root)))
    assert all(st != "MISMATCH" for st, _ in check_round(Oracle(w, cfg), out, H, root))
    assert b.device_status() == 0
    b.close()
