"""The wide paged attention kernel's failure path: a bounded wait that runs out.

As in test_gpu_timeout.py: a wait bound of 2 ns (GraftAttnTuning.wait_ns) makes the first waits run out on small, valid
inputs; every load stays in bounds and completes.  The call returns with the TIMEOUT bit set, and the next normal call
on the same stream, with its workspace zeroed anew, is right: the CTAs waited for what they had in flight and freed
their tensor memory.
"""
import pytest
import torch

from tests.helpers import gb
from tests.test_gpu_paged import DEV, Setup, check_attention, run_attention, tree_masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree,Hkv,G,page,new,lens", [
    (True, 8, 4, 16, [64], [4096]),                          # one item, split by keys, single tiles
    (False, 8, 4, 16, [9], [20]),                            # one block a CTA: the producer ends without any wait
    (False, 2, 16, 64, [64] * 3, [1500, 300, 129]),          # pairs
    (True, 8, 4, 32, [20, 40, 20, 64, 9, 30] * 4, [700, 650, 130, 600, 64, 0] * 4),  # several items a CTA, both kinds
    (False, 2, 8, 128, [200, 1, 1, 1], [5, 900, 300, 0]),    # few rows beside the wide ones
])
def test_bounded_wait_runs_out_and_the_device_stays_usable(dtype, tree, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=len(new) + G)
    mask = tree_masks(s.rng, new) if tree else None
    md = torch.from_numpy(mask.view("int64")).to(DEV) if tree else None
    N = int(s.starts[-1])
    Q = s.randn(N, Hkv * G, 128).to(DEV)
    for _ in range(3):
        s.cache.plan(s.q_start, N, Hkv * G, max(new), tree=tree)
        s.cache.attend(0, Q, 0.09, mask=md, tuning=dict(wait_ns=2))
        torch.cuda.synchronize()
        assert s.status() == gb().STATUS_TIMEOUT
        s.cache._buffers["attention"].zero_()
        Q2, O = run_attention(s, G, mask=mask)
        check_attention(s, O, Q2, 0.09, mask)


def test_a_bound_that_is_long_enough_changes_nothing():
    s = Setup([700, 20], [64, 40], 2, 16, seed=3)
    Q = s.randn(104, 16, 128).to(DEV)
    s.cache.plan(s.q_start, 104, 16, 64)
    a = s.cache.attend(0, Q, 0.09)
    b = s.cache.attend(0, Q, 0.09, tuning=dict(wait_ns=400000000))
    assert s.status() == 0 and torch.equal(a, b)
