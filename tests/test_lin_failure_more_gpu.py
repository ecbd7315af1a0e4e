"""Waits that run out in the instance with the output stage, whose gate has a warp and copies of its own, and where blocks
take one item after another (test_lin_failure_gpu.py for the other instances)."""
import time

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from test_lin_gpu import Prefill

pytestmark = pytest.mark.gpu
TIMEOUT = 6


def give_up(p, copy, segments=0):
    a, b = p.args()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: kda.lin_prefill(*a, **b, n_segments=segments, dev_status=st)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    assert int(st) == 0
    kda.debug_stall_next_linear(copy)
    begin = time.monotonic()
    call()
    torch.cuda.synchronize()
    took = time.monotonic() - begin
    assert int(st) == TIMEOUT and took < 60, (int(st), took)
    st.zero_()
    got = call()
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("segments,copy", [(1, 0), (1, 1), (1, 8), (2, 2)])
def test_output_stage(segments, copy):
    give_up(Prefill([700, 600], 2, 1, seed=1, gated=True), copy, segments)


# Three items of 3, 2 and 3 chunks for each of 64 heads: some blocks have one, the others two.  A chunk has three copies:
# number 1 is in every block's first item, number 10 in some blocks' second.
@pytest.mark.parametrize("gated,copy", [(False, 10), (True, 1), (True, 10)])
def test_blocks_with_several_items(gated, copy):
    p = Prefill([300, 200, 260], 64, 8, seed=2, gated=gated)
    assert kda.lin_prefill_workspace_size(3, 64, 760) > 0
    give_up(p, copy)
