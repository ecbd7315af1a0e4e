"""Waits of linear attention's prefill that run out (test_kv_attn_failure_gpu.py for the attention cache): the test
hook leaves out a copy, every warp gives up in order, the host reads KDA_ERR_TIMEOUT, and the next call gives the bits
that it gave before."""
import time

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from test_lin_gpu import Prefill

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.mark.parametrize("segments,copy", [(1, 0), (1, 1), (1, 2), (1, 7), (2, 1)])
def test_missing_copy_times_out_and_the_context_survives(segments, copy):
    p = Prefill([700, 600], 2, 1, seed=1)
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
    assert int(st) == TIMEOUT
    assert took < 60, took
    st.zero_()
    got = call()
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
