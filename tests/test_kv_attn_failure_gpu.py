"""Waits of the attention cache's kernels that run out (test_failure_gpu.py for the prefill).

The test hook kda_debug_stall_next_attention makes each block leave out one copy of its keys.  The
waits for it run out, lanes of a warp and warps that meet at barriers deciding together; everybody
leaves, copies and products in flight land, and the host reads KDA_ERR_TIMEOUT from dev_status.
The context stays usable: the next call gives the bits that it gave before."""
import time

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kv_attn_util import D, Cache
from test_kv_attn_gpu import gen, i32, offsets

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kernel,copy", [("decode", 0), ("decode, many rows", 1), ("few rows", 0), ("many rows", 0), ("many rows", 1)])
def test_missing_copy_times_out_and_the_context_survives(kernel, fp8, copy):
    g = gen(7)
    lens, new = [3000, 2500], [200, 31]
    c = Cache(lens, 2, 64, fp8, g, max_pages=2048 if kernel == "many rows" else None)
    rows = {"decode": 4, "decode, many rows": 48}.get(kernel, 12)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kernel.startswith("decode"):
        q = torch.randn(2, 1, rows * 2, D, generator=g).to(torch.bfloat16).cuda()
        call = lambda: kda.attn_decode_paged(q, *c.args, i32(*lens), **c.scales, dev_status=st)
    else:
        if kernel == "few rows":
            new = [5, 3]
        q = torch.randn(sum(new), rows, D, generator=g).to(torch.bfloat16).cuda()
        call = lambda: kda.attn_prefill_paged(q, *c.args, offsets(new), i32(*lens), **c.scales, dev_status=st)
    want = call()
    torch.cuda.synchronize()
    assert int(st) == 0
    kda.debug_stall_next_attention(copy)
    begin = time.monotonic()
    call()
    torch.cuda.synchronize()
    took = time.monotonic() - begin
    assert int(st) == TIMEOUT
    assert took < 60, took
    st.zero_()
    assert torch.equal(call(), want)
    torch.cuda.synchronize()
    assert int(st) == 0
