"""attn_prefill_paged on its tensor-core kernel (kda_attn_chunk.cu) against the 64-bit statements.

Calls of little work go to the warp-level kernel; the work is bounded by the page table's width, so
a table much wider than the sequences sends small inputs through the tensor-core kernel."""
import math

import pytest
import torch

from kv_attn_util import D, Cache, attention, check
from test_kv_attn_gpu import gen, reference, run_prefill

pytestmark = pytest.mark.gpu

WIDE = 1 << 17  # tokens that the page tables have room for


def wide(page):
    return WIDE // page


@pytest.mark.parametrize("new,past,window,sink", [([900, 60], [0, 400], 20, 0), ([700], [500], 100, 5), ([60] * 12, [3 * i for i in range(12)], 0, 0),
                                                  ([300, 1, 260], [0, 0, 700], 130, 129)])
def test_edge_tiles_in_a_row(new, past, window, sink):
    """Every tile, or nearly every one, has rows that do not see all of it: the look through one edge
    tile's values follows that of the one before directly, within items and from item to item."""
    g = gen(sum(new) + window)
    lens = [a + b for a, b in zip(new, past)]
    c = Cache(lens, 2, 64, False, g, max_pages=wide(64))
    q = torch.randn(sum(new), 6, D, generator=g).to(torch.bfloat16)
    ref = reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5)
    q = q.cuda()
    for _ in range(5):
        o, lse = run_prefill(c, q, new, lens, window, sink)
        check(o, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_items_before_the_first_token(fp8):
    """More new tokens than the cache holds, by several items: their rows see nothing."""
    g = gen(31)
    new, lens = [300, 140], [40, 0]
    c = Cache(lens, 2, 16, fp8, g, max_pages=wide(16))
    q = torch.randn(sum(new), 12, D, generator=g).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens)
    see = torch.arange(40) <= torch.arange(-260, 40)[:, None]
    check(o[:300], lse[:300], attention(q[:300], c.value["k"][0], c.value["v"][0], see, D ** -0.5, fp8))
    assert (o[300:] == 0).all() and torch.isneginf(lse[300:]).all()


@pytest.mark.parametrize("window,sink", [(0, 0), (40, 3)])
@pytest.mark.parametrize("last", [1, 2, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_keys_alone_in_a_tile(fp8, last, window, sink):
    """The only keys of the last tile are NaN: rows that do not see them are as if there were none."""
    g = gen(last)
    new, lens = [100, 256 + last], [128 * 2 + last, 256 + last]

    def values(n, i, x):
        if n == "k":
            x[256:, :, 5] = math.nan
        return x

    c = Cache(lens, 2, 32, fp8, g, values=values, max_pages=wide(32))
    q = torch.randn(sum(new), 8, D, generator=g).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens, window, sink)
    ref = reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5)
    bad = torch.isnan(ref[0]).any(-1)
    assert int(bad.sum()) == 2 * last * 8
    assert torch.isnan(lse[bad.cuda()]).all()
    lse[bad.cuda()] = 0
    ref[1][bad] = 0
    check(o, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_too_small_to_tell_apart(fp8):
    """A scale and queries whose product is below 2^-126: every visible key has the same weight."""
    g = gen(77)
    new, lens = [200], [300]
    c = Cache(lens, 2, 64, fp8, g, max_pages=wide(64))
    q = (torch.randn(200, 8, D, generator=g) * 2.0 ** -100).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens, scale=2.0 ** -120)
    check(o, lse, reference(c, [q], new, lens, 0, 0, 2.0 ** -120))
