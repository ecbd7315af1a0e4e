"""attn_prefill_paged on its tensor-core kernel (kda_attn_chunk.cu) against the 64-bit statements.

Calls of little work go to the warp-level kernel; the work is bounded by the page table's width, so
a table much wider than the sequences sends small inputs through the tensor-core kernel."""
import pytest
import torch

from kv_attn_util import D, Cache, check
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
