"""The step between blocks over many rows: every row of h and x' against the 64-bit statement, in outputs that held NaN."""
import pytest
import torch

from lin_util import U16, U32, block, check
from test_block_norm_gpu import BF, make, run

pytestmark = pytest.mark.gpu


def every_row(T, W, wide, parts):
    a = make(T, W, wide, T + W, parts)
    nan = lambda dtype: torch.full((T, W), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    out = dict(h=nan(BF))
    if "y" in parts:
        out["x_out"] = nan(a["x"].dtype)
    h, x = run(a, **out)
    assert h is out["h"] and x is out.get("x_out", x)
    want_h, want_x, far_h, far_x = block(**a)
    check(h, want_h, far_h + U16 * (want_h.abs() + far_h), "h")
    if "y" in parts:
        check(x, want_x, far_x + (U32 if wide else U16) * (want_x.abs() + far_x), "x")


PARTS = [(False, "wynpgs"), (True, "wynpgs"), (False, ""), (True, "wyp")]


@pytest.mark.parametrize("W", [8, 264, 1928, 2056, 4104, 8192, 12288, 16392])
@pytest.mark.parametrize("wide,parts", PARTS)
def test_widths(W, wide, parts):
    every_row(1500 if W < 3000 else 650, W, wide, parts)


@pytest.mark.parametrize("rounds,more", [(4, -1), (4, 0), (4, 1), (9, 7), (33, -5)])
@pytest.mark.parametrize("wide,parts", PARTS)
def test_numbers_of_rows(rounds, more, wide, parts):
    """Around the number that decides between the two ways (four an SM), and rows left over in the last round."""
    every_row(rounds * torch.cuda.get_device_properties(0).multi_processor_count + more, 520, wide, parts)
