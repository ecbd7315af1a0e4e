"""What kda_block_norm refuses of an output that lies over its input (no GPU needed)."""
import pytest

from test_lin_abi import HAS_GPU, INVALID, OK, CUDA, UNSUPPORTED, _norm, lib  # noqa: F401 (fixture)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("parts", [dict(), dict(gate=0, pw=0, post=0)])
def test_rows_apart_are_not_updated_in_place(lib, dtype, parts):  # noqa: F811
    """x' is written without gaps: over rows of x that have gaps it would come upon rows that are still to be read."""
    assert _norm(lib, dtype=dtype, xs=72, x_out=0x1000, **parts) == INVALID
    assert _norm(lib, dtype=dtype, xs=128, x_out=0x1000, rows=2, **parts) == INVALID
    assert _norm(lib, dtype=dtype, xs=32, x_out=0x1000, rows=2, **parts) == INVALID
    assert _norm(lib, dtype=dtype, xs=72, x_out=0x1000, rows=0, **parts) == OK
    if not HAS_GPU:  # one row, or rows without gaps: as far as the launch
        assert _norm(lib, dtype=dtype, xs=72, x_out=0x1000, rows=1, **parts) in (CUDA, UNSUPPORTED)
        assert _norm(lib, dtype=dtype, xs=64, x_out=0x1000, **parts) in (CUDA, UNSUPPORTED)
