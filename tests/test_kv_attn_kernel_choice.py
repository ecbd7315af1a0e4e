"""Which kernel a chunk takes (no GPU needed): tests that are written for one of them rely on it."""
import pytest

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def test_bad_sizes():
    for sizes in ((-1, 5, 8, 2, 64), (1, -5, 8, 2, 64), (1, 5, 0, 1, 64), (1, 5, 8, 0, 64), (1, 5, 8, 3, 64), (1, 5, 8, 2, -1)):
        assert kda.debug_attention_kernel(*sizes) == -1


def test_rule():
    few, many = 0, 1
    assert kda.debug_attention_kernel(1, 8192, 96, 8, 8192) == many
    assert kda.debug_attention_kernel(8, 128, 96, 8, 8128) == many
    assert kda.debug_attention_kernel(3, 77, 16, 2, 1536) == few
    # up to 64 rows (tokens times shared heads) a sequence on average, whatever the table's width
    assert kda.debug_attention_kernel(4, 64, 32, 8, 1 << 30) == few
    assert kda.debug_attention_kernel(4, 65, 32, 8, 1 << 30) == many
    # little work altogether, bounded by the table's width
    assert kda.debug_attention_kernel(1, 100, 8, 2, 6000) == few
    assert kda.debug_attention_kernel(1, 100, 8, 2, 6200) == many
