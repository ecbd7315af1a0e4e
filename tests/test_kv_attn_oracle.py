"""The plain statements that the attention cache is held to (kv_attn_util.py), checked by hand
values and by torch's own conversions (no GPU needed)."""
import math

import torch

from kv_attn_util import D, Cache, attention, pow2, quantise, stored, visible


def test_quantise_hand_values():
    x = torch.zeros(6, D)
    x[0, 0] = 448.0            # 448 * 2^0
    x[1, 0] = 450.0            # the next power of two
    x[2, 0], x[2, 1] = 1.0, 1.0 / 16 + 1.0 / 512  # 1 = 256 * 2^-8: the second value is 16.5 * 2^-8, a tie to 16
    x[3, 0] = 2.0 ** -60
    x[4, 0] = math.inf
    codes, byte = quantise(x.to(torch.bfloat16))
    assert byte.tolist() == [127, 128, 127 - 8, 87, 255, 87]
    assert codes[0, 0] == 448 and codes[1, 0] == 224  # 450 is 450 = 225 * 2: rounds to 224
    assert codes[2, 0] == 256 and codes[2, 1] == 16
    assert codes[3, 0] == 0 and codes[4].abs().sum() == 0


def test_quantise_matches_torch_rounding():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(200, D, generator=g) * torch.exp2(8 * torch.randn(200, 1, generator=g))).to(torch.bfloat16)
    codes, byte = quantise(x)
    scaled = x.double() / pow2(byte.to(torch.int64) - 127)[:, None]
    assert torch.equal(scaled.float().to(torch.float8_e4m3fn).double(), codes)
    assert (scaled.abs().amax(1) <= 448).all() and (scaled.abs().amax(1) > 224).all()


def test_visible_hand_values():
    assert visible(2, 5, 0, 0).tolist() == [[True] * 4 + [False], [True] * 5]
    assert visible(1, 6, 2, 1).tolist() == [[True, False, False, False, True, True]]
    assert visible(3, 2, 0, 0).tolist() == [[False, False], [True, False], [True, True]]


def test_attention_closed_forms():
    """Equal keys average the values; one key far above the others returns its value; a row that
    sees nothing is zero with a sum of log 0; shared heads read their head."""
    v = torch.randn(4, 2, D, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    q = torch.ones(1, 4, D)
    o, lse, bo, bl = attention(q, torch.zeros(4, 2, D, dtype=torch.float64), v, visible(1, 4, 0, 0), 0.1, False)
    assert torch.allclose(o[0, 1], v[:, 0].mean(0)) and torch.allclose(o[0, 3], v[:, 1].mean(0))
    assert torch.allclose(lse, torch.full((1, 4), math.log(4), dtype=torch.float64))
    k = torch.zeros(4, 2, D, dtype=torch.float64)
    k[2] = 10.0
    o, _, bo, _ = attention(q, k, v, visible(1, 4, 0, 0), 1.0, False)
    assert torch.allclose(o[0, 0], v[2, 0]) and (bo > 0).all()
    o, lse, _, _ = attention(q, k, v, torch.zeros(1, 4, dtype=torch.bool), 1.0, False)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_cache_holds_what_it_says():
    for fp8 in (False, True):
        c = Cache([5, 40], 2, 16, fp8, torch.Generator().manual_seed(3), device="cpu")
        for i, t in enumerate((5, 40)):
            for j in range(t):
                p, s = int(c.table[i, j // 16]), j % 16
                row = c.k[p, :, s].float().double()
                if fp8:
                    row = row * pow2(c.scales["k_scale"][p, :, s].to(torch.int64) - 127)[:, None]
                assert torch.equal(row, c.value["k"][i][j])
    rows, byte, val = stored(torch.full((1, 1, D), math.nan, dtype=torch.bfloat16), True)
    assert int(byte) == 255 and torch.isnan(val).all() and (rows.float() == 0).all()
