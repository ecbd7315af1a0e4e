"""attn_prefill_paged on its tensor-core kernel (kda_attn_chunk.cu) against the 64-bit statements.

Calls of little work go to the warp-level kernel; the work is bounded by the page table's width, so
a table much wider than the sequences sends small inputs through the tensor-core kernel."""
import functools
import inspect
import math

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
import test_kv_attn_gpu as base
from kv_attn_util import D, Cache, attention, check, visible
from test_kv_attn_gpu import gen, reference, run_decode, run_prefill

pytestmark = pytest.mark.gpu

WIDE = 1 << 17  # tokens that the page tables have room for


def wide(page):
    return WIDE // page


@pytest.fixture(autouse=True)
def kernel_is_named(request, monkeypatch):
    """Every prefill call here is of the kernel that the test says: its "kernel" parameter, or the
    tensor-core kernel."""
    params = getattr(getattr(request.node, "callspec", None), "params", {})
    want = 0 if params.get("kernel") == "few rows" else 1
    call = kda.attn_prefill_paged

    def attn_prefill_paged(q, k_pool, v_pool, page_table, *a, **kw):
        got = kda.debug_attention_kernel(page_table.shape[0], q.shape[0], q.shape[1], k_pool.shape[1],
                                         page_table.shape[1] * k_pool.shape[2])
        assert got == want, "the call goes to the other kernel"
        return call(q, k_pool, v_pool, page_table, *a, **kw)

    monkeypatch.setattr(kda, "attn_prefill_paged", attn_prefill_paged)


# ---------------------------------------------- the tests of small prefill calls, on this kernel
def again(test):
    """A test of test_kv_attn_gpu.py, with its parameters, over wide tables."""
    @functools.wraps(test)
    def run(monkeypatch, **kw):
        monkeypatch.setattr(base, "Cache", lambda lens, Hkv, page, *a, **k: Cache(lens, Hkv, page, *a, max_pages=wide(page), **k))
        test(**kw)

    names = list(inspect.signature(test).parameters)
    run.__signature__ = inspect.Signature([inspect.Parameter(n, inspect.Parameter.POSITIONAL_OR_KEYWORD) for n in names + ["monkeypatch"]])
    return run


test_prefill = again(base.test_prefill)
test_prefill_edges_far_apart = again(base.test_prefill_edges_far_apart)
test_prefill_rows_before_the_first_token = again(base.test_prefill_rows_before_the_first_token)
test_strided_queries_scales_and_long_range = again(base.test_strided_queries_scales_and_long_range)
test_nonfinite_rows_reach_only_rows_that_see_them = again(base.test_nonfinite_rows_reach_only_rows_that_see_them)
test_prefill_scales_far_apart = again(base.test_prefill_scales_far_apart)
test_same_bits_again_on_other_streams_and_in_graphs = again(base.test_same_bits_again_on_other_streams_and_in_graphs)


def test_rows_at_the_least_scale(monkeypatch):
    again(base.test_rows_at_the_least_scale)(monkeypatch, decode=False)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_behind_the_window_are_not_needed(fp8, page):
    g = gen(page)
    new, lens = [200, 1], [900, 50]
    c = Cache(lens, 2, page, fp8, g, max_pages=wide(page))
    q = torch.randn(201, 8, D, generator=g).to(torch.bfloat16)
    ref = reference(c, torch.split(q, new), new, lens, 100, 20, D ** -0.5)
    c.table[0, -(-20 // page):601 // page] = -1  # visible: 0 .. 19 and 601 .. 899
    o, lse = run_prefill(c, q.cuda(), new, lens, 100, 20)
    check(o, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths_report(fp8):
    """Bad entries among visible pages, lengths and offsets are reported; other sequences keep their bits."""
    g = gen(4)
    new, lens = [120, 150, 90], [300, 400, 90]
    c = Cache(lens, 2, 32, fp8, g, max_pages=wide(32))
    q = torch.randn(360, 4, D, generator=g).to(torch.bfloat16).cuda()
    good, _ = run_prefill(c, q, new, lens)
    ends = torch.tensor(new).cumsum(0).tolist()
    for entry in (-1, 9999, -5):
        table = c.table.clone()
        c.table[1, 3] = entry
        o, _ = run_prefill(c, q, new, lens, status=base.DEVICE_CHECK)
        c.table.copy_(table)
        for a, b in ((0, ends[0]), (ends[1], ends[2])):
            check_close(o[a:b], good[a:b])
    for bad in (-1, WIDE + 1):
        o = torch.full_like(good, 3.0)
        run_prefill(c, q, new, [lens[0], bad, lens[2]], status=base.DEVICE_CHECK, o=o)
        assert (o[ends[0]:ends[1]] == 3).all()
        for a, b in ((0, ends[0]), (ends[1], ends[2])):
            check_close(o[a:b], good[a:b])


def check_close(a, b):
    """Sequences of another batch: split elsewhere, so the sums' last bits and one rounding of o may
    differ; 2^-8 of the largest is far above that."""
    assert ((a.float() - b.float()).abs().max() <= 2.0 ** -8 * 2 * b.float().abs().max())


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


@pytest.mark.parametrize("kernel", ["many rows", "few rows", "decode"])
@pytest.mark.parametrize("k_down,v_down", [([50], [50]), ([0, 47], [0]), ([0], [0, 45, 62]), ([40, 47, 50, 57], [40, 41]), ([-55], [-55, -20]),
                                           ([72], [72]), ([-84], [-84]), ([-30, 30], [-49, 49])])
def test_scales_that_others_write(kernel, k_down, v_down):
    """Scale bytes below and above those that kda_kv_append writes, alone and next to ordinary ones, rows of zeros among them."""
    g = gen(len(k_down) + 10 * len(v_down))
    new = [150, 130]
    lens = [400, 130]

    def values(n, i, x):
        x[3::11] = 0
        return x

    c = Cache(lens, 2, 32, True, g, values=values, max_pages=wide(32) if kernel == "many rows" else None)
    for n, down in (("k", k_down), ("v", v_down)):
        byte = c.scales[n + "_scale"].cpu()
        for i, t in enumerate(lens):  # the rows' scales go down, a choice by row and head
            by = torch.tensor(down)[torch.randint(len(down), (t, 2), generator=g)]
            j = torch.arange(t)
            page, slot = c.table[i].cpu().long()[j // 32], j % 32
            byte[page, :, slot] = (byte[page, :, slot].long() - by).to(torch.uint8)
            c.value[n][i] = c.value[n][i] * torch.exp2(-by.double())[..., None]
        c.scales[n + "_scale"].copy_(byte)
    q = (torch.randn(sum(new), 8, D, generator=g) * 2.0 ** (sum(k_down) / len(k_down))).to(torch.bfloat16)
    if kernel == "decode":
        q = q[:4]
        o, lse = run_decode(c, q.view(2, 2, 8, D).cuda(), lens)
        o, lse, new = o.flatten(0, 1), lse.flatten(0, 1), [2, 2]
    elif kernel == "few rows":
        new = [10, 5]
        q = q[:15]
        o, lse = run_prefill(c, q.cuda(), new, lens)
    else:
        o, lse = run_prefill(c, q.cuda(), new, lens)
    check(o, lse, reference(c, torch.split(q, new), new, lens, 0, 0, D ** -0.5))


@pytest.mark.parametrize("exponent", [119, 100, 0, -110])
@pytest.mark.parametrize("rise", [5.0, 12.0, 40.0])
def test_rising_scores_and_values_of_any_size(exponent, rise):
    """Scores that rise along the keys, by tiles, with values near the ends of bf16's range."""
    g = gen(exponent + 200)
    new, lens = [140, 60], [1100, 700]

    def values(n, i, x):
        if n == "v":
            return (x.clamp(-4, 4).float() * 2.0 ** exponent).to(torch.bfloat16)
        x = x * 0.1
        x[..., 0] = torch.linspace(-0.5, 0.5, x.shape[0])[:, None] * rise  # times the queries' first channel
        return x

    c = Cache(lens, 2, 64, False, g, values=values, max_pages=wide(64))
    q = torch.randn(sum(new), 8, D, generator=g)
    q[..., 0] = D ** 0.5
    q = q.to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens)
    check(o, lse, reference(c, torch.split(q, new), new, lens, 0, 0, D ** -0.5))


@pytest.mark.parametrize("kernel", ["many rows", "few rows", "decode"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("exponent", [18, 23, 26, 28, 30, 34, 50])
def test_scores_far_beyond_what_32_bits_tell_apart(kernel, fp8, exponent):
    """Scores of 2^20 to 2^53: whichever key wins, every result is finite and a mean of values."""
    g = gen(exponent)
    new, lens = [150, 70], [700, 70]
    c = Cache(lens, 2, 64, fp8, g, max_pages=wide(64) if kernel == "many rows" else None)
    q = (torch.randn(sum(new), 8, D, generator=g) * 2.0 ** exponent).to(torch.bfloat16)
    if kernel == "decode":
        q, new = q[:4], [2, 2]
        o, lse = run_decode(c, q.view(2, 2, 8, D).cuda(), lens)
        o, lse = o.flatten(0, 1), lse.flatten(0, 1)
    elif kernel == "few rows":
        q, new = q[:15], [10, 5]
        o, lse = run_prefill(c, q.cuda(), new, lens)
    else:
        o, lse = run_prefill(c, q.cuda(), new, lens)
    check(o, lse, reference(c, torch.split(q, new), new, lens, 0, 0, D ** -0.5))


def e4m3_bounds(c, i, q, see, loss):
    """The bounds of kv_attn_util.attention with the f16 weights' own term: a weight times 2^ev is off by
    2^-11 of itself or by `loss` of the largest that the row sees."""
    k, v = c.value["k"][i], c.value["v"][i]
    total, Hkv = k.shape[:2]
    ro, rl, bo, bl = attention(q, k, v, see, D ** -0.5, True)
    j = torch.arange(total)
    byte = c.scales["v_scale"].cpu()[c.table[i].cpu().long()[j // c.page], :, j % c.page].long()
    size = torch.exp2(byte.double() - 127)  # [total, Hkv]
    for h in range(q.shape[1]):
        kh, vh, ev = k[:, h * Hkv // q.shape[1]], v[:, h * Hkv // q.shape[1]], size[:, h * Hkv // q.shape[1]]
        qh = q[:, h].double()
        x = torch.where(see, qh @ kh.T * D ** -0.5, -math.inf)
        w = torch.exp(x - torch.logsumexp(x, 1)[:, None])
        dx = 136 * 2.0 ** -24 * (qh.abs() @ kh.abs().T * D ** -0.5).amax(1) + 8 * 2.0 ** -24 * x.masked_fill(~see, 0).abs().amax(1)
        rel = 2 * dx + 2.0 ** -20 + 2 * total * 2.0 ** -24 + 2.0 ** -11
        codes = torch.where(see[:, :, None], (vh / ev[:, None]).abs(), 0.0).sum(1)
        bo[:, h] = 2.0 ** -8 * ro[:, h].abs() + 1.01 * rel[:, None] * (w @ vh.abs()) + loss * (w * ev).amax(1)[:, None] * codes
    return ro, rl, bo, bl


@pytest.mark.parametrize("kernel", ["many rows", "few rows", "decode"])
@pytest.mark.parametrize("above,score", [(7, -12), (8, -12), (9, -12), (12, -12), (14, -12), (15, -12), (16, -12), (24, -12), (24, -1)])
def test_one_large_value_row(kernel, above, score):
    """A value row 2^above times the others', in one channel, that hardly any row attends to, and one
    that stands behind the queries of its tile.  A key that takes most of the weight is zero in half of
    the channels, which are then those of 1500 ordinary keys with some 2^-13 of its weight each."""
    g = gen(above)
    new, lens = [300], [1500]

    def values(n, i, x):
        x = x / x.abs().amax(-1, keepdim=True)  # a scale for all
        if n == "k":
            x[:, :, 0] = 0
            for j, s in ((3, 9.0), (70, score), (1390, 0.0)):
                x[j] = 0
                x[j, :, 0] = s  # times the queries' first channel
        else:
            x[3, :, 64:] = 0
            for j in (70, 1390):
                x[j] = 0
                x[j, :, 3] = 2.0 ** above
        return x

    c = Cache(lens, 2, 64, True, g, values=values, max_pages=wide(64) if kernel == "many rows" else None)
    q = torch.randn(300, 4, D, generator=g)
    q[..., 0] = D ** 0.5
    q = q.to(torch.bfloat16)
    if kernel == "decode":
        q, new = q[:3], [3]
        o, lse = run_decode(c, q[None].cuda(), lens)
        o, lse = o[0], lse[0]
    elif kernel == "few rows":
        q, new = q[:20], [20]
        o, lse = run_prefill(c, q.cuda(), new, lens)
    else:
        o, lse = run_prefill(c, q.cuda(), new, lens)
    see = visible(new[0], lens[0], 0, 0)
    check(o, lse, e4m3_bounds(c, 0, q, see, 2.0 ** -24 if kernel == "many rows" else 2.0 ** -39))


@pytest.mark.parametrize("kernel", ["many rows", "few rows", "decode"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("score", [-10.0, -150.0, -400.0])
@pytest.mark.parametrize("at", [40, 995])
def test_nan_values_of_keys_without_weight(kernel, fp8, score, at):
    """A NaN value row makes the rows that see it NaN, however small its weight; in a tile that all rows
    see and in the last one."""
    g = gen(at)
    new, lens = [130], [1000]

    def values(n, i, x):
        if n == "k":
            x[:, :, 0] = 0
            x[at] = 0
            x[at, :, 0] = score  # times the queries' first channel
        else:
            x[at, :, 9] = math.nan
        return x

    c = Cache(lens, 2, 64, fp8, g, values=values, max_pages=wide(64) if kernel == "many rows" else None)
    q = torch.randn(130, 8, D, generator=g)
    q[..., 0] = D ** 0.5
    q = q.to(torch.bfloat16)
    if kernel == "decode":
        q, new = q[:4], [4]
        o, lse = run_decode(c, q[None].cuda(), lens)
        o, lse = o[0], lse[0]
    elif kernel == "few rows":
        q, new = q[:12], [12]
        o, lse = run_prefill(c, q.cuda(), new, lens)
    else:
        o, lse = run_prefill(c, q.cuda(), new, lens)
    ro, rl, bo, bl = reference(c, torch.split(q, new), new, lens, 0, 0, D ** -0.5)
    bad = torch.isnan(ro).any(-1)
    assert bad.any() and (at == 40 or kernel == "decode" or not bad.all())
    lse[bad.cuda()] = 0
    rl[bad] = 0
    check(o, lse, (ro, rl, bo, bl))


@pytest.mark.parametrize("kernel", ["many rows", "few rows"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [1023, 1025, 2600])
def test_more_sequences_than_a_plan_takes_at_a_time(kernel, fp8, N):
    """The list of row tiles is made 1024 sequences, then 1024 tiles, at a time; some sequences are empty."""
    g = gen(N)
    H = 72 if kernel == "many rows" else 6
    new = [(1, 0, 3, 1, 2)[i % 5] for i in range(N)]
    new[N // 2] = 40
    lens = [n + i % 7 for i, n in enumerate(new)]
    c = Cache(lens, 1, 16, fp8, g, max_pages=wide(16) if kernel == "many rows" else None)
    q = torch.randn(sum(new), H, D, generator=g).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens)
    parts = torch.split(q, new)
    some = [i for i in range(N) if new[i] and (i % 37 == 0 or abs(i - N // 2) < 3 or i > N - 8 or 1018 < i < 1030)]
    at = torch.tensor([0] + new).cumsum(0).tolist()
    for i in some:
        see = visible(new[i], lens[i], 0, 0)
        check(o[at[i]:at[i + 1]], lse[at[i]:at[i + 1]], attention(parts[i], c.value["k"][i], c.value["v"][i], see, D ** -0.5, fp8))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("kernel", ["many rows", "few rows"])
@pytest.mark.parametrize("cu", [[0, 50, 20, 70], [-5, 20, 40, 70], [0, 30, 50, 71], [0, 80, 60, 70]])
def test_bad_offsets_report(kernel, cu):
    """Offsets that run backwards, begin before the rows or end past them."""
    g = gen(6)
    c = Cache([60, 90, 80], 2, 32, False, g, max_pages=wide(32) if kernel == "many rows" else None)
    H = 32 if kernel == "many rows" else 4
    q = torch.randn(70, H, D, generator=g).to(torch.bfloat16).cuda()
    st = base.i32(0)
    around = torch.full((90, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.attn_prefill_paged(q, *c.args, base.i32(*cu), base.i32(60, 90, 80), o=around[10:80], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == base.DEVICE_CHECK
    assert (around[:10] == 5).all() and (around[80:] == 5).all()
