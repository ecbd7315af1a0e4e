"""The attention cache's operators against plain statements in 64 bits (kv_attn_util.py)."""
import math

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kv_attn_util import D, Cache, attention, check, quantise, stored, visible

pytestmark = pytest.mark.gpu

DEVICE_CHECK = 7


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(new):
    return i32(0, *torch.tensor(new).cumsum(0).tolist()) if new else i32(0)


def reference(c, q_of, new, lens, window, sink, scale):
    parts = [attention(q_of[i], c.value["k"][i], c.value["v"][i], visible(new[i], lens[i], window, sink), scale, c.fp8)
             for i in range(len(lens))]
    return [torch.cat(x) for x in zip(*parts)]


def run_prefill(c, q, new, lens, window=0, sink=0, scale=None, status=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kda.attn_prefill_paged(q, *c.args, offsets(new), i32(*lens), **c.scales, window=window, n_sink=sink, scale=scale,
                                    return_lse=True, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    return o, lse


def run_decode(c, q, lens, window=0, sink=0, scale=None, status=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kda.attn_decode_paged(q, *c.args, i32(*lens), **c.scales, window=window, n_sink=sink, scale=scale, return_lse=True,
                                   dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    return o, lse


# ------------------------------------------------------------------------------ append, read
def special_rows():
    x = torch.zeros(12, D)
    x[0, 3] = math.nan
    x[1, 127] = math.inf
    x[2, 5] = -math.inf
    x[3] = 448.0                      # the largest code
    x[4] = 449.0 * 1.01               # just above: the next scale
    x[5, 0], x[5, 1] = 1.0, 2.0 ** -30  # far below the row's top
    x[6] = 2.0 ** -60                 # under the least scale
    x[7, 9] = 448.0 * 2.0 ** 40
    x[8, 9] = 448.0 * 2.0 ** 41       # above the greatest scale
    x[9] = -0.0
    x[10] = torch.linspace(-1, 1, D)
    x[11] = 17.0 * 2.0 ** -9 * torch.arange(D)  # ties
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,new,start", [(1, [1], [0]), (2, [5, 0, 33, 1], [0, 7, 15, 130]), (8, [70, 3], [250, 1]),
                                           (3, [12] * 9, [0, 1, 2, 3, 4, 5, 6, 7, 8])])
def test_append_then_read(fp8, page, Hkv, new, start):
    g = gen(page + Hkv)
    T, N = sum(new), len(new)
    lens = [a + b for a, b in zip(new, start)]
    n_of = [(t + page - 1) // page for t in lens]
    n_pages = sum(n_of) + 2
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((N, max(n_of)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(n_of):
        table[i, :n] = perm[at:at + n]
        at += n
    x = {n: (torch.randn(T, Hkv, D, generator=g) * torch.exp2(4 * torch.randn(T, Hkv, 1, generator=g))).to(torch.bfloat16) for n in "kv"}
    if T >= 12:
        x["k"][:12, 0] = special_rows()
        x["v"][:12, Hkv - 1] = special_rows()
    fused = torch.stack([x["k"], x["v"]], 1).cuda()  # [T, 2, Hkv, D]: strided rows
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    raw = torch.uint8 if fp8 else torch.int16
    pools = [torch.full((n_pages, Hkv, page, D), 77, dtype=raw, device="cuda").view(kind) for _ in range(2)]
    scales = dict(k_scale=torch.full((n_pages, Hkv, page), 99, dtype=torch.uint8, device="cuda"),
                  v_scale=torch.full((n_pages, Hkv, page), 99, dtype=torch.uint8, device="cuda")) if fp8 else {}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, s0 = offsets(new), i32(*start)
    kda.kv_append(fused[:, 0], fused[:, 1], *pools, table.cuda(), cu, s0, **scales, dev_status=st)
    back = kda.kv_read(*pools, table.cuda(), cu, s0, T, **scales, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    touched = torch.zeros(n_pages, page, dtype=torch.bool)
    for m, n in enumerate("kv"):
        rows, byte, value = stored(x[n], fp8)
        pool = pools[m].cpu()
        at = 0
        for i in range(N):
            for t in range(new[i]):
                p, s = int(table[i, (start[i] + t) // page]), (start[i] + t) % page
                touched[p, s] = True
                assert torch.equal(pool[p, :, s].float(), rows[at].float()) or torch.isnan(rows[at].float()).any()
                assert torch.equal(torch.isnan(pool[p, :, s].float()), torch.isnan(rows[at].float()))
                if fp8:
                    assert torch.equal(scales["kv"[m] + "_scale"].cpu()[p, :, s], byte[at])
                at += 1
        want = value.to(torch.bfloat16)
        got = back[m].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))
        left = pool.view(raw).transpose(1, 2)[~touched]
        assert (left == 77).all()
        if fp8:
            assert (scales["kv"[m] + "_scale"].cpu().transpose(1, 2)[~touched] == 99).all()


def test_append_bad_tables_skip_rows():
    """-1 leaves a token unwritten; bad pages, positions past the table and negative starts are
    reported, and only their rows are skipped."""
    k = torch.ones(6, 2, D, dtype=torch.bfloat16, device="cuda")
    for table, start, status in (([[0, -1, 2]], [0], 0), ([[0, 9, 2]], [0], DEVICE_CHECK), ([[0, -7, 2]], [0], DEVICE_CHECK),
                                 ([[0, 1, 2]], [44], DEVICE_CHECK), ([[0, 1, 2]], [-1], DEVICE_CHECK)):
        kp, vp = (torch.zeros(4, 2, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        # rows at positions 14 .. 19 (pages 0 and 1), 44 .. 49 (48 is past the table)
        s0 = start[0] + 14 if start[0] == 0 else start[0]
        kda.kv_append(k, k, kp, vp, torch.tensor(table, dtype=torch.int32, device="cuda"), i32(0, 6), i32(s0), dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == status
        written = int(kp[:, 0, :, 0].sum())
        assert written == {0: 2, DEVICE_CHECK: {14: 2, 44: 4, -1: 0}[s0]}[status]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko = torch.full((6, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.kv_read(kp, vp, torch.tensor([[0, -1, 2]], dtype=torch.int32, device="cuda"), i32(0, 6), i32(14), 6, k=ko, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == DEVICE_CHECK
    assert (ko[2:] == 5).all() and (ko[:2] == kp[0, :, 14:16].transpose(0, 1)).all()


# ------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,layout", [(16, "heads"), (32, "tokens"), (64, "pair"), (128, "heads")])
@pytest.mark.parametrize("H,Hkv,n_tok", [(2, 2, 1), (12, 1, 1), (8, 2, 4), (12, 2, 4), (16, 1, 4), (30, 1, 3)])
def test_decode(fp8, page, layout, H, Hkv, n_tok):
    g = gen(H + n_tok + page)
    lens = [n_tok, 64, 65, 1000, n_tok + 1, 127, 300]
    c = Cache(lens, Hkv, page, fp8, g, layout)
    q = torch.randn(len(lens), n_tok, H, D, generator=g).to(torch.bfloat16)
    for window, sink in ((0, 0), (37, 0), (64, 5), (200, 70)):
        o, lse = run_decode(c, q.cuda(), lens, window, sink)
        ref = reference(c, q, [n_tok] * len(lens), lens, window, sink, D ** -0.5)
        check(o.flatten(0, 1), lse.flatten(0, 1), ref)


def test_decode_idle_and_short_slots():
    """Slots with nothing cached, or fewer tokens than the step has: rows before the first token see nothing."""
    g = gen(3)
    lens = [0, 2, 5, 0, 1]
    c = Cache(lens, 2, 16, False, g)
    q = torch.randn(len(lens), 3, 4, D, generator=g).to(torch.bfloat16)
    o, lse = run_decode(c, q.cuda(), lens)
    for i, t in enumerate(lens):
        see = (torch.arange(t) <= torch.arange(t - 3, t)[:, None]) if t else torch.zeros(3, 0, dtype=torch.bool)
        check(o[i], lse[i], attention(q[i], c.value["k"][i], c.value["v"][i], see, D ** -0.5, False))


@pytest.mark.parametrize("B", [1, 161, 500])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_batches_and_one_long(B, fp8):
    """More sequences than a block has threads, one of them long: shares begin and end anywhere."""
    g = gen(B)
    lens = [1 + (37 * i) % 90 for i in range(B)]
    lens[B // 2] = 6000
    c = Cache(lens, 1, 64, fp8, g)
    q = torch.randn(B, 1, 3, D, generator=g).to(torch.bfloat16)
    o, lse = run_decode(c, q.cuda(), lens)
    check(o.flatten(0, 1), lse.flatten(0, 1), reference(c, q, [1] * B, lens, 0, 0, D ** -0.5))


def test_decode_bad_lengths_and_pages_report():
    g = gen(9)
    lens = [40, 40, 40]
    c = Cache(lens, 2, 16, False, g)
    q = torch.randn(3, 1, 4, D, generator=g).to(torch.bfloat16).cuda()
    good, _ = run_decode(c, q, lens)
    for bad in (-1, 49):
        o = torch.full_like(good, 3.0)
        run_decode(c, q, [40, bad, 40], status=DEVICE_CHECK, o=o)
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and (o[1] == 3).all()
    for entry in (-1, 99, -5):
        table = c.table.clone()
        table[1, 1] = entry
        o, _ = kda.attn_decode_paged(q, c.k, c.v, table, i32(*lens), dev_status=(st := i32(0)), return_lse=True)
        torch.cuda.synchronize()
        assert int(st) == DEVICE_CHECK
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])


# ----------------------------------------------------------------------------------- prefill
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,layout", [(16, "pair"), (32, "heads"), (64, "tokens"), (128, "heads")])
@pytest.mark.parametrize("H,Hkv,new,past", [
    (2, 2, [1, 130, 64], [0, 3, 500]), (12, 1, [11, 0, 300, 1], [0, 9, 100, 257]), (6, 2, [257], [0]), (96, 8, [23, 5], [40, 0]),
    (3, 1, [128, 129, 127], [128, 127, 129])])
def test_prefill(fp8, page, layout, H, Hkv, new, past):
    g = gen(H + sum(new) + page)
    lens = [a + b for a, b in zip(new, past)]
    c = Cache(lens, Hkv, page, fp8, g, layout)
    q = torch.randn(sum(new), H, D, generator=g).to(torch.bfloat16)
    for window, sink in ((0, 0), (50, 0), (33, 3), (128, 140)):
        o, lse = run_prefill(c, q.cuda(), new, lens, window, sink)
        check(o, lse, reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,past,window,sink", [([700, 64, 300], [2500, 900, 0], 1100, 4), ([900], [3100], 0, 0),
                                                  ([130, 1500], [1700, 20], 640, 200)])
def test_prefill_edges_far_apart(fp8, new, past, window, sink):
    """Masked tiles with runs of whole tiles between them, longer than the ring of stages."""
    g = gen(window)
    lens = [a + b for a, b in zip(new, past)]
    c = Cache(lens, 1, 128, fp8, g)
    q = torch.randn(sum(new), 2, D, generator=g).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), new, lens, window, sink)
    check(o, lse, reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5))


def test_prefill_rows_before_the_first_token():
    """More new tokens than the cache holds: the first rows see nothing."""
    g = gen(31)
    c = Cache([40], 2, 16, False, g)
    q = torch.randn(60, 4, D, generator=g).to(torch.bfloat16)
    o, lse = run_prefill(c, q.cuda(), [60], [40])
    see = torch.arange(40) <= torch.arange(-20, 40)[:, None]
    check(o, lse, attention(q, c.value["k"][0], c.value["v"][0], see, D ** -0.5, False))


@pytest.mark.parametrize("fp8", [False, True])
def test_strided_queries_scales_and_long_range(fp8):
    """Queries inside a fused projection, a scale of its own (negative too), queries of very different size."""
    g = gen(17)
    new, lens = [70, 9], [200, 9]
    c = Cache(lens, 2, 64, fp8, g)
    wide = torch.randn(79, 3, 4, D, generator=g) * torch.exp2(6 * torch.randn(79, 1, 4, 1, generator=g))
    wide = (wide * torch.where(torch.rand(wide.shape, generator=g) < 0.01, 30.0, 1.0)).to(torch.bfloat16)
    q = wide[:, 1]
    for scale in (0.01, -0.02, 0.0):
        o, lse = run_prefill(c, wide.cuda()[:, 1], new, lens, scale=scale)
        check(o, lse, reference(c, torch.split(q, new), new, lens, 0, 0, scale))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nonfinite_rows_reach_only_rows_that_see_them(fp8, what, where):
    """A non-finite key or value row of a new token spoils that token and later ones, no earlier
    one; of a token behind the window, only those whose window still holds it."""
    g = gen(5)
    new, lens = [150, 40], [300, 40]

    def values(n, i, x):
        if n == where:
            for j in (20, 151, 230):
                if j < x.shape[0]:
                    x[j, 0, 7] = what
        return x

    c = Cache(lens, 2, 32, fp8, g, values=values)
    q = torch.randn(190, 4, D, generator=g).to(torch.bfloat16)
    for window, sink in ((0, 0), (30, 0), (30, 24)):
        if where == "k" and not fp8 and math.isinf(what):
            continue  # an infinite score may be either infinity: nothing is promised but the rows that do not see it
        o, lse = run_prefill(c, q.cuda(), new, lens, window, sink)
        ro, rl, bo, bl = reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5)
        bad = torch.isnan(ro).any(-1)
        lse[bad.cuda()] = 0
        rl[bad] = 0
        check(o, lse, (ro, rl, bo, bl))


def test_pages_behind_the_window_are_not_needed():
    g = gen(8)
    lens = [700]
    c = Cache(lens, 1, 16, False, g)
    q = torch.randn(1, 2, 4, D, generator=g).to(torch.bfloat16)
    ref = reference(c, q, [2], lens, 100, 20, D ** -0.5)
    c.table[0, 2:37] = -1  # tokens 32 .. 591; visible: 0 .. 19 and 599 .. 699
    o, lse = run_decode(c, q.cuda(), lens, 100, 20)
    check(o[0], lse[0], ref)
    o, lse = run_prefill(c, q[0].cuda(), [2], lens, 100, 20)
    check(o, lse, ref)


def test_extreme_value_scales():
    """Value rows whose scales lie 2^80 apart: the large ones' weights vanish against e^-x."""
    g = gen(12)

    def values(n, i, x):
        if n == "v":
            x[::3] *= 2.0 ** -38
            x[1::3] *= 2.0 ** 30
        return x

    c = Cache([200, 130], 1, 16, True, g, values=values)
    q = torch.randn(2, 2, 5, D, generator=g).to(torch.bfloat16)
    o, lse = run_decode(c, q.cuda(), [200, 130])
    check(o.flatten(0, 1), lse.flatten(0, 1), reference(c, q, [2, 2], [200, 130], 0, 0, D ** -0.5))


@pytest.mark.parametrize("where", ["k", "v", "kv"])
@pytest.mark.parametrize("spread", [3, 15, 16, 38])
def test_prefill_scales_far_apart(where, spread):
    """Rows whose scales lie just within and beyond what one f16 tile can hold, all-zero rows among them."""
    g = gen(spread)

    def values(n, i, x):
        if n in where:
            x *= torch.where(torch.rand(x.shape[0], 1, 1, generator=g) < 0.1, 2.0 ** -spread, 1.0).to(x.dtype) * 2.0 ** (spread // 2)
        x[5::17] = 0
        return x

    new, lens = [150, 70], [400, 70]
    c = Cache(lens, 2, 32, True, g, values=values)
    q = (torch.randn(220, 4, D, generator=g) * 2.0 ** -(spread // 2 if "k" in where else 0)).to(torch.bfloat16)
    for window, sink in ((0, 0), (90, 3)):
        o, lse = run_prefill(c, q.cuda(), new, lens, window, sink)
        check(o, lse, reference(c, torch.split(q, new), new, lens, window, sink, D ** -0.5))


@pytest.mark.parametrize("decode", [False, True])
def test_rows_at_the_least_scale(decode):
    """Keys and values so small that their scales are the least one, or a few steps above it."""
    g = gen(41)

    def values(n, i, x):
        return x * torch.where(torch.rand(x.shape[0], 1, 1, generator=g) < 0.3, 2.0 ** -30, 2.0 ** -37).to(x.dtype)

    lens = [333, 70]
    c = Cache(lens, 2, 64, True, g, values=values)
    n = [1, 1] if decode else [150, 70]
    q = (torch.randn(sum(n), 4, D, generator=g) * 2.0 ** 30).to(torch.bfloat16)
    if decode:
        o, lse = run_decode(c, q.cuda()[:, None], lens)
        o, lse = o[:, 0], lse[:, 0]
    else:
        o, lse = run_prefill(c, q.cuda(), n, lens)
    check(o, lse, reference(c, torch.split(q, n), n, lens, 0, 0, D ** -0.5))


def test_scores_of_any_size():
    """Rows whose scores spread over hundreds, all very negative or very positive."""
    g = gen(14)
    c = Cache([333], 2, 64, False, g)
    for mul in (40.0, 400.0):
        q = (mul * torch.randn(1, 1, 4, D, generator=g)).to(torch.bfloat16)
        o, lse = run_decode(c, q.cuda(), [333])
        check(o[0], lse[0], reference(c, q, [1], [333], 0, 0, D ** -0.5))


def test_offsets_past_32_bits():
    """Pages 1.2 G elements apart: element offsets of later pages exceed 2^31 and 2^32."""
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 20 GB")
    g = gen(15)
    c = Cache([60], 2, 16, False, g, spare=0)
    step = 1_200_000_000
    far = [torch.empty(4 * step, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wide = [f.as_strided((4, 2, 16, D), (step, 16 * D, D, 1)) for f in far]
    for w, p in zip(wide, (c.k, c.v)):
        w.copy_(p)
    q = torch.randn(1, 2, 4, D, generator=g).to(torch.bfloat16)
    want, _ = run_decode(c, q.cuda(), [60])
    got = kda.attn_decode_paged(q.cuda(), *wide, c.table, i32(60))
    k, v = kda.kv_read(*wide, c.table, i32(0, 60), i32(0), 60)
    assert torch.equal(got, want)
    assert torch.equal(k.cpu().double(), c.value["k"][0]) and torch.equal(v.cpu().double(), c.value["v"][0])
    k.neg_()
    kda.kv_append(k, v, *wide, c.table, i32(0, 60), i32(0))
    assert torch.equal(kda.kv_read(*wide, c.table, i32(0, 60), i32(0), 60)[0], k)


def test_same_bits_again_on_other_streams_and_in_graphs():
    """A call gives the same bits each time, on another stream, with a dirty workspace, and replayed from a graph."""
    g = gen(21)
    new, lens = [200, 31], [5000, 31]
    for fp8 in (False, True):
        c = Cache(lens, 2, 64, fp8, g)
        q = torch.randn(231, 8, D, generator=g).to(torch.bfloat16).cuda()
        q1 = q[:2].unsqueeze(1).contiguous()
        cu, kv = offsets(new), i32(*lens)
        o0 = kda.attn_prefill_paged(q, *c.args, cu, kv, **c.scales)
        d0 = kda.attn_decode_paged(q1, *c.args, kv, **c.scales)
        ws = torch.randint(0, 255, (kda.attn_prefill_workspace_size(2, 231, 8, 2),), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        o1 = kda.attn_prefill_paged(q, *c.args, cu, kv, **c.scales, workspace=ws, stream=s)
        with torch.cuda.stream(s):
            d1 = kda.attn_decode_paged(q1, *c.args, kv, **c.scales)
        torch.cuda.synchronize()
        assert torch.equal(o0, o1) and torch.equal(d0, d1)
        graph = torch.cuda.CUDAGraph()
        k = torch.randn(231, 2, D, generator=g).to(torch.bfloat16).cuda()
        with torch.cuda.graph(graph):
            kda.kv_append(k, k, *c.args, cu, kv - torch.diff(cu), **c.scales)
            o2 = kda.attn_prefill_paged(q, *c.args, cu, kv, **c.scales)
            d2 = kda.attn_decode_paged(q1, *c.args, kv, **c.scales)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, kda.attn_prefill_paged(q, *c.args, cu, kv, **c.scales))
        assert torch.equal(d2, kda.attn_decode_paged(q1, *c.args, kv, **c.scales))
        assert not torch.equal(o2, o0)


def test_empty_calls():
    kp = torch.zeros(2, 2, 16, D, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, 2, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    kda.kv_append(none, none, kp, kp, table, i32(0), i32())
    assert kda.kv_read(kp, kp, table, i32(0), i32(), 0)[0].shape == (0, 2, D)
    assert kda.attn_prefill_paged(none, kp, kp, table, i32(0), i32()).shape == (0, 2, D)
    assert kda.attn_decode_paged(none[:, None], kp, kp, table, i32()).shape == (0, 1, 2, D)
