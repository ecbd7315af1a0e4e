"""The step between blocks on the GPU against its 64-bit statement (lin_util.block)."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from lin_util import U16, U32, block, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(T, W, wide, seed, parts):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = dict(x=r(T, W) * 3 if wide else (r(T, W) * 3).to(BF), weight=1 + 0.2 * r(W) if "w" in parts else None)
    if "y" in parts:
        a.update(y=r(T, W).to(BF), post_norm="n" in parts, post_weight=1 + 0.2 * r(W) if "p" in parts else None,
                 gate=(2 * r(T, W)).to(BF) if "g" in parts else None, scale=0.37 if "s" in parts else 1.0)
    return a


def run(a, **kw):
    c = lambda t: t.cuda() if isinstance(t, torch.Tensor) else t  # noqa: E731
    out = kda.block_norm(**{n: c(t) for n, t in a.items()}, **kw)
    torch.cuda.synchronize()
    return out


def verify(a, h, x, eps=1e-5):
    want_h, want_x, far_h, far_x = block(**a, eps=eps)
    check(h, want_h, far_h + U16 * (want_h.abs() + far_h), "h")
    if "y" in a:
        check(x, want_x, far_x + (U32 if a["x"].dtype == torch.float32 else U16) * (want_x.abs() + far_x), "x")


PARTS = ["", "w", "y", "wy", "wyn", "wynp", "wyp", "wyg", "wynpgs", "ygs", "ynps"]


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("wide", [False, True])
def test_parts(parts, wide):
    a = make(7, 520, wide, 3, parts)
    verify(a, *run(a))


@pytest.mark.parametrize("T,W", [(1, 8), (3, 16), (1, 248), (2, 256), (5, 264), (2, 4096), (1, 8192), (3, 8200), (2, 12288),
                                 (1, 16384), (2, 16392), (1, 32768), (1, 24), (700, 40), (5000, 512)])
@pytest.mark.parametrize("wide", [False, True])
def test_sizes(T, W, wide):
    a = make(T, W, wide, T + W, "wynpgs")
    verify(a, *run(a))


@pytest.mark.parametrize("T,W", [(640, 8), (700, 24), (1000, 264), (650, 1000), (1500, 1928), (650, 2056), (700, 4096), (650, 4104),
                                 (620, 6144), (640, 8192), (620, 8200), (610, 12288), (610, 12296), (609, 16384)])
@pytest.mark.parametrize("wide,parts", [(False, "wynpgs"), (True, "wynpgs"), (False, ""), (True, "wyp"), (False, "yn"), (True, "w")])
def test_many_rows(T, W, wide, parts):
    """Enough rows for blocks that walk over several: some of them against the statement, all against a call of few."""
    a = make(T, W, wide, T + W, parts)
    h, x = run(a)
    some = torch.cat([torch.arange(5), torch.randperm(T, generator=torch.Generator().manual_seed(1))[:20], torch.arange(T - 5, T)])
    few = {n: t[some] if isinstance(t, torch.Tensor) and t.dim() == 2 else t for n, t in a.items()}
    verify(few, h[some.cuda()], x[some.cuda()])
    assert bool(torch.isfinite(h).all()) and bool(torch.isfinite(x).all())
    rms = lambda t: t.float().square().mean(-1).sqrt()  # noqa: E731
    want, _ = run({n: t[:600] if isinstance(t, torch.Tensor) and t.dim() == 2 else t for n, t in a.items()})
    assert float((rms(h[:600]) - rms(want)).abs().max()) < 1e-3 and int((h[:600] != want).sum()) <= h.numel() // 1000


@pytest.mark.parametrize("wide", [False, True])
def test_many_strided_rows_in_place_and_bad_ones(wide):
    T, W = 900, 520
    a = make(T, W, wide, 5, "wynpgs")
    h0, x0 = run(a)

    def spread(t):
        b = torch.full((T, W + 24), float("nan"), dtype=t.dtype, device="cuda")
        b[:, 8:W + 8] = t.cuda()
        return b[:, 8:W + 8]

    h, x = run({n: spread(a[n]) if n in ("x", "y", "gate") else t for n, t in a.items()})
    assert torch.equal(h, h0) and torch.equal(x, x0)
    x = a["x"].cuda()
    h, x1 = run({**a, "x": x}, x_out=x)
    assert x1 is x and torch.equal(h, h0) and torch.equal(x, x0)
    bad = [0, 3, 500, 611, T - 1]
    a["y"][bad] = float("nan")
    h, x = run(a)
    same = torch.ones(T, dtype=torch.bool)
    same[bad] = False
    assert torch.equal(h[same.cuda()], h0[same.cuda()]) and torch.equal(x[same.cuda()], x0[same.cuda()])
    assert not bool(torch.isfinite(h[~same.cuda()]).any())


def test_no_rows():
    a = make(0, 64, False, 1, "wynpgs")
    h, x = run(a)
    assert h.shape == x.shape == (0, 64)


@pytest.mark.parametrize("wide", [False, True])
def test_strided_rows_and_in_place(wide):
    a = make(9, 136, wide, 5, "wynpgs")
    h0, x0 = run(a)

    def spread(t):
        b = torch.full((9, 136 + 24), float("nan"), dtype=t.dtype, device="cuda")
        b[:, 8:144] = t.cuda()
        return b[:, 8:144]

    h, x = run({n: spread(a[n]) if n in ("x", "y", "gate") else t for n, t in a.items()})
    assert torch.equal(h, h0) and torch.equal(x, x0)
    x = a["x"].cuda()
    h, x1 = run({**a, "x": x}, x_out=x)
    assert x1 is x and torch.equal(h, h0) and torch.equal(x, x0)


def test_rows_keep_to_themselves():
    """Rows of NaN, infinities and zeros; the others keep their bits."""
    a = make(40, 264, False, 6, "wynpg")
    h0, x0 = run(a)
    a["x"][3], a["y"][7, 5], a["gate"][9], a["x"][11] = float("nan"), float("inf"), float("nan"), 0.0
    a["y"][11] = 0.0
    h, x = run(a)
    same = torch.tensor([i not in (3, 7, 9, 11) for i in range(40)]).cuda()
    assert torch.equal(h[same], h0[same]) and torch.equal(x[same], x0[same])
    assert not bool(torch.isfinite(h[[3, 9]]).any()) and not bool(h[11].any()) and not bool(x[11].any())


def test_closed_and_open_gates():
    a = make(4, 64, True, 7, "wyg")
    a["gate"][0], a["gate"][1] = float("-inf"), float("inf")
    a["gate"][2], a["gate"][3] = -200.0, 200.0
    verify(a, *run(a))


@pytest.mark.parametrize("eps", [0.0, 1e-5, 3.0])
def test_eps(eps):
    a = make(5, 72, False, 8, "wynp")
    verify(a, *run(a, eps=eps), eps=eps)


def test_replayed_graph():
    a = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in make(50, 520, False, 9, "wynpgs").items()}
    want = kda.block_norm(**a)
    x = a["x"].clone()
    a["x"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.block_norm(**a)
    a["x"].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
