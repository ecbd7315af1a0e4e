"""Linear attention with a decay a head on the GPU against the 64-bit statement, token by token (lin_util)."""
import math

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from lin_util import D, U16, check, decode_far, prefill_far, stage, stage_far, tokens

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CHECK = 7


def gen(seed):
    return torch.Generator().manual_seed(seed)


def unit(g, *shape):
    x = torch.randn(*shape, D, generator=g)
    return (x / x.norm(dim=-1, keepdim=True)).to(BF)


def decays(g, kind, *shape):
    x = torch.randn(*shape, generator=g)
    if kind == "mixed":      # memories from a token to thousands
        return -torch.exp(2.5 * x - 3)
    if kind == "strong":
        return -torch.exp(x + 2)
    if kind == "none":
        return torch.zeros(shape)
    if kind == "resets":     # now and then everything before a token is forgotten
        return torch.where(torch.rand(shape, generator=g) < 0.03, -math.inf, -torch.exp(x - 4))
    raise ValueError(kind)


class Prefill:
    def __init__(self, lens, H, Hk, seed, kind="mixed", entry=True, gated=False, scale=1.0, fixed=False, weight=True):
        g = gen(seed)
        T = sum(lens)
        self.lens, self.H = lens, H
        self.q, self.k, self.v = unit(g, T, Hk), unit(g, T, Hk), torch.randn(T, H, D, generator=g).to(BF)
        self.g = decays(g, kind, H) if fixed else decays(g, kind, T, H)
        self.S = 0.1 * torch.randn(len(lens), H, D, D, generator=g) if entry else None
        self.gate = torch.randn(T, H, D, generator=g).to(BF) if gated else None
        self.weight = 1 + 0.1 * torch.randn(D, generator=g) if gated and weight else None
        self.scale, self.eps = scale, 1e-5

    def cu(self):
        return torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).cuda()

    def args(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return (c(self.q), c(self.k), c(self.v), c(self.g), self.cu()), dict(
            S_in=c(self.S), scale=self.scale, gate=c(self.gate), norm_weight=c(self.weight), eps=self.eps)

    def run(self, **kw):
        a, b = self.args()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, S = kda.lin_prefill(*a, **{**b, **kw}, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == 0
        return o, S

    def check(self, o, S, heads=None):
        """Against the statement, on some heads where the whole is much."""
        heads = range(self.H) if heads is None else heads
        r, at = self.H // self.q.shape[1], 0
        for i, n in enumerate(self.lens):
            rows = slice(at, at + n)
            at += n
            for h in heads:
                one = slice(h, h + 1)
                q, k, v = self.q[rows, h // r:h // r + 1], self.k[rows, h // r:h // r + 1], self.v[rows, one]
                g = self.g[one].expand(n, 1) if self.g.dim() == 1 else self.g[rows, one]
                S0 = None if self.S is None else self.S[i, one]
                want, states = tokens(q, k, v, g, S0, self.scale)
                far, s_far = prefill_far(q, k, v, g, S0, self.scale)
                if self.gate is not None:
                    gate = self.gate[rows, one]
                    far = stage_far(want, far, gate, self.weight, self.eps)
                    want = stage(want, gate, self.weight, self.eps)
                check(o[rows, one], want, far + U16 * (want.abs() + far), f"o of sequence {i}, head {h}")
                check(S[i, one], states[-1], s_far, f"state of sequence {i}, head {h}")


@pytest.mark.parametrize("lens", [[1], [127], [128], [129], [256], [0, 1, 0, 300, 64, 0], [1] * 9, [513, 2, 130, 31, 65]])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2)])
def test_lengths(lens, H, Hk):
    p = Prefill(lens, H, Hk, seed=len(lens) + H)
    p.check(*p.run())


@pytest.mark.parametrize("kind", ["mixed", "strong", "none", "resets"])
@pytest.mark.parametrize("fixed", [False, True])
def test_decays(kind, fixed):
    p = Prefill([400, 77], 3, 1, seed=5, kind=kind, fixed=fixed)
    p.check(*p.run())


@pytest.mark.parametrize("entry", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("scale", [1.0, D ** -0.5, -0.3, 0.0])
def test_output_stage(entry, weight, scale):
    p = Prefill([200, 1, 150], 4, 4, seed=9, entry=entry, gated=True, scale=scale, weight=weight)
    p.check(*p.run())


@pytest.mark.parametrize("segments", [1, 2, 3, 7, 50])
def test_split(segments):
    p = Prefill([1100, 130, 0, 257, 128], 2, 1, seed=segments, scale=0.5)
    p.check(*p.run(n_segments=segments))


def test_split_by_the_library():
    """Few heads and a long sequence: split over the SMs without being asked; ragged neighbours."""
    p = Prefill([9000, 40, 5000], 2, 2, seed=3, scale=0.5)
    o, S = p.run()
    p.check(o, S)
    o1, S1 = p.run(n_segments=1)
    assert float((S - S1).norm() / S1.norm()) < 1e-4


@pytest.mark.parametrize("segments", [0, 3])
def test_states_in_place(segments):
    p = Prefill([700, 300, 0], 2, 1, seed=4)
    a, b = p.args()
    o, S = p.run(n_segments=segments)
    b["S_in"] = b["S_in"].clone()
    o2, S2 = kda.lin_prefill(*a, **b, S_out=b["S_in"], n_segments=segments)
    assert torch.equal(o, o2) and torch.equal(S, S2) and S2 is b["S_in"]


def test_rows_as_they_lie():
    """q, k, v and the gate in one projection's rows, g a column of another tensor."""
    p = Prefill([300, 45], 4, 2, seed=6, gated=True)
    T = 345
    wide = torch.full((T + 2, 14, D), float("nan"), dtype=BF)
    rows = wide[1:T + 1]
    rows[:, :2], rows[:, 2:4], rows[:, 5:9], rows[:, 10:14] = p.q, p.k, p.v, p.gate
    rows = rows.cuda()
    q, k, v, gate = rows[:, :2], rows[:, 2:4], rows[:, 5:9], rows[:, 10:14]
    g = torch.full((T, 9), float("nan"))
    g[:, 1::2] = p.g
    g = g.cuda()[:, 1::2]
    a, b = p.args()
    b["gate"] = gate
    o, S = kda.lin_prefill(q, k, v, g, a[4], **b)
    p.check(o, S)
    o1, S1 = p.run()
    assert torch.equal(o, o1) and torch.equal(S, S1)


@pytest.mark.parametrize("what", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("segments", [0, 2])
def test_what_is_not_finite_stays_where_it_belongs(what, value, segments):
    """One bad value in the middle of a chunk: earlier tokens, other heads and other sequences keep their bits."""
    if what == "g" and value > 0:
        value = float("nan")
    p = Prefill([300, 300, 200], 2, 2, seed=8)
    o0, S0 = p.run(n_segments=segments)
    t, h = 300 + 170, 1
    if what == "g":
        p.g[t, h] = value
    else:
        getattr(p, what)[t, h, 5] = value
    o, S = p.run(n_segments=segments)
    same = torch.ones(800, 2, dtype=torch.bool)
    if what == "q":
        same[t, h] = False
    else:
        same[t:600, h] = False
    assert torch.equal(o[same.cuda()], o0[same.cuda()])
    bad = ~torch.isfinite(o).all(-1).cpu()
    if what == "v":  # one channel
        assert bool((~torch.isfinite(o[t:600, h, 5])).all())
        rest = torch.arange(D) != 5
        rest = rest.cuda()
        assert torch.equal(o[:, :, rest], o0[:, :, rest]) and torch.equal(S[:, :, :, rest], S0[:, :, :, rest])
    elif what != "k":
        assert torch.equal(bad, ~same)
    else:
        assert bool(bad[t, h])
    assert torch.equal(S[0], S0[0]) and torch.equal(S[2], S0[2]) and torch.equal(S[1, 0], S0[1, 0])
    assert torch.equal(S[1, 1], S0[1, 1]) if what == "q" else not bool(torch.isfinite(S[1, 1]).all())


@pytest.mark.parametrize("channel", [3, 70])
def test_a_bad_value_takes_its_whole_row_through_the_output_stage(channel):
    """The row's root mean square is not finite then, whichever warps have the channel."""
    p = Prefill([300, 257], 12, 4, seed=9, gated=True)
    o0, S0 = p.run()
    t = [20 * h + 9 for h in range(12)]
    for h in range(12):
        p.v[t[h], h, channel] = float("nan") if h % 2 else float("inf")
    o, S = p.run()
    for h in range(12):
        assert torch.equal(o[:t[h], h], o0[:t[h], h]) and torch.equal(o[300:, h], o0[300:, h])
        assert not bool(torch.isfinite(o[t[h]:300, h]).any())
    rest = torch.arange(D, device="cuda") != channel
    assert torch.equal(S[:, :, :, rest], S0[:, :, :, rest]) and not bool(torch.isfinite(S[0, :, :, channel]).any())


def test_neighbours_and_rows_outside_do_not_reach_a_sequence():
    """The tail of a chunk holds the next sequence's rows, here NaN; another sequence is all infinities."""
    p = Prefill([130, 140, 90], 2, 1, seed=12)
    o0, S0 = p.run()
    p.q[130:270], p.k[130:270], p.v[130:270], p.g[130:270] = float("nan"), float("inf"), float("nan"), float("nan")
    o, S = p.run()
    for a, b in ((o, o0),):
        assert torch.equal(a[:130], b[:130]) and torch.equal(a[270:], b[270:])
    assert torch.equal(S[0], S0[0]) and torch.equal(S[2], S0[2])


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, 50, 101, 100], [0, -5, 60, 100]])
def test_bad_offsets_write_nothing(cu):
    p = Prefill([50, 10, 40], 2, 1, seed=2)
    a, b = p.args()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = torch.full((100, 2, D), 7.0, dtype=BF, device="cuda"), torch.full((3, 2, D, D), 7.0, device="cuda")
    kda.lin_prefill(*a[:4], torch.tensor(cu, dtype=torch.int32, device="cuda"), **b, o=o, S_out=S, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == CHECK
    assert bool((o == 7).all()) and bool((S == 7).all())


@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("gated", [False, True])
def test_a_block_each_and_a_plan(H, gated):
    """As many (sequence, head) pairs as there are blocks, and more: sequences without tokens, a bad value, the state
    in place, and offsets that are wrong."""
    p = Prefill([130, 0, 70, 0, 1, 257], H, 4, seed=51, gated=gated)
    size = kda.lin_prefill_workspace_size(6, H, 458)
    assert (size > 0) == (6 * H > torch.cuda.get_device_properties(0).multi_processor_count)
    o, S = p.run()
    p.check(o, S, heads=(0, H - 1))
    assert torch.equal(S[1].cpu(), p.S[1]) and torch.equal(S[3].cpu(), p.S[3])
    states = p.S.cuda()
    o1, S1 = p.run(S_in=states, S_out=states)
    assert S1 is states and torch.equal(o, o1) and torch.equal(S, S1)
    o1, S1 = p.run(S_in=None)
    assert not bool(S1[1].any()) and not bool(S1[3].any())
    p.v[130 + 40, H - 1, 9] = float("nan")
    o1, S1 = p.run()
    bad = torch.zeros(458, H, dtype=torch.bool)
    bad[170:200, H - 1] = True
    assert torch.equal(o1[~bad], o[~bad]) and bool(o1[bad][:, 9].isnan().all())
    assert bool(o1[bad].isnan().all()) == gated
    assert bool(S1[2, H - 1, :, 9].isnan().all()) and torch.equal(S1[5], S[5])
    a, b = p.args()
    for i, wrong in ((2, 129), (6, 457), (0, 1), (4, 10 ** 9)):
        cu = a[4].clone()
        cu[i] = wrong
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        keep = [torch.full_like(t, 7) for t in (o, S)]
        kda.lin_prefill(*a[:4], cu, **b, o=keep[0], S_out=keep[1], dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == CHECK and bool((keep[0] == 7).all()) and bool((keep[1] == 7).all())


@pytest.mark.parametrize("n", [0, 3])
def test_no_tokens(n):
    S0 = torch.randn(n, 2, D, D, device="cuda")
    e = torch.empty(0, 2, D, dtype=BF, device="cuda")
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    o, S = kda.lin_prefill(e, e, e, torch.empty(0, 2, device="cuda"), cu, S_in=S0)
    assert o.shape == (0, 2, D) and torch.equal(S, S0)
    _, S = kda.lin_prefill(e, e, e, torch.empty(0, 2, device="cuda"), cu)
    assert not bool(S.any())


def test_chunks_of_a_prompt_equal_the_prompt():
    """Sequences in two calls, the second from the first's states."""
    p = Prefill([500, 260], 2, 1, seed=21, scale=0.2)
    a, b = p.args()
    cut = [300, 128]
    first = torch.cat([torch.arange(0, 300), torch.arange(500, 628)]).cuda()
    second = torch.cat([torch.arange(300, 500), torch.arange(628, 760)]).cuda()
    cu = lambda lens: torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()  # noqa: E731
    o = torch.empty(760, 2, D, dtype=BF, device="cuda")
    o[first], S = kda.lin_prefill(*(t[first] for t in a[:4]), cu(cut), **b)
    o[second], S = kda.lin_prefill(*(t[second] for t in a[:4]), cu([200, 132]), **{**b, "S_in": S})
    p.check(o, S)


def test_many_short_sequences():
    lens = [i % 7 for i in range(700)]
    p = Prefill(lens, 1, 1, seed=31)
    p.check(*p.run())


@pytest.mark.parametrize("segments", [0, 4])
def test_replayed_graph_and_two_streams(segments):
    """A captured call replayed on other inputs, and calls on two streams at once with workspaces of their own."""
    p = Prefill([600, 90], 2, 1, seed=41)
    a, b = p.args()
    want = kda.lin_prefill(*a, **b, n_segments=segments)
    keep = [t.clone() for t in a[:4]]
    for t in a[:4]:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.lin_prefill(*a, **b, n_segments=segments)
    for t, x in zip(a[:4], keep):
        t.copy_(x)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [kda.lin_prefill(*a, **b, n_segments=segments, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(S, want[1]) for o, S in outs)


# ------------------------------------------------------------------------------------- decode
class Step:
    def __init__(self, B, n, H, Hk, seed, kind="mixed", gated=False, scale=1.0, fixed=False):
        g = gen(seed)
        self.q, self.k, self.v = unit(g, B, n, Hk), unit(g, B, n, Hk), torch.randn(B, n, H, D, generator=g).to(BF)
        self.g = decays(g, kind, H) if fixed else decays(g, kind, B, n, H)
        self.S = 0.1 * torch.randn(B, H, D, D, generator=g)
        self.gate = torch.randn(B, n, H, D, generator=g).to(BF) if gated else None
        self.weight = 1 + 0.1 * torch.randn(D, generator=g) if gated else None
        self.scale, self.eps = scale, 1e-5

    def run(self, n_commit=None, **kw):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        S = self.S.cuda()
        commit = None if n_commit is None else torch.tensor(n_commit, dtype=torch.int32, device="cuda")
        args = {**dict(q=c(self.q), k=c(self.k), v=c(self.v), g=c(self.g), gate=c(self.gate)), **kw}
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = kda.lin_decode(args["q"], args["k"], args["v"], args["g"], S, n_commit=commit, scale=self.scale,
                           gate=args["gate"], norm_weight=c(self.weight), eps=self.eps, dev_status=st)
        torch.cuda.synchronize()
        return o, S, int(st)

    def check(self, o, S, n_commit=None):
        B, n, H = self.v.shape[:3]
        for b in range(B):
            g = self.g.expand(n, H) if self.g.dim() == 1 else self.g[b]
            want, states = tokens(self.q[b], self.k[b], self.v[b], g, self.S[b], self.scale)
            far, s_far = decode_far(self.q[b], self.k[b], self.v[b], g, self.S[b], self.scale)
            if self.gate is not None:
                far = stage_far(want, far, self.gate[b], self.weight, self.eps)
                want = stage(want, self.gate[b], self.weight, self.eps)
            check(o[b], want, far, f"o of sequence {b}")
            m = n if n_commit is None else n_commit[b]
            check(S[b], states[m], s_far[m], f"state of sequence {b}")


@pytest.mark.parametrize("n", [1, 2, 3, 4])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2)])
@pytest.mark.parametrize("gated", [False, True])
def test_decode(n, H, Hk, gated):
    s = Step(5, n, H, Hk, seed=n, gated=gated, scale=0.3)
    o, S, st = s.run()
    assert st == 0
    s.check(o, S)
    commit = [0, n, 1, max(0, n - 1), n]
    o2, S2, st = s.run(commit)
    assert st == 0 and torch.equal(o, o2)
    s.check(o2, S2, commit)
    assert torch.equal(S2[0].cpu(), s.S[0])


@pytest.mark.parametrize("kind", ["mixed", "strong", "none", "resets"])
@pytest.mark.parametrize("fixed", [False, True])
def test_decode_decays(kind, fixed):
    s = Step(3, 4, 40, 8, seed=3, kind=kind, fixed=fixed)
    o, S, st = s.run()
    assert st == 0
    s.check(o, S)


def test_decode_rows_as_they_lie():
    s = Step(3, 2, 4, 2, seed=7, gated=True)
    wide = torch.full((3, 3, 13, D), float("nan"), dtype=BF)
    wide[:, 1:, :2], wide[:, 1:, 2:4], wide[:, 1:, 4:8], wide[:, 1:, 9:13] = s.q, s.k, s.v, s.gate
    wide = wide.cuda()[:, 1:]
    g = torch.zeros(3, 5, 4)
    g[:, :2] = s.g
    o, S, st = s.run(q=wide[:, :, :2], k=wide[:, :, 2:4], v=wide[:, :, 4:8], gate=wide[:, :, 9:13], g=g.cuda()[:, :2])
    assert st == 0
    s.check(o, S)


def test_decode_accepted_tokens_out_of_range():
    s = Step(3, 2, 2, 1, seed=7)
    o, S, st = s.run([2, 3, -1])
    assert st == CHECK
    s.check(o, S, [2, 0, 0])
    assert torch.equal(S[1:].cpu(), s.S[1:])


def test_decode_rejected_tokens_do_not_reach_the_state():
    s = Step(2, 4, 2, 2, seed=17)
    o0, S0, _ = s.run([2, 2])
    for t in (s.q, s.k, s.v, s.g):
        t[:, 2:] = float("nan")
    o, S, _ = s.run([2, 2])
    assert torch.equal(S, S0) and torch.equal(o[:, :2], o0[:, :2])


def test_prompt_then_tokens():
    """A prompt by chunks and the rest token by token equal the whole sequence."""
    p = Prefill([140], 3, 1, seed=51)
    a, b = p.args()
    q, k, v, g = a[:4]
    cu = torch.tensor([0, 131], dtype=torch.int32, device="cuda")
    _, S = kda.lin_prefill(q[:131], k[:131], v[:131], g[:131], cu, S_in=b["S_in"])
    outs = []
    for lo, hi in ((131, 132), (132, 136), (136, 138), (138, 140)):
        outs.append(kda.lin_decode(*(t[None, lo:hi] for t in (q, k, v, g)), S)[0])
    want, states = tokens(p.q, p.k, p.v, p.g, p.S[0])
    far, s_far = prefill_far(p.q, p.k, p.v, p.g, p.S[0], 1.0)
    check(torch.cat(outs), want[131:], far[131:], "o")
    check(S[0], states[-1], s_far, "state")
