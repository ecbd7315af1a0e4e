"""Decode steps of linear attention with more (sequence, head) pairs than SMs, whose blocks fetch a later pair's state and
rows ahead; captured and replayed steps; steps on two streams."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from test_lin_gpu import BF, D, Step

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("n", [1, 2, 3, 4])
@pytest.mark.parametrize("gated,fixed", [(False, True), (True, False)])
def test_more_pairs_than_sms(n, gated, fixed):
    s = Step(6, n, 64, 16, seed=20 + n, gated=gated, fixed=fixed, scale=0.3)
    commit = [n, 0, 1, n, max(0, n - 1), n]
    assert s.S.shape[0] * s.S.shape[1] > 2 * sms()
    o, S, st = s.run(commit)
    assert st == 0
    s.check(o, S, commit)
    assert torch.equal(S[1].cpu(), s.S[1])


@pytest.mark.parametrize("over", [0, 1, 2])
def test_as_many_pairs_as_sms_and_one_more(over):
    s = Step(sms() + over, 2, 1, 1, seed=over, gated=True)
    o, S, st = s.run()
    assert st == 0
    s.check(o, S)


def test_many_pairs_of_rows_as_they_lie():
    """Rows of a wider projection: what is fetched ahead lies between rows of NaN, as the rest does."""
    s = Step(7, 3, 48, 12, seed=8, gated=True)
    wide = torch.full((7, 4, 130, D), float("nan"), dtype=BF)
    wide[:, 1:, :12], wide[:, 1:, 13:25], wide[:, 1:, 26:74], wide[:, 1:, 80:128] = s.q, s.k, s.v, s.gate
    wide = wide.cuda()[:, 1:]
    o, S, st = s.run(q=wide[:, :, :12], k=wide[:, :, 13:25], v=wide[:, :, 26:74], gate=wide[:, :, 80:128])
    assert st == 0
    s.check(o, S)


def arguments(s):
    rows = [t.cuda() for t in (s.q, s.k, s.v, s.g)]
    return rows, dict(scale=s.scale, gate=s.gate.cuda(), norm_weight=s.weight.cuda(), eps=s.eps)


def test_replayed_graph():
    """Two replays are two steps; the second on other rows and other accepted tokens."""
    s = Step(5, 4, 40, 8, seed=31, gated=True)
    rows, kw = arguments(s)
    commits = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([4, 0, 2, 1, 3], [1, 4, 0, 4, 2])]
    others = [rows, [t.flip(0) for t in rows]]
    S, want = s.S.cuda(), []
    for r, c in zip(others, commits):
        want.append((kda.lin_decode(*r, S, n_commit=c, **kw), S.clone()))
    held, commit, S = [torch.zeros_like(t) for t in rows], torch.zeros_like(commits[0]), s.S.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.lin_decode(*held, S, n_commit=commit, **kw)
    for r, c, (o, after) in zip(others, commits, want):
        for t, x in zip(held, r):
            t.copy_(x)
        commit.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, o) and torch.equal(S, after)


def test_two_streams():
    """Two batches, three steps each, at once."""
    steps = [Step(4, 2, 60, 6, seed=41 + i, gated=True) for i in range(2)]
    args = [arguments(s) for s in steps]
    want = []
    for s, (rows, kw) in zip(steps, args):
        S = s.S.cuda()
        want.append(([kda.lin_decode(*rows, S, **kw) for _ in range(3)], S))
    states, got = [s.S.cuda() for s in steps], [[], []]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (rows, kw) in enumerate(args):
            got[i].append(kda.lin_decode(*rows, states[i], **kw, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (outs, S) in enumerate(want):
        assert all(torch.equal(a, b) for a, b in zip(got[i], outs)) and torch.equal(states[i], S)
