"""Weights of linear attention's prefill where the decays in front of them are deep: the sums of a chunk's decays run
into the thousands, the differences that matter stay small.  Values alternate, so that what is near cancels and an
error of the weights is not hidden by the rounding of o."""
import math

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from lin_util import D, GROUP, U16, U32, check, stage, stage_far, tokens
from test_lin_gpu import gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# What a weight may be off by, relative: 2^-17 by its two bf16 parts (half a step of what the first leaves of it) and half as
# much for a sum of 128 products of two parts in 32 bits; its exponent, with up to 64 whole factors of 2 in it, by a rounding of the sum
# (64 x 2^-24) and of two parts (2^-24); exponentials and products by 2^-21; the score's 128 products by 2^-17.
WEIGHT = 2.0 ** -17 + 2.0 ** -18 + math.log(2) * 65 * U32 + 2.0 ** -21 + 2.0 ** -17


def inputs(n, H, decays, seed, spread=0.02):
    """Keys and queries all near one direction; values near alternating copies of one row."""
    g = gen(seed)
    near = lambda x: torch.nn.functional.normalize(x + spread * torch.randn(n, H, D, generator=g), dim=-1).to(BF)  # noqa: E731
    base = torch.nn.functional.normalize(torch.randn(1, H, D, generator=g), dim=-1)
    v = torch.randn(1, H, D, generator=g) * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)[:, None, None]
    slow = -torch.rand(n, H, generator=g) * 0.01
    return near(base), near(base), (v + 0.001 * torch.randn(n, H, D, generator=g)).to(BF), decays(slow, g)


def first(m, by):
    def f(slow, g):
        slow[:m] = by
        return slow
    return f


def mixed(p, by):
    def f(slow, g):
        return torch.where(torch.rand(slow.shape, generator=g) < p, by, slow)
    return f


CASES = [("first 8 reset", first(8, -math.inf)), ("first 64 reset", first(64, -math.inf)), ("first 90 reset", first(90, -math.inf)),
         ("first 120 reset", first(120, -math.inf)), ("first 100 at -80", first(100, -80.0)), ("a third reset", mixed(0.33, -math.inf)),
         ("two thirds reset", mixed(0.67, -math.inf)), ("a tenth at -100", mixed(0.1, -100.0)), ("a third at -2", mixed(0.33, -2.0))]


def far(q, k, v, g):
    A, _ = tokens(q.abs(), k.abs(), v.abs(), g)
    return WEIGHT * A


@pytest.mark.parametrize("name,decays", CASES)
@pytest.mark.parametrize("gated", [False, True])
def test_weights_after_deep_decays(name, decays, gated):
    """One chunk from zeros: nothing but the weights stands between the inputs and o."""
    n, H = GROUP, 4
    q, k, v, g = inputs(n, H, decays, len(name))
    gate = torch.randn(n, H, D, generator=gen(1)).to(BF) if gated else None
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, _ = kda.lin_prefill(q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu, gate=gate.cuda() if gated else None)
    torch.cuda.synchronize()
    want, _ = tokens(q, k, v, g)
    off = far(q, k, v, g)
    if gated:
        off, want = stage_far(want, off, gate, None, 1e-5), stage(want, gate, None, 1e-5)
    check(o, want, off + U16 * (want.abs() + off), "o")


@pytest.mark.parametrize("segments", [1, 3])
def test_later_chunks_and_sequences(segments):
    """Each chunk begins with a reset, so that the rounded state in front of it is not in any output; ragged."""
    lens, H = [384, 131, 300], 4
    parts = [inputs(n, H, mixed(0.3, -math.inf), 70 + n) for n in lens]
    for x in parts:
        x[3][::GROUP] = -math.inf
    q, k, v, g = (torch.cat([x[i] for x in parts]).cuda() for i in range(4))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o, _ = kda.lin_prefill(q, k, v, g, cu, n_segments=segments)
    torch.cuda.synchronize()
    for got, x in zip(o.split(lens), parts):
        want, off = tokens(*x)[0], far(*x)
        check(got, want, off + U16 * (want.abs() + off), "o")
