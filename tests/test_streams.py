"""Tensors that a call of the binding makes belong to the stream that the call runs on.  A workspace
made on the current stream and dropped when the call returns would go to the next allocation of that
stream while the kernels on the other still use it.

The library and the stream are stand-ins here, so that no kernel runs (no GPU needed); the GPU test
looks at the addresses that the library gets."""
import contextlib

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Device(torch.Tensor):
    """A host tensor that passes for a device tensor."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        NOTES.append(("kept for", stream))


class Stream:
    cuda_stream = 7777
    device = torch.device("cpu")


class Library:
    """Takes any call; sizes are 512 bytes."""

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 512
        return lambda *a: 0


NOTES = []


@pytest.fixture
def fakes(monkeypatch):
    """Notes every tensor made during a call: (inside the stream's context or not)."""
    here = []
    made = torch.empty

    @contextlib.contextmanager
    def on(stream):
        here.append(stream)
        yield
        here.pop()

    def empty(*a, **kw):
        NOTES.append(("made on", here[-1] if here else None))
        return made(*a, **kw).as_subclass(Device)

    NOTES.clear()
    lib = Library()
    monkeypatch.setattr(kda, "_lib", lib)
    monkeypatch.setattr(kda, "library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch, "empty", empty)


def dev(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(Device)


def calls():
    rows, gates = [dev(5, 2, 128) for _ in range(3)], [dev(5, 2, 128, dtype=F32), dev(5, 2, dtype=F32)]
    step = [t.unsqueeze(0)[:, :4] for t in rows + gates]
    cu, table = dev(2, dtype=I32), dev(1, 4, dtype=I32)
    pool = dev(8, 2, 16, 128)
    states = dev(1, 2, 128, 128, dtype=F32)
    pages = dev(2, dtype=I32)
    cache = (pool, pool, table)
    return {
        "prefill": lambda s: kda.prefill(*rows, *gates, cu, stream=s),
        "prefill_paged": lambda s: kda.prefill_paged(*rows, *gates, cu, states[0], stream=s),
        "prefill_noalloc": lambda s: kda.prefill_noalloc(*rows, *gates, cu, stream=s),
        "prefill_pairs": lambda s: kda.prefill_pairs(*rows, *gates, cu, stream=s),
        "combine_pairs": lambda s: kda.combine_pairs(states[None], states[None], stream=s),
        "decode": lambda s: kda.decode(*step, states, stream=s),
        "decode_paged": lambda s: kda.decode_paged(*step, states[0], pages, stream=s),
        "kv_read": lambda s: kda.kv_read(*cache, cu, dev(1, dtype=I32), 5, stream=s),
        "attn_prefill_paged": lambda s: kda.attn_prefill_paged(rows[0], *cache, cu, dev(1, dtype=I32), return_lse=True, stream=s),
        "attn_decode_paged": lambda s: kda.attn_decode_paged(step[0], *cache, dev(1, dtype=I32), return_lse=True, stream=s),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_made_on_the_call_s_stream(fakes, name):
    s = Stream()
    calls()[name](s)
    made = [n for n in NOTES if n[0] == "made on"]
    assert made and all(n[1] is s for n in made), made
    outputs = len(made) - (name in ("prefill", "prefill_paged", "decode_paged", "attn_prefill_paged", "attn_decode_paged"))
    # the caller's stream reads the outputs: their memory waits for it too
    assert NOTES.count(("kept for", "current")) == outputs


@pytest.mark.gpu
def test_workspaces_of_two_streams_are_apart(monkeypatch):
    """Calls on another stream, and the current stream's next allocations, do not share memory."""
    lib, seen = kda.library(), []

    class Spy:
        def __getattr__(self, name):
            f = getattr(lib, name)
            if name not in ("kda_attn_prefill_paged", "kda_attn_decode_paged"):
                return f
            return lambda *a: (seen.append((a[-4], a[-3])), f(*a))[1]  # workspace, bytes

    monkeypatch.setattr(kda, "_lib", Spy())
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)
    q, pool = rnd(300, 8, 128), rnd(2, 64, 2, 64, 128)
    table = torch.arange(64, dtype=I32, device="cuda")[None]
    cu, kv = torch.tensor([0, 300], dtype=I32, device="cuda"), torch.tensor([4000], dtype=I32, device="cuda")
    step = q[:1, None].contiguous()
    want = kda.attn_prefill_paged(q, *pool, table, cu, kv), kda.attn_decode_paged(step, *pool, table, kv)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i, call in enumerate((lambda **kw: kda.attn_prefill_paged(q, *pool, table, cu, kv, **kw),
                              lambda **kw: kda.attn_decode_paged(step, *pool, table, kv, **kw))):
        for _ in range(3):
            o = call(stream=s)
            at, n = seen[-1]
            held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]  # what the freed memory would go to
            assert all(t.data_ptr() + n <= at or at + n <= t.data_ptr() for t in held)
            o2 = call()
            assert seen[-1][0] != at
            torch.cuda.synchronize()
            assert torch.equal(o, want[i]) and torch.equal(o2, want[i])


@pytest.mark.gpu
def test_capture_with_the_stream_given():
    """A call captured into a graph with its stream named makes its tensors in the graph's memory."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)
    q, pool = rnd(300, 8, 128), rnd(2, 64, 2, 64, 128)
    table = torch.arange(64, dtype=I32, device="cuda")[None]
    cu, kv = torch.tensor([0, 300], dtype=I32, device="cuda"), torch.tensor([4000], dtype=I32, device="cuda")
    want = kda.attn_prefill_paged(q, *pool, table, cu, kv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = kda.attn_prefill_paged(q, *pool, table, cu, kv, stream=torch.cuda.current_stream())
        k, v = kda.kv_read(*pool, table, cu, kv - 300, 300, stream=torch.cuda.current_stream())
    for _ in range(2):
        held = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(k, pool[0].transpose(1, 2).reshape(-1, 2, 128)[3700:4000])
        del held
