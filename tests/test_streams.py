"""Buffers that a call on a given stream makes for itself come out of that
stream's own memory: nothing orders the stream behind work that is still queued
on the caller's.  Without a GPU, on stand-ins for the library and torch's streams."""
import contextlib
import types

import pytest
import torch


class Stream:
    cuda_stream = 77


class Buffer:
    """A torch tensor that notes the streams it is recorded on."""

    def __init__(self, t):
        self.t, self.recorded = t, []

    def __getattr__(self, name):
        return getattr(self.t, name)

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.fixture
def world(monkeypatch):
    from bit_quantization_aware_amd import pq
    w = types.SimpleNamespace(pq=pq, current="the caller's", made=[], launched=[])

    @contextlib.contextmanager
    def on(s):
        before, w.current = w.current, s
        yield
        w.current = before
    empty = torch.empty

    def spy(*shape, device=None, **kw):
        b = Buffer(empty(*shape, **kw))
        w.made.append((w.current, b))
        return b

    def launch(*args):
        w.launched.append(args[-1])
        return 0
    size = lambda *a: 64  # noqa: E731
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: w.current)
    monkeypatch.setattr(pq, "lib", types.SimpleNamespace(
        pq_attn_decode=launch, pq_rope_table=launch, pq_gemm=launch, pq_w2a16_gemm=launch,
        pq_attn_decode_workspace_bytes=size, pq_gemm_workspace_bytes=size))
    w.spy = lambda: monkeypatch.setattr(torch, "empty", spy)
    return w


STREAMS = [(Stream(), 77), (77, 77)]


def owner(stream):
    return ("external", stream) if isinstance(stream, int) else stream


@pytest.mark.parametrize("stream,handle", STREAMS)
def test_attention_workspace(world, stream, handle):
    pq = world.pq
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    cache = pq.KVCache(pq.PQ_KV_16, 16, k, k.clone())
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    world.spy()
    pq.pq_attn_decode(cache, q, table, lens, q.clone(), stream=stream)
    assert [s for s, _ in world.made] == [owner(stream)] and world.launched == [handle]
    assert world.current == "the caller's"


@pytest.mark.parametrize("stream,handle", STREAMS)
def test_gemm_workspace(world, stream, handle):
    pq = world.pq
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    world.spy()
    pq.pq_w2a16_gemm(1, 64, 64, x, x, x, x, stream=stream)
    assert [s for s, _ in world.made] == [owner(stream)] and world.launched == [handle]


@pytest.mark.parametrize("stream,handle", STREAMS)
def test_rope_table(world, stream, handle):
    """The table is the caller's to use: it is also marked as used on the stream that the caller is on."""
    world.spy()
    table = world.pq.pq_rope_table(8, 64, stream=stream)
    (made_on, buffer), = world.made
    assert buffer is table and made_on == owner(stream) and world.launched == [handle]
    assert table.recorded == ["the caller's"]


@pytest.mark.gpu
def test_workspace_belongs_to_the_launch_stream():
    from bit_quantization_aware_amd import pq
    k, v = (torch.randn(200, 16, 1, 64, device="cuda").to(torch.bfloat16).transpose(1, 2) for _ in range(2))
    cache = pq.KVCache(pq.PQ_KV_16, 16, k, v)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    table, lens = torch.arange(200, dtype=torch.int32, device="cuda")[None], torch.tensor([3200], dtype=torch.int32, device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    pq.pq_attn_decode(cache, q, table, lens, want, workspace=pq.attn_workspace(cache, 1, 4))
    made, make = [], pq.attn_workspace

    def spy(*args):
        t = make(*args)
        made.append(t.data_ptr())
        return t
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with pytest.MonkeyPatch.context() as m:
        m.setattr(pq, "attn_workspace", spy)
        pq.pq_attn_decode(cache, q, table, lens, got, stream=side)
        pq.pq_attn_decode(cache, q, table, lens, got, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    segments = [s for s in torch.cuda.memory_snapshot() for p in made if s["address"] <= p < s["address"] + s["total_size"]]
    assert len(segments) == 2 and all(s["stream"] == side.cuda_stream for s in segments)
