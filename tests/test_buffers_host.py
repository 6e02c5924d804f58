"""CPU tests of the buffers that the blocks keep between calls: every stream that used a set is told to the allocator before
the set is dropped for a larger one, or memory that kernels on that stream still use would be handed out again.  The streams
here are stand-ins; nothing is launched."""
import numpy as np
import pytest

pytest.importorskip("dl_fusion_amd", reason="libdlfusion.so not built")
torch = pytest.importorskip("torch")


class Streams:
    """The current stream's handle, and which streams each tensor was recorded on."""

    def __init__(self, monkeypatch):
        self.now, self.seen, self.capturing = 1, {}, False
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: self.now)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda _: self.now, raising=False)
        monkeypatch.setattr(torch.Tensor, "is_cuda", True)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.seen.setdefault(t.data_ptr(), set()).add(s))

    def on(self, tensors):
        """The streams that all of the tensors with any bytes were recorded on."""
        return set.intersection(*(self.seen.get(t.data_ptr(), set()) for t in tensors if t.numel() > 0))


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


def feed_forward(rows=0):
    from dl_fusion_amd.feed_forward import GatedFeedForward, pack, pack_gate_up
    r = np.random.RandomState(0)
    w = [r.randn(*s).astype(np.float32) for s in ((288, 256), (288, 256), (256, 288))]
    return GatedFeedForward(pack_gate_up(w[0], w[1], "cpu"), pack(w[2], "cpu"), rows=rows)


NAMES = ("x", "x_scale", "h", "q", "q_scale", "ws")


def test_feed_forward_buffers_are_recorded_on_every_stream_that_uses_them(streams):
    block = feed_forward()
    first = block._buffers(8)
    old = [first[n] for n in NAMES]                 # kept, so that no other tensor gets their addresses
    streams.now = 2
    again = block._buffers(8)
    assert [again[n].data_ptr() for n in NAMES] == [t.data_ptr() for t in old]
    assert 2 in streams.on(old)
    streams.now = 3
    assert block._buffers(5)["x"].data_ptr() == old[0].data_ptr()
    grown = block._buffers(64)
    assert {2, 3} <= streams.on(old)
    assert grown["x"].data_ptr() != old[0].data_ptr()
    assert 3 in streams.on([grown[n] for n in NAMES])
    # a stream has to be told of the new set too
    streams.now = 2
    assert {2, 3} <= streams.on([block._buffers(64)[n] for n in NAMES])


def test_feed_forward_buffers_of_its_own_are_recorded_too(streams):
    block = feed_forward(rows=8)
    for streams.now in (4, 5):
        own = block._buffers(8)
    assert {4, 5} <= streams.on([own[n] for n in NAMES])


def attention(requests=4):
    from dl_fusion_amd.decode import PagedAttentionBlock
    heads, kv, dim, hidden, rank = 4, 2, 64, 256, 16
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    width = (heads + 2 * kv) * dim
    return PagedAttentionBlock(bf(width, hidden), bf(hidden, heads * dim), heads, kv, dim, requests, 16, 16, 4,
                               (bf(2, rank, hidden), bf(2, width, rank), None), norm=(None, 1e-5))


def test_prompts_buffers_of_an_attention_block_are_recorded_on_every_stream_that_uses_them(streams):
    block = attention()
    names = ("slots", "rows", "qkv", "normed", "lora_ws")
    old = [block._buffers(9)[n] for n in names]
    for streams.now in (2, 3):
        assert [block._buffers(9)[n].data_ptr() for n in names] == [t.data_ptr() for t in old]
    grown = block._buffers(3000)
    assert {2, 3} <= streams.on(old)
    assert grown["qkv"].data_ptr() != old[2].data_ptr()
    assert 3 in streams.on([grown[n] for n in names])


def test_step_buffers_of_an_attention_block_are_recorded_too(streams):
    block = attention()
    for streams.now in (4, 5):
        own = block._buffers(4)
    assert {4, 5} <= streams.on([own[n] for n in ("slots", "rows", "qkv", "normed")])
