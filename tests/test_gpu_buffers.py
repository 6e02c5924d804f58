"""The buffers that the blocks keep between calls, on more than one stream: what a longer call drops is not handed out again
while kernels on another stream than the buffers' own still use it."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in tensors if t.numel() > 0]


def apart(taken, tensors):
    return all(hi <= a or b <= lo for a, b in taken for lo, hi in spans(tensors))


def test_feed_forward_grows_on_another_stream():
    from test_gpu_feed_forward import build, rows_of
    block, _ = build(512, 1408)
    x, long = rows_of(40, 512, 1), rows_of(300, 512, 2)
    first, second, y = torch.empty_like(x), torch.empty_like(x), torch.empty_like(long)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        block(x, first)
    old = block._shared
    sizes, taken = [(t.shape, t.dtype) for t in old.values()], spans(old.values())
    del old
    b.wait_stream(a)
    with torch.cuda.stream(b):
        torch.cuda._sleep(100_000_000)          # the call behind it has not begun when the buffers are dropped
        block(x, second)
        block(long, y)
        done = b.record_event()
    with torch.cuda.stream(a):
        new = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes * 3]
        for t in new:
            t.view(torch.uint8).fill_(0xFF)
    assert not done.query(), "the second stream was done before anything was made on the first"
    assert apart(taken, new)
    torch.cuda.synchronize()
    assert torch.equal(first, second)
    again = torch.empty_like(y)
    block(long, again)
    torch.cuda.synchronize()
    assert torch.equal(y, again)


def test_prompts_grow_on_another_stream():
    from test_gpu_decode_block import HIDDEN, build, rand
    g = torch.Generator().manual_seed(3)
    requests = 3
    blocks = [build(requests, torch.Generator().manual_seed(4)) for _ in range(2)]
    for b in blocks:
        b.ids.copy_(torch.tensor([0, -1, 2]))
    batches = [(rand(g, sum(n), HIDDEN), torch.tensor(n, dtype=torch.int32, device="cuda")) for n in ([9, 3, 0], [2, 0, 10], [300, 40, 7])]
    # what the caches hold when nothing is dropped while it is in use
    for x, fresh in batches:
        blocks[1].admit(x, fresh)
        torch.cuda.synchronize()
    block = blocks[0]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        block.admit(*batches[0])
    sizes, taken = [(t.shape, t.dtype) for t in block._prompts.values()], spans(block._prompts.values())
    b.wait_stream(a)
    with torch.cuda.stream(b):
        torch.cuda._sleep(100_000_000)
        block.admit(*batches[1])
        block.admit(*batches[2])
        done = b.record_event()
    with torch.cuda.stream(a):
        new = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes * 3]
        for t in new:
            t.view(torch.uint8).fill_(0xFF)
    assert not done.query(), "the second stream was done before anything was made on the first"
    assert apart(taken, new)
    torch.cuda.synchronize()
    for n in ("cached", "table", "k_cache", "v_cache"):
        assert torch.equal(getattr(blocks[0], n), getattr(blocks[1], n)), n
