"""The gated feed-forward block on 8-bit weights (dl_fusion_amd/feed_forward.py), and the norm before an attention block's
projection (dl_fusion_amd/decode.py): the operators run together, against their definitions in 64 bits and captured in a
graph.

Each stage is checked from the stage before it as the device has it, with the bounds that the operators' own tests derive
(test_gpu_row_blocks.py, test_gpu_gemm_blocks.py)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from test_gpu_gemm_blocks import definition, within  # noqa: E402
from test_gpu_row_blocks import check_blocks  # noqa: E402
from test_gpu_row_blocks import definition as norm_definition  # noqa: E402

U = 2.0 ** -24
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def build(d_model, d_ff, rows=0, gate="silu", norm=True, seed=1):
    from dl_fusion_amd.feed_forward import GatedFeedForward, pack, pack_gate_up
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn(*s, generator=g) * s[1] ** -0.5 for s in ((d_ff, d_model), (d_ff, d_model), (d_model, d_ff))]
    weight = (torch.randn(d_model, generator=g) * 0.2 + 1).cuda() if norm else None
    return GatedFeedForward(pack_gate_up(w[0].numpy(), w[1].numpy()), pack(w[2].numpy()), weight, gate=gate, rows=rows), w


def rows_of(m, d_model, seed):
    return (torch.randn(m, d_model, generator=torch.Generator().manual_seed(seed)) * 3).bfloat16().cuda()


@pytest.mark.parametrize("m,d_model,d_ff,gate,norm", [(1, 256, 512, "silu", True), (37, 768, 1280, "silu", False),
                                                      (64, 1024, 2816, "gelu_tanh", True), (300, 512, 400, "gelu_erf", True)])
def test_stage_by_stage(m, d_model, d_ff, gate, norm):
    block, w = build(d_model, d_ff, gate=gate, norm=norm)
    x = rows_of(m, d_model, 2)
    y = torch.empty_like(x)
    block(x, y)
    torch.cuda.synchronize()
    b = block._buffers(m)
    blocks = lambda k: -(-k // 128)  # noqa: E731
    _, want = norm_definition(x.cpu(), None, None if block.norm is None else block.norm.cpu(), block.eps)
    check_blocks(want, b["x"].cpu(), b["x_scale"][:, :blocks(d_model)].cpu(), (d_model / 128 + 29) * U)
    s = dict(m=m, n=2 * d_ff, k=d_model, gated=True, blocks=blocks(d_model), whole=False, a=b["x"], a_scale=b["x_scale"],
             b=block.gate_up[0], b_scale=block.gate_up[1], shift=None, residual=None)
    want, off = definition(s, gate=gate)
    assert within(b["h"], want, off).all()
    check_blocks(b["h"].cpu().double(), b["q"].cpu(), b["q_scale"][:, :blocks(d_ff)].cpu(), 0.0)
    s = dict(m=m, n=d_model, k=d_ff, gated=False, blocks=blocks(d_ff), whole=False, a=b["q"], a_scale=b["q_scale"],
             b=block.down[0], b_scale=block.down[1], shift=None, residual=x)
    want, off = definition(s)
    assert within(y, want, off).all()
    # the block on the weights as they were: e4m3 rounds each factor by 2^-4 at most, 2.6% in the mean (2^-4 / sqrt(3) / 1.4);
    # five such factors a term, the sums average them
    if gate == "silu":
        _, n = norm_definition(x.cpu(), None, None if block.norm is None else block.norm.cpu(), block.eps)
        g, u = n @ w[0].double().t(), n @ w[1].double().t()
        want = (g * torch.sigmoid(g) * u) @ w[2].double().t()
        assert (y.cpu().double() - x.cpu().double() - want).norm() < 0.15 * want.norm()


def test_captured_beside_calls_of_other_lengths():
    block, _ = build(512, 1408, rows=40)
    x = rows_of(40, 512, 3)
    y = torch.empty_like(x)
    block(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, y)
    for i in range(3):
        x.copy_(rows_of(40, 512, 4 + i))
        long = rows_of(700 + 300 * i, 512, 9)
        other = torch.empty_like(long)
        block(long, other)                              # grows the shared buffers, not the captured ones
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # rows do not depend on what they are called with, but sums over k may be cut otherwise: the same length again
        again = torch.empty_like(x)
        block(x, again)
        torch.cuda.synchronize()
        assert torch.equal(y, again)
        first = torch.empty_like(long)
        block(long, first)
        torch.cuda.synchronize()
        assert torch.equal(first, other)


def test_a_call_that_shares_its_buffers_is_refused_under_capture():
    block, _ = build(256, 512, rows=8)
    x = rows_of(9, 256, 1)
    y = torch.zeros_like(x)
    block(x, y)
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError), torch.cuda.graph(graph):
        block(x, y)
    block(x, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_no_rows():
    block, _ = build(256, 512)
    block(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("weight", [True, False])
def test_attention_block_with_a_norm(weight):
    """The block with a norm attends as the block without one does to rows that were normalised before."""
    import dl_fusion_amd as dl
    from dl_fusion_amd.decode import PagedAttentionBlock
    hidden, heads, kv, dim, page, cols, requests = 256, 4, 2, 64, 16, 8, 5
    g = torch.Generator().manual_seed(6)
    bf = lambda *s: (torch.randn(*s, generator=g) * s[1] ** -0.5).bfloat16().cuda()  # noqa: E731
    w_qkv, w_o = bf((heads + 2 * kv) * dim, hidden), bf(hidden, heads * dim)
    adapters = (bf(2, 16, hidden), bf(2, (heads + 2 * kv) * dim, 16), None)
    f = torch.rand(hidden, generator=g).add(0.5).cuda() if weight else None
    blocks = [PagedAttentionBlock(w_qkv, w_o, heads, kv, dim, requests, requests * cols, page, cols, adapters, norm=n)
              for n in ((f, 1e-5), None)]
    for b in blocks:
        b.ids.copy_(torch.tensor([0, 1, -1, 1, 0]))

    def normed(x):
        n = torch.empty_like(x)
        dl.dlf_rms_norm(dl.rms_norm_desc(x.shape[0], hidden, 1e-5), x, None, f, None, n, None)
        return n
    fresh = torch.tensor([9, 0, 33, 1, 20], dtype=torch.int32, device="cuda")
    x = rows_of(63 + 4, hidden, 7)
    for b, rows in zip(blocks, (x, normed(x))):
        b.admit(rows, fresh)
    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    for i in range(3):
        x = rows_of(requests, hidden, 8 + i)
        y = torch.empty_like(x)
        blocks[0].step(x, one, y)
        blocks[1].step(normed(x), one, torch.empty_like(x))
        torch.cuda.synchronize()
        assert torch.equal(blocks[0].attended, blocks[1].attended)
        want = torch.empty_like(x)
        dl.dlf_gemm_fused(dl.gemm_desc(requests, hidden, heads * dim), blocks[0].attended.view(requests, -1), w_o, None, None, x, want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
