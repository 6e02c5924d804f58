"""Each large tile of the products with block scales, by name: 128 x 128 two on a CU and alone on it, 256 x 256; with the sum whole
and in parts, every activation and gate, shift and residual, columns that are whole 16 bytes of output, even and odd.  Bounds:
those that test_gpu_gemm_blocks.py derives."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from test_gemm_blocks_plan_host import CASES, plan  # noqa: E402
from test_gpu_gemm_blocks import check, definition, make, product, within  # noqa: E402

NAMES = {5: "128", 6: "128deep", 7: "256"}
ALL = [pytest.param(kind, parts, at, id=f"{NAMES[kind]}-{'parts' if parts else 'whole'}-{('whole16', 'even', 'odd')[at]}")
       for (kind, parts), sizes in CASES.items() for at in range(3)]
EVEN = [p for p in ALL if p.values[2] < 2]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def size_of(kind, parts, at):
    size = CASES[kind, parts][at]
    got = plan(*size)
    assert (got[0], got[1] > 1) == (kind, parts)
    return size


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("kind,parts,at", ALL)
def test_epilogues(kind, parts, at, act):
    check(make(*size_of(kind, parts, at), shift=True, residual=True), act)


@pytest.mark.parametrize("shift,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("kind,parts,at", ALL)
def test_parts_of_the_epilogue(kind, parts, at, shift, residual):
    check(make(*size_of(kind, parts, at), shift=shift, residual=residual))


@pytest.mark.parametrize("gate", ["silu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("kind,parts,at", EVEN)
def test_gates(kind, parts, at, gate):
    check(make(*size_of(kind, parts, at), True, shift=gate != "silu"), gate=gate)


@pytest.mark.parametrize("gate", [None, "silu"])
@pytest.mark.parametrize("kind,parts,at", EVEN)
def test_codes_of_all_magnitudes_and_wide_scale_strides(kind, parts, at, gate):
    check(make(*size_of(kind, parts, at), gate is not None, whole=False, more=(12, 4)), gate=gate)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind,parts", CASES)
def test_each_block_has_its_own_scale(kind, parts, gated):
    """One value a block, powers of two: the sums are whole numbers below 2^24, exact, and name every scale that they used; a
    gate's own rounding comes on top."""
    m, n, k = size_of(kind, parts, 0)
    s = make(m, n, k, gated)
    for x in (s["a"], s["b"]):
        x.copy_(torch.zeros_like(x, dtype=torch.float32))
        x[:, 7::128] = torch.ones_like(x[:, 7::128], dtype=torch.float32).to(x.dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    for sc in (s["a_scale"], s["b_scale"]):
        sc[:, :s["blocks"]] = 2.0 ** torch.randint(0, 3, (sc.shape[0], s["blocks"]), generator=g, device="cuda").float()
    if gated:
        want, off = definition(s, gate="silu")
        assert within(product(s, gate="silu"), want, off).all()
    else:
        want, _ = definition(s)
        assert torch.equal(product(s), want.float().bfloat16())


@pytest.mark.parametrize("gate", [None, "silu"])
@pytest.mark.parametrize("kind,parts", CASES)
def test_the_same_bits_again_beside_another_call_and_from_a_graph(kind, parts, gate):
    import dl_fusion_amd as dl
    m, n, k = size_of(kind, parts, 0)
    s = make(m, n, k, gate is not None, residual=gate is None, seed=2)
    first = product(s, gate=gate).clone()
    d = dl.gemm_blocks_desc(m, n, k)
    size = dl.dlf_gemm_blocks_workspace_bytes(d)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(first), torch.empty(size, dtype=torch.uint8, device="cuda")) for _ in range(2)]

    def call(c, ws, stream=None):
        if gate:
            dl.dlf_gemm_blocks_gated(d, s["a"], s["a_scale"], s["b"], s["b_scale"], None, gate, c, ws, size, stream)
        else:
            dl.dlf_gemm_blocks(d, s["a"], s["a_scale"], s["b"], s["b_scale"], None, s["residual"], c, ws, size, stream)
    torch.cuda.synchronize()
    for _ in range(4):
        for (c, ws), stream in zip(outs, streams):
            call(c, ws, stream)
    torch.cuda.synchronize()
    for c, _ in outs:
        assert torch.equal(c, first)
        c.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*outs[0])
    for _ in range(3):
        outs[0][0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], first)
        call(*outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[1][0], first)


@pytest.mark.parametrize("kind,parts", CASES)
def test_values_that_are_not_finite(kind, parts):
    """A NaN code, and an infinite or NaN scale, reach the rows and columns that use them and no others."""
    m, n, k = size_of(kind, parts, 0)
    s = make(m, n, k, residual=True)
    want, off = definition(s)
    keep = s["a_scale"][1, 0].item(), s["b_scale"][1, 3].item()
    codes = s["a"].view(torch.uint8)[m - 1, k - 1].item(), s["b"].view(torch.uint8)[7, 130].item()
    s["a"].view(torch.uint8)[m - 1, k - 1], s["b"].view(torch.uint8)[7, 130] = 0x7F, 0xFF
    s["a_scale"][1, 0], s["b_scale"][1, 3] = float("inf"), float("nan")
    c = product(s)
    assert c[m - 1].isnan().all() and c[:, 7].isnan().all() and c[:, 128:256].isnan().all()
    assert (~torch.isfinite(c[1])).all()
    clean = torch.ones(m, n, dtype=torch.bool, device="cuda")
    clean[m - 1], clean[1], clean[:, 7], clean[:, 128:256] = False, False, False, False
    assert within(c, want, off)[clean].all()
    s["a"].view(torch.uint8)[m - 1, k - 1], s["b"].view(torch.uint8)[7, 130] = codes
    s["a_scale"][1, 0], s["b_scale"][1, 3] = keep
    assert within(product(s), want, off).all()


@pytest.mark.parametrize("m", [1, 64, 1057])
@pytest.mark.parametrize("small", [1.0, 2.0, 3.25, 3.5, 5.0, 9.0, 13.0, 30.0, "positive", "normal"])
def test_what_an_outlier_takes_from_its_neighbours(m, small):
    """One product of 448 x 448, 2^17 at its power of two, among 127 others: 7 neighbours lose less than 2^-14 of that each.  The
    shift takes the large product away again, so that the others' sum is seen; fp32 sums of 2^18 round by 2^-6 at most."""
    import dl_fusion_amd as dl
    n, k = (64, 128) if m < 1000 else (7376, 128)
    g = torch.Generator().manual_seed(5)
    draw = {"positive": lambda: torch.rand(k, generator=g) * 3, "normal": lambda: torch.randn(k, generator=g) * 3}
    a, b = (draw[small]() if small in draw else torch.full((k,), small) for _ in range(2))
    a[0] = b[0] = 448.0
    a, b = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    want = float((a.double() * b.double())[1:].sum())
    sa, sb = torch.ones(m, 4, device="cuda"), torch.ones(-(-n // 128), 4, device="cuda")
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    shift = torch.full((n,), -448.0 * 448.0, device="cuda")
    d = dl.gemm_blocks_desc(m, n, k)
    assert dl.dlf_gemm_blocks_workspace_bytes(d) == 0
    dl.dlf_gemm_blocks(d, a.repeat(m, 1).cuda(), sa, b.repeat(n, 1).cuda(), sb, shift, None, c, None, 0)
    assert ((c.double() - want).abs() <= 7 * 2.0 ** -14 * 2 ** 17 + 2.0 ** -6 + 2.0 ** -9 * c.double().abs()).all(), (float(c[0, 0]), want)
