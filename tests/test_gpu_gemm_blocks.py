"""Products of e4m3 matrices with block scales on the GPU against their definition in 64 bits.

Bound, derived before its first run, with u = 2^-24 and everything exact in the inputs.  T blocks of k, S =
sum_t a_scale b_scale sum |a| |b|.  The matrix cores align a block's products to the largest and cut them 2^-14 below
its power of two.  Codes that are whole numbers up to 8 have products of at most 2^6 in whole numbers, and sums below
2^24: nothing is cut, a block's sum is exact.  Codes of all magnitudes lose less than 2^-14 P a product, P the
power of two of a block's largest product |a| |b|, and 2 u S in sums: 128 (2^-14 P + 2 u P).  The product of the two
scales, the FMA that adds a block and the joins of waves' and workgroups' shares are T + 42 more of u S.  Shift and
residual add u each.  act and gates have a slope of at most 1.13, are off by at most 2^-15 relative (exp2 of an
argument below 90 that is off by 4 u, and a reciprocal), the erf form by 1e-7 |v| more.  c is the rounding to bf16 of a
value that is off by at most d: it lies between the roundings of c - d and c + d, rounding being monotone.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dl_fusion_amd  # noqa: F401  (loud failure if the library is missing)
    torch.cuda.set_device(0)


def make(m, n, k, gated=False, shift=False, residual=False, seed=0, more=(0, 0), whole=True):
    """Codes that are whole numbers up to 8, or of all magnitudes, and scales that differ from block to block; between
    the scales' rows NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * m + n + 31 * k)
    blocks = -(-k // 128)
    stride = -(-blocks // 4) * 4
    slabs = 2 * -(-n // 256) if gated else -(-n // 128)

    def codes(rows):
        if whole:
            return torch.randint(-8, 9, (rows, k), generator=g, device="cuda").to(FP8)
        return (torch.randn(rows, k, generator=g, device="cuda") * 60).clamp(-448, 448).to(FP8)

    def scales(rows, more):
        s = torch.full((rows, stride + more), float("nan"), device="cuda")
        s[:, :blocks] = torch.exp(torch.randn(rows, blocks, generator=g, device="cuda"))
        return s
    size = 2.0 ** -3 if whole else 2.0 ** -7
    return dict(m=m, n=n, k=k, gated=gated, blocks=blocks, whole=whole, a=codes(m), b=codes(n),
                a_scale=scales(m, more[0]) * size, b_scale=scales(slabs, more[1]) * size * max(k, 1) ** -0.5,
                shift=torch.randn(n, generator=g, device="cuda") if shift else None,
                residual=torch.randn(m, n, generator=g, device="cuda").bfloat16() if residual else None)


def act64(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "gelu_erf":
        return v * torch.special.ndtr(v)
    return v


def definition(s, act="none", gate=None):
    """The exact result and how far it may be off before it is rounded."""
    m, n, k, t = s["m"], s["n"], s["k"], s["blocks"]
    r = torch.arange(n, device="cuda")
    row = 2 * (r // 256) + r % 2 if s["gated"] else r // 128
    wide = lambda x, sc: x.double() * sc[:, :t].double().repeat_interleave(128, 1)[:, :k]  # noqa: E731
    a, b = wide(s["a"], s["a_scale"]), wide(s["b"], s["b_scale"][row])
    v = a @ b.t()
    d = (t + 42) * U * (a.abs() @ b.abs().t())
    if not s["whole"]:
        for j in range(t):
            top = [x[:, 128 * j:128 * j + 128].abs().amax(1) for x in (a, b)]
            d += 128 * (2.0 ** -14 + 2 * U) * top[0][:, None] * top[1]
    for x in (s["shift"], s["residual"]):
        if x is not None:
            v = v + x.double()
            d = d + U * v.abs()
    name = gate or act
    z, dz = (v[:, 0::2], d[:, 0::2]) if gate else (v, d)
    out = act64(name, z)
    off = dz if name in ("none", "relu") else 1.13 * dz + 2.0 ** -15 * out.abs() + (1e-7 * z.abs() if name == "gelu_erf" else 0)
    if gate:
        up, dup = v[:, 1::2], d[:, 1::2]
        off = off * (up.abs() + dup) + out.abs() * dup + U * (out * up).abs()
        out = out * up
    return out, off


def product(s, act="none", gate=None, stream=None):
    import dl_fusion_amd as dl
    m, n = s["m"], s["n"]
    width = n // 2 if gate else n
    buf = torch.empty(m * width + 512, dtype=torch.bfloat16, device="cuda")
    buf.view(torch.uint8).fill_(0xA5)
    c = buf[:m * width].view(m, width)
    d = dl.gemm_blocks_desc(m, n, s["k"], act, *((s["a_scale"].stride(0), s["b_scale"].stride(0)) if s["k"] else (0, 0)))
    size = dl.dlf_gemm_blocks_workspace_bytes(d)
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda").fill_(0xFF)      # NaN: read only where written
    torch.cuda.synchronize()
    if gate:
        dl.dlf_gemm_blocks_gated(d, s["a"], s["a_scale"], s["b"], s["b_scale"], s["shift"], gate, c, ws, size, stream)
    else:
        dl.dlf_gemm_blocks(d, s["a"], s["a_scale"], s["b"], s["b_scale"], s["shift"], s["residual"], c, ws, size, stream)
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all(), "store beyond the workspace"
    assert (buf[m * width:].view(torch.uint8) == 0xA5).all(), "store beyond the output"
    return c


def within(c, want, off):
    """Whether c is a rounding to bf16 of values between want - off and want + off.  (torch rounds 64 bits to 32 first:
    u of the value more.)"""
    off = off + U * want.abs()
    return ((want - off).bfloat16() <= c) & (c <= (want + off).bfloat16())


def check(s, act="none", gate=None):
    c = product(s, act, gate)
    want, off = definition(s, act, gate)
    bad = ~within(c, want, off)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((c.double() - want).abs().max()))


ROWS = [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 257, 300, 512, 1000]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", [(256, 512), (100, 144), (1000, 4096)])
def test_rows(m, n, k):
    check(make(m, n, k, shift=True, residual=True))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 15, 16, 17, 30, 63, 64, 66, 127, 128, 129, 130, 255, 256, 258, 384, 514, 1026, 4096])
@pytest.mark.parametrize("m", [1, 40, 300])
def test_columns(m, n):
    check(make(m, n, 400))
    check(make(m, n, 128, shift=True, residual=True))


@pytest.mark.parametrize("k", [0, 16, 32, 112, 128, 144, 240, 256, 272, 384, 512, 640, 1040, 2048, 4112, 8192, 11008, 20480])
@pytest.mark.parametrize("m,n", [(1, 130), (24, 72), (70, 256), (260, 320)])
def test_depths(m, n, k):
    check(make(m, n, k, residual=True))


@pytest.mark.parametrize("gate", ["silu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("m,n,k", [(1, 2, 16), (3, 256, 384), (16, 514, 128), (33, 1000, 272), (64, 768, 1024), (200, 700, 144),
                                   (300, 510, 640), (700, 1280, 512)])
def test_gated(gate, m, n, k):
    check(make(m, n, k, True, shift=m % 2 == 1), gate=gate)


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "gelu_erf"])
@pytest.mark.parametrize("m,n,k", [(5, 300, 256), (130, 200, 144), (520, 520, 384)])
def test_epilogues(act, m, n, k):
    check(make(m, n, k, shift=True), act)
    check(make(m, n, k, residual=True), act)


@pytest.mark.parametrize("m,n,k,gate", [(64, 22016, 4096, "silu"), (64, 4096, 11008, None), (1, 4096, 4096, None),
                                        (777, 5000, 4112, None), (2048, 4096, 4096, None), (1500, 2816, 4096, "silu")])
def test_large(m, n, k, gate):
    check(make(m, n, k, gate is not None), gate=gate)


@pytest.mark.parametrize("m,n,k,gate", [(1000, 4000, 2064, None), (900, 3900, 1424, "gelu_tanh"), (700, 5001, 4096, None),
                                        (1024, 4096, 1536, "silu"), (520, 6100, 3000 // 16 * 16, None), (130, 15000, 1680, None),
                                        (2000, 2050, 6000, "gelu_erf"), (385, 4098, 11008, None)])
def test_about_as_many_tiles_as_cus(m, n, k, gate):
    check(make(m, n, k, gate is not None, shift=True, residual=gate is None), gate=gate)


@pytest.mark.parametrize("m", [1, 16, 17, 32])
@pytest.mark.parametrize("n", [6144, 6146, 6161, 8200])
def test_few_rows_and_many_columns(m, n):
    check(make(m, n, 272, shift=True, residual=True))
    if n % 2 == 0:
        check(make(m, n, 384, True), gate="silu")


@pytest.mark.parametrize("m,n,k,gate", [(1, 256, 11008, None), (20, 301, 11008, None), (32, 1026, 8192, "gelu_tanh"), (33, 5, 8192, None),
                                        (50, 1023, 8192, None), (40, 514, 8208, "silu"), (300, 130, 20480, None), (129, 258, 5000 // 16 * 16, "silu"),
                                        (64, 2048, 4096, None), (200, 700, 16384, None), (1000, 256, 8192, None)])
def test_sums_in_parts(m, n, k, gate):
    import dl_fusion_amd as dl
    assert dl.dlf_gemm_blocks_workspace_bytes(dl.gemm_blocks_desc(m, n, k)) > 0
    s = make(m, n, k, gate is not None, shift=True, residual=gate is None)
    check(s, "none" if gate else "gelu_tanh", gate)


def test_two_streams_at_once():
    import dl_fusion_amd as dl
    cases = [(make(m, n, k, seed=i), dl.gemm_blocks_desc(m, n, k)) for i, (m, n, k) in
             enumerate([(64, 4096, 11008), (500, 2048, 2048), (16, 4096, 4096), (300, 1024, 8192)])]
    want = [product(s) for s, _ in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(w) for w in want]
    ws = [torch.empty(dl.dlf_gemm_blocks_workspace_bytes(d), dtype=torch.uint8, device="cuda") for _, d in cases]
    torch.cuda.synchronize()
    for turn in range(3):
        for i, (s, d) in enumerate(cases):
            dl.dlf_gemm_blocks(d, s["a"], s["a_scale"], s["b"], s["b_scale"], None, None, got[i], ws[i], ws[i].numel(), streams[i % 2])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
            g.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("m,n,k,gate", [(9, 300, 1024, None), (80, 300, 400, None), (400, 512, 1024, "silu"), (900, 768, 256, None)])
def test_codes_of_all_magnitudes(m, n, k, gate):
    check(make(m, n, k, gate is not None, whole=False), gate=gate)


@pytest.mark.parametrize("m", [3, 70, 300])
def test_every_code(m):
    """Rows with one code of each kind against rows with a single 1: the result is the code's value."""
    k, n = 256, 256
    s = make(m, n, k)
    a = torch.zeros(m, k, dtype=torch.uint8)
    b = torch.zeros(n, k, dtype=torch.uint8)
    a[m - 1] = torch.arange(256)
    a[m - 1, [0x7F, 0xFF]] = 0
    b[torch.arange(n), torch.arange(n)] = 0x38
    s["a"], s["b"] = a.cuda().view(FP8), b.cuda().view(FP8)
    s["a_scale"][:, :2], s["b_scale"][:, :2] = 1.0, 1.0
    c = product(s)
    assert torch.equal(c[m - 1].cpu(), a[m - 1].view(FP8).bfloat16()) and (c[:m - 1] == 0).all()


@pytest.mark.parametrize("m", [7, 90, 600])
def test_scale_strides(m):
    check(make(m, 300, 1000 // 16 * 16, more=(12, 4)))


@pytest.mark.parametrize("m", [20, 64, 130, 600])
def test_largest_scale_strides(m):
    check(make(m, 300, 400, more=((1 << 20) - 4, (1 << 20) - 4)))


def test_tensors_off_the_current_device_are_refused():
    import dl_fusion_amd as dl
    s = make(4, 256, 512)
    d = dl.gemm_blocks_desc(4, 256, 512)
    c = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    rows, norm, quant = torch.zeros(4, 512, device="cuda"), dl.rms_norm_desc(4, 512, dtype="f32", out_dtype="f32"), dl.quant_blocks_desc(4, 512, "f32")
    for off in ("a", "c"):
        a, out = (s["a"].cpu(), c) if off == "a" else (s["a"], c.cpu())
        with pytest.raises(ValueError):
            dl.dlf_gemm_blocks(d, a, s["a_scale"], s["b"], s["b_scale"], None, None, out, None, 0)
        with pytest.raises(ValueError):
            dl.dlf_gemm_blocks_gated(d, a, s["a_scale"], s["b"], s["b_scale"], None, "silu", out[:, :128].contiguous(), None, 0)
        x, y = (rows.cpu(), rows) if off == "a" else (rows, rows.cpu())
        with pytest.raises(ValueError):
            dl.dlf_rms_norm(norm, x, None, None, None, y, None)
        with pytest.raises(ValueError):
            dl.dlf_quant_blocks(quant, x, torch.empty(4, 512, dtype=FP8, device=y.device), s["a_scale"])


@pytest.mark.parametrize("m", [3, 60, 140, 600])
def test_each_block_has_its_own_scale(m):
    """One value a block, powers of two: the result is exact, and names every scale that it used."""
    n, k = 260, 640
    s = make(m, n, k)
    for x in (s["a"], s["b"]):
        x.copy_(torch.zeros_like(x, dtype=torch.float32))
        x[:, 77::128] = torch.ones_like(x[:, 77::128], dtype=torch.float32).to(FP8)
    g = torch.Generator(device="cuda").manual_seed(1)
    for sc in (s["a_scale"], s["b_scale"]):
        sc[:, :s["blocks"]] = 2.0 ** torch.randint(0, 5, (sc.shape[0], s["blocks"]), generator=g, device="cuda").float()
    want, _ = definition(s)
    assert torch.equal(product(s), want.bfloat16())


@pytest.mark.parametrize("m", [3, 60, 140, 600])
def test_values_that_are_not_finite(m):
    """A NaN code, and an infinite or NaN scale, reach the rows and columns that use them and no others."""
    n, k = 300, 400
    s = make(m, n, k)
    s["a"].view(torch.uint8)[2, 399] = 0x7F
    s["b"].view(torch.uint8)[7, 130] = 0xFF
    clean = torch.ones(m, n, dtype=torch.bool, device="cuda")
    clean[2], clean[:, 7] = False, False
    s["b_scale"][2, 3] = float("nan")
    clean[:, 256:] = False
    s["a_scale"][1, 0] = float("inf")
    c = product(s)
    assert c[2].isnan().all() and c[:, 7].isnan().all() and c[:, 256:].isnan().all()
    clean[1] = False
    assert (~torch.isfinite(c[1])).all()
    s["a"].view(torch.uint8)[2, 399], s["b"].view(torch.uint8)[7, 130] = 0, 0
    s["b_scale"][2, 3], s["a_scale"][1, 0] = 1.0, 1.0
    want, off = definition(s)
    assert within(c, want, off)[clean].all()


@pytest.mark.parametrize("m,n,k,gate", [(1, 4096, 4096, None), (16, 512, 2048, "silu"), (64, 4096, 4096, None), (64, 256, 11008, None),
                                        (200, 1024, 4096, None), (1024, 2048, 1024, "silu")])
def test_the_same_bits_again_on_another_stream_and_from_a_graph(m, n, k, gate):
    import dl_fusion_amd as dl
    s = make(m, n, k, gate is not None, seed=3)
    first = product(s, gate=gate).clone()
    assert torch.equal(first, product(s, gate=gate))
    assert torch.equal(first, product(s, gate=gate, stream=torch.cuda.Stream()))
    d = dl.gemm_blocks_desc(m, n, k)
    ws = torch.empty(dl.dlf_gemm_blocks_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    c = torch.empty(m, n // 2 if gate else n, dtype=torch.bfloat16, device="cuda")

    def call(c):
        if gate:
            dl.dlf_gemm_blocks_gated(d, s["a"], s["a_scale"], s["b"], s["b_scale"], None, gate, c, ws, ws.numel())
        else:
            dl.dlf_gemm_blocks(d, s["a"], s["a_scale"], s["b"], s["b_scale"], None, None, c, ws, ws.numel())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c)
    other = torch.empty_like(c)
    for i in range(3):
        s["a_scale"].mul_(1 + i)
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        call(other)                 # the same workspace, in stream order
        torch.cuda.synchronize()
        assert torch.equal(c, other)
        assert (c == first).all() if i == 0 else not torch.equal(c, first)


def test_offsets_past_4_gigabytes():
    """a, b and c beyond 2^32 bytes: rows and columns far from the start, against their own small products."""
    import dl_fusion_amd as dl
    m, n, k = 70000, 40000, 128
    s = make(m, n, k)
    c = product(s)
    for r, col in ((0, 0), (m - 40, n - 200), (m // 2, n - 130), (m - 3, 0)):
        part = dict(s, m=3, n=128, a=s["a"][r:r + 3], b=s["b"][col // 128 * 128:col // 128 * 128 + 128], a_scale=s["a_scale"][r:r + 3],
                    b_scale=s["b_scale"][col // 128:col // 128 + 1])
        part["n"] = part["b"].shape[0]
        want, off = definition(part)
        assert within(c[r:r + 3, col // 128 * 128:col // 128 * 128 + part["n"]], want, off).all(), (r, col)
    del c, s
    m, n, k = 40, 600000, 8192          # b of 4.9 GB
    b = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda").view(FP8)      # all magnitudes
    s = make(m, 64, k)
    bs = torch.rand(-(-n // 128), 64, device="cuda") * 1e-4
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    d = dl.gemm_blocks_desc(m, n, k)
    ws = torch.empty(dl.dlf_gemm_blocks_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    dl.dlf_gemm_blocks(d, s["a"], s["a_scale"], b, bs, None, None, c, ws, ws.numel())
    for col in (0, 256 * 1024, n - 64):
        first = col // 128 * 128
        part = dict(s, n=64, whole=False, b=b[first:first + 64], b_scale=bs[col // 128:col // 128 + 1])
        want, off = definition(part)
        assert within(c[:, first:first + 64], want, off).all(), col
    # a of 4.9 GB
    s = make(64, 40, k)
    scale = torch.rand(n, 64, device="cuda") * 1e-4
    c = torch.empty(n, 40, dtype=torch.bfloat16, device="cuda")
    d = dl.gemm_blocks_desc(n, 40, k)
    ws = torch.empty(dl.dlf_gemm_blocks_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    dl.dlf_gemm_blocks(d, b, scale, s["b"], s["b_scale"], None, None, c, ws, ws.numel())
    for r in (0, 300000, n - 64):
        want, off = definition(dict(s, m=64, whole=False, a=b[r:r + 64], a_scale=scale[r:r + 64]))
        assert within(c[r:r + 64], want, off).all(), r


def test_norm_product_gate_quantise_product():
    """The operators together, as a feed-forward block has them, against the block in 64 bits.

    Codes stand for their values, so each product is compared from the codes that it was given (its bound holds),
    and each quantiser from the values that it was given."""
    import dl_fusion_amd as dl
    m, d_model, d_ff = 50, 768, 1280
    g = torch.Generator().manual_seed(4)
    w1 = torch.randn(2 * d_ff, d_model, generator=g) * d_model ** -0.5
    w2 = torch.randn(d_model, d_ff, generator=g) * d_ff ** -0.5
    (c1, s1), (c2, s2) = dl.dlf_quant_blocks_weights(w1.numpy(), gated=True), dl.dlf_quant_blocks_weights(w2.numpy())
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    c1, c2, s1, s2 = dev(c1).view(FP8), dev(c2).view(FP8), dev(s1), dev(s2)
    x = (torch.randn(m, d_model, generator=g) * 3).bfloat16().cuda()
    a, sa = torch.empty(m, d_model, dtype=FP8, device="cuda"), torch.full((m, dl.scale_stride(d_model)), float("nan"), device="cuda")
    dl.dlf_rms_norm(dl.rms_norm_desc(m, d_model, 1e-5, "bf16", "fp8"), x, None, None, None, a, sa)
    first = dict(m=m, n=2 * d_ff, k=d_model, gated=True, blocks=6, whole=False, a=a, a_scale=sa, b=c1, b_scale=s1, shift=None, residual=None)
    check(first, gate="silu")
    h = product(first, gate="silu").contiguous()
    q, sq = torch.empty(m, d_ff, dtype=FP8, device="cuda"), torch.full((m, dl.scale_stride(d_ff)), float("nan"), device="cuda")
    dl.dlf_quant_blocks(dl.quant_blocks_desc(m, d_ff), h, q, sq)
    second = dict(m=m, n=d_model, k=d_ff, gated=False, blocks=10, whole=False, a=q, a_scale=sq, b=c2, b_scale=s2, shift=None, residual=x)
    check(second)
    y = product(second).double()
    # the whole block in 64 bits from the unquantised weights: three roundings to e4m3 (2^-4 at most, uniform within a
    # step: a root mean square of 2^-4 / sqrt(3) / 1.4 = 2.6% at most) a product's term, averaged over d_model and d_ff terms
    xd, W1, W2 = x.double(), w1.double().cuda(), w2.double().cuda()
    n = xd / (xd.square().mean(1, keepdim=True) + 1e-5).sqrt()
    v = n @ W1.t()
    want = (act64("silu", v[:, 0::2]) * v[:, 1::2]) @ W2.t()
    assert ((y - xd - want).norm() / want.norm()) < 0.1
