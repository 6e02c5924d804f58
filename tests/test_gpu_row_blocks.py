"""The root-mean-square norm and the block quantiser on the GPU against their definitions in 64 bits.

Bounds, derived before any run, with u = 2^-24 (fp32) and D = cols / 64 + 40 (no sum of a row is a chain of
more additions: at least 64 threads share it, at most 24 steps join them).  h = x + residual is off by u.  A
row's sum of squares has 2 u from h, u from each product and D u from its order; the mean, eps, the root and
the reciprocal add 4 u; the square root halves what it is given.  Two products follow.  So before it is
rounded y is off by at most
    e = (D / 2 + 9) u   relative to |y|
and stored as bf16 by 2^-8 more; sum by u and 2^-8 (bf16).  A block's scale is off by e + 2 u.  A code is the
rounding of a value that is off by at most e + 4 u (the scale's reciprocal and the product by it): it lies
between the codes of t (1 - d) and t (1 + d) for t the exact quotient and d = 2 e + 6 u, rounding being
monotone.  The quantiser alone has e = 0.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
FP8 = torch.float8_e4m3fn
LEAST = 2.0 ** -110
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dl_fusion_amd  # noqa: F401  (loud failure if the library is missing)
    torch.cuda.set_device(0)


def dtype_of(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def rows_of(rows, cols, dtype, seed, wide=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, wide or cols, generator=g) * torch.exp(3 * torch.rand(rows, 1, generator=g))
    x[:, ::13] *= 30
    return x.to(dtype_of(dtype))


def guarded(rows, stride, dtype, extra=64):
    """A buffer of `rows` rows of `stride` elements and some more, of a pattern that no result has."""
    buf = torch.empty(rows * stride + extra, dtype=dtype, device="cuda")
    buf.view(torch.uint8).fill_(0xA5)
    return buf, buf[:rows * stride].view(rows, stride)


def untouched(buf, view, cols):
    """Whether everything in buf beside view[:, :cols] is as it was."""
    raw = buf.clone().view(torch.uint8)
    size = buf.element_size()
    raw[:view.numel() * size].view(view.shape[0], -1)[:, :cols * size] = 0xA5
    return bool((raw == 0xA5).all())


def q(t):
    return t.clamp(-448, 448).to(FP8).double()


def blocked(v):
    """v [rows][cols] as [rows][blocks][128], zeros behind the last."""
    rows, cols = v.shape
    return torch.nn.functional.pad(v, (0, -cols % 128)).view(rows, -1, 128)


def check_blocks(y, codes, scale, e):
    """codes and scales of exact values y, which are off by e (relative) where they are quantised."""
    b = blocked(y)
    top = b.abs().amax(2).clamp(min=LEAST)
    got = scale.double()
    assert ((got - top / 448).abs() <= (e + 2 * U) * top / 448).all()
    t = b / top[:, :, None] * 448
    d = 2 * e + 6 * U
    lo, hi = q(t - d * t.abs()), q(t + d * t.abs())
    c = blocked(codes.double())
    assert ((lo <= c) & (c <= hi)).all(), ((c < lo) | (c > hi)).sum()


def norm(x, residual, weight, out, want_sum, strides=(0, 0, 0, 0), eps=EPS, inv=1.0, scale_more=0, stream=None):
    """One call on guarded buffers; `strides`: elements between rows beyond cols of x, residual, sum and y.
    x and residual come with their strides.  (sum, y, scale) on the CPU."""
    import dl_fusion_amd as dl
    rows = x.shape[0]
    cols = x.shape[1] - strides[0]
    dtype = "f32" if x.dtype == torch.float32 else "bf16"
    xd = x.cuda()[:, :cols]
    rd = None if residual is None else residual.cuda()[:, :cols]
    wd = None if weight is None else weight.cuda()
    sbuf, s = guarded(rows, cols + strides[2], x.dtype)
    ytype = FP8 if out in ("static", "blocks") else dtype_of(out)
    ybuf, y = guarded(rows, cols + strides[3], ytype)
    blocks = -(-cols // 128)
    stride = dl.scale_stride(cols) + scale_more
    cbuf, c = guarded(rows, stride, torch.float32)
    d = dl.rms_norm_desc(rows, cols, eps, dtype, "fp8" if out in ("static", "blocks") else out, inv, cols + strides[0],
                         cols + strides[1], cols + strides[2], cols + strides[3], stride)
    torch.cuda.synchronize()
    dl.dlf_rms_norm(d, xd, rd, wd, s[:, :cols] if want_sum else None, y[:, :cols], c if out == "blocks" else None, stream)
    torch.cuda.synchronize()
    assert untouched(sbuf, s, cols if want_sum else 0), "store beside the sum"
    assert untouched(ybuf, y, cols), "store beside the output"
    assert untouched(cbuf, c, blocks if out == "blocks" else 0), "store beside the scales"
    return s[:, :cols].cpu() if want_sum else None, y[:, :cols].cpu(), c[:, :blocks].cpu()


def definition(x, residual, weight, eps=EPS):
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / (h.square().mean(1, keepdim=True) + eps).sqrt()
    return h, y if weight is None else y * weight.double()


def check(x, residual, weight, out, want_sum=True, strides=(0, 0, 0, 0), eps=EPS, inv=1.0, **kw):
    s, y, c = norm(x, residual, weight, out, want_sum, strides, eps, inv, **kw)
    cols = x.shape[1] - strides[0]
    h, want = definition(x[:, :cols], None if residual is None else residual[:, :cols], weight, eps)
    if want_sum:
        assert ((s.double() - h).abs() <= (U + (2.0 ** -8 if s.dtype == torch.bfloat16 else 0)) * h.abs()).all()
    e = (cols / 64 / 2 + 20 + 9) * U
    if out == "blocks":
        check_blocks(want, y, c, e)
    elif out == "static":
        t = want * inv
        d = e + 2 * U
        got = y.double()
        assert ((q(t - d * t.abs()) <= got) & (got <= q(t + d * t.abs()))).all()
    else:
        assert ((y.double() - want).abs() <= (e + (2.0 ** -8 if out == "bf16" else 0)) * want.abs()).all()


WIDTHS = [1, 7, 8, 64, 127, 128, 129, 512, 520, 1023, 1024, 1032, 2048, 2049, 4096, 4104, 8192, 8200, 11008, 16384, 16392, 33001]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype,out", [("bf16", "blocks"), ("f32", "f32"), ("bf16", "bf16")])
def test_norm_widths(cols, dtype, out):
    rows = 5
    w = torch.randn(cols, generator=torch.Generator().manual_seed(1))
    check(rows_of(rows, cols, dtype, cols), rows_of(rows, cols, dtype, cols + 1), w, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32", "static", "blocks"])
@pytest.mark.parametrize("residual,want_sum,weight", [(False, False, True), (False, True, False), (True, False, False), (True, True, True)])
def test_norm_types_and_parts(dtype, out, residual, want_sum, weight):
    rows, cols = 9, 1288
    w = torch.randn(cols, generator=torch.Generator().manual_seed(2)) if weight else None
    check(rows_of(rows, cols, dtype, 3), rows_of(rows, cols, dtype, 4) if residual else None, w, out, want_sum, inv=20.0)


@pytest.mark.parametrize("strides", [(8, 16, 24, 32), (1, 3, 5, 7), (200, 0, 0, 9)])
@pytest.mark.parametrize("dtype,out", [("bf16", "blocks"), ("bf16", "bf16"), ("f32", "static"), ("f32", "f32")])
@pytest.mark.parametrize("cols", [300, 2500, 17000])
def test_norm_strides(strides, dtype, out, cols):
    rows = 6
    check(rows_of(rows, cols, dtype, 5, cols + strides[0]), rows_of(rows, cols, dtype, 6, cols + strides[1]), None, out,
          strides=strides, inv=30.0, scale_more=8)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 1025])
@pytest.mark.parametrize("cols", [200, 1500])
def test_norm_rows(rows, cols):
    check(rows_of(rows, cols, "bf16", rows), rows_of(rows, cols, "bf16", 7), None, "blocks")


def test_norm_of_more_rows_than_a_launch_has_workgroups_for():
    import dl_fusion_amd as dl
    rows, cols = (4 << 20) + 4099, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(rows, cols, dtype=torch.float32, device="cuda")
    dl.dlf_rms_norm(dl.rms_norm_desc(rows, cols, EPS, "bf16", "f32"), x, None, None, None, y, None)
    h = x.double()
    want = h / (h.square().mean(1, keepdim=True) + EPS).sqrt()
    assert ((y - want).abs() <= 50 * U * want.abs()).all()


@pytest.mark.parametrize("cols", [5, 13, 96, 1003, 4096, 4099, 12301, 20000, 20003])
@pytest.mark.parametrize("where", ["sum is x", "sum is residual", "y is x", "y is residual", "y is x, sum is residual"])
def test_norm_in_place(cols, where):
    import dl_fusion_amd as dl
    rows = 7
    x, r = rows_of(rows, cols, "bf16", 8), rows_of(rows, cols, "bf16", 9)
    s0, y0, _ = norm(x, r, None, "bf16", True)
    xd, rd = x.cuda(), r.cuda()
    s, y = torch.empty_like(xd), torch.empty_like(xd)
    if "sum is x" in where:
        s = xd
    if "sum is residual" in where:
        s = rd
    if "y is x" in where:
        y = xd
    if "y is residual" in where:
        y = rd
    dl.dlf_rms_norm(dl.rms_norm_desc(rows, cols, EPS), xd, rd, None, s, y, None)
    assert torch.equal(s.cpu(), s0) and torch.equal(y.cpu(), y0)


@pytest.mark.parametrize("cols", [520, 4096, 20000])
def test_norm_of_values_past_the_range_of_squares(cols):
    x = rows_of(4, cols, "f32", 10)
    x[0] *= 1e30
    x[1] *= 1e-30        # nothing beside eps
    x[2] = 3e38
    check(x, None, None, "f32")
    check(x, None, None, "blocks")


@pytest.mark.parametrize("cols", [520, 4096, 20000])
def test_norm_of_rows_that_are_not_finite(cols):
    nan, inf = float("nan"), float("inf")
    x = rows_of(5, cols, "bf16", 11)
    x[0, 3] = nan
    x[1, 4] = inf
    x[2, 5], x[2, cols - 1] = inf, -inf
    _, y, _ = norm(x, None, None, "f32", True)
    assert y[0].isnan().all()
    for row, places in ((1, [4]), (2, [5, cols - 1])):
        bad = torch.zeros(cols, dtype=torch.bool)
        bad[places] = True
        assert torch.equal(y[row].isnan(), bad) and (y[row][~bad] == 0).all()
    _, want = definition(x[3:], None, None)
    assert ((y[3:] - want).abs() <= (cols / 128 + 29) * U * want.abs()).all()
    # codes: NaN stays, the others of its block are as if it were not there
    _, y, c = norm(x, None, None, "blocks", True)
    assert y[0].float().isnan().all() and torch.equal(y[1].float().isnan(), torch.arange(cols) == 4)
    assert torch.isfinite(c).all()


def test_rows_past_4_gigabytes():
    """Four rows 2^30 + 8 elements apart, of the norm and of the quantiser."""
    import dl_fusion_amd as dl
    rows, cols, stride = 4, 4096, (1 << 30) + 8
    x, r = rows_of(rows, cols, "bf16", 20), rows_of(rows, cols, "bf16", 21)
    s0, y0, c0 = norm(x, r, None, "blocks", True)
    q0, qs0 = quant(x)
    far = [torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").view(rows, stride)[:, :cols] for _ in range(3)]
    codes = [torch.empty(rows * stride, dtype=torch.uint8, device="cuda").view(FP8).view(rows, stride)[:, :cols] for _ in range(2)]
    far[0].copy_(x)
    far[1].copy_(r)
    c, qs = torch.empty(rows, 32, device="cuda"), torch.empty(rows, 32, device="cuda")
    dl.dlf_rms_norm(dl.rms_norm_desc(rows, cols, EPS, "bf16", "fp8", 1.0, stride, stride, stride, stride), far[0], far[1], None,
                    far[2], codes[0], c)
    dl.dlf_quant_blocks(dl.quant_blocks_desc(rows, cols, "bf16", stride, stride), far[0], codes[1], qs)
    torch.cuda.synchronize()
    for got, want in ((far[2], s0), (c, c0), (qs, qs0)):
        assert torch.equal(got.cpu(), want)
    for got, want in zip(codes, (y0, q0)):
        assert torch.equal(got.view(torch.uint8).cpu(), want.view(torch.uint8))


def test_norm_of_zeros():
    for out in ("bf16", "blocks"):
        _, y, c = norm(torch.zeros(3, 300, dtype=torch.bfloat16), None, None, out, True)
        assert (y.float() == 0).all()
    assert (c == LEAST / 448).all()


def test_norm_gives_the_same_bits_again_and_beside_other_rows():
    x = rows_of(40, 4096, "bf16", 12)
    s, y, c = norm(x, x, None, "blocks", True)
    s2, y2, c2 = norm(x[17:18], x[17:18], None, "blocks", True)
    assert torch.equal(s[17:18], s2) and torch.equal(y.view(torch.uint8)[17:18], y2.view(torch.uint8)) and torch.equal(c[17:18], c2)


# ---------------------------------------------------------------------------
# Quantiser
# ---------------------------------------------------------------------------
def quant(x, cols=None, codes_more=0, scale_more=0, stream=None):
    import dl_fusion_amd as dl
    rows = x.shape[0]
    cols = cols or x.shape[1]
    dtype = "f32" if x.dtype == torch.float32 else "bf16"
    xd = x.cuda()
    ybuf, y = guarded(rows, cols + codes_more, FP8)
    stride = dl.scale_stride(cols) + scale_more
    cbuf, c = guarded(rows, stride, torch.float32)
    d = dl.quant_blocks_desc(rows, cols, dtype, xd.stride(0), cols + codes_more, stride)
    torch.cuda.synchronize()
    dl.dlf_quant_blocks(d, xd[:, :cols], y[:, :cols], c, stream)
    torch.cuda.synchronize()
    assert untouched(ybuf, y, cols) and untouched(cbuf, c, -(-cols // 128)), "store beside the output"
    return y[:, :cols].cpu(), c[:, :-(-cols // 128)].cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 127), (2, 128), (7, 129), (1, 4096), (64, 11008), (33, 1000), (300, 64), (2, 65537)])
def test_quant(dtype, rows, cols):
    x = rows_of(rows, cols, dtype, rows + cols)
    y, c = quant(x)
    check_blocks(x.double(), y, c, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [(8, 16, 4), (1, 3, 0), (5, 0, 12)])
def test_quant_strides(dtype, more):
    x = rows_of(11, 700, dtype, 13, 700 + more[0])
    y, c = quant(x, 700, more[1], more[2])
    check_blocks(x[:, :700].double(), y, c, 0.0)


def test_quant_of_more_blocks_than_a_launch_has_workgroups_for():
    import dl_fusion_amd as dl
    rows, cols = (16 << 20) + 77, 8
    x = torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).bfloat16()
    codes = torch.zeros(rows, cols, dtype=FP8, device="cuda")
    scale = torch.zeros(rows, 4, device="cuda")
    dl.dlf_quant_blocks(dl.quant_blocks_desc(rows, cols), x, codes, scale)
    v = x.double()
    top = v.abs().amax(1, keepdim=True).clamp(min=LEAST)
    assert ((scale[:, :1] - top / 448).abs() <= 2 * U * top / 448).all() and (scale[:, 1:] == 0).all()
    # off by half a step of e4m3 at most: 2^-4 of the value, 2^-10 scales below the smallest normal code
    assert ((codes.float() * scale[:, :1] - v).abs() <= (2.0 ** -4 + 8 * U) * v.abs() + (2.0 ** -10 + 8 * U) * top / 448).all()


def test_quant_of_values_that_are_not_finite_and_of_the_smallest_and_largest():
    nan, inf = float("nan"), float("inf")
    x = rows_of(6, 256, "f32", 14)
    x[0, 3], x[0, 200] = nan, -nan
    x[1, 4], x[1, 5] = inf, -inf
    x[2, :128], x[2, 128:] = nan, inf
    x[3, :128], x[3, 128:] = 0.0, -0.0
    x[4] *= 1e-42                                   # below 2^-110
    x[5, :128], x[5, 128:] = 3.4e38, -1e-30
    y, c = quant(x)
    v = x.double()
    assert torch.equal(y.float().isnan(), x.isnan())
    clean = torch.where(v.isfinite(), v, 0.0)
    want = blocked(clean).abs().amax(2).clamp(min=LEAST)
    assert ((c - want / 448).abs() <= 2 * U * want / 448).all()
    assert y[1, 4].float() == 448 and y[1, 5].float() == -448
    ok = v.isfinite()
    t = (blocked(clean) / want[:, :, None] * 448).view(6, 256)
    got = torch.where(ok, y.double(), 0.0)
    assert ((q(t - 6 * U * t.abs()) <= got) & (got <= q(t + 6 * U * t.abs())))[ok].all()
    assert (y[3].float() == 0).all()


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------
def test_on_another_stream_and_captured():
    import dl_fusion_amd as dl
    rows, cols = 33, 4096
    x, r = rows_of(rows, cols, "bf16", 15), rows_of(rows, cols, "bf16", 16)
    side = torch.cuda.Stream()
    s0, y0, c0 = norm(x, r, None, "blocks", True)
    s1, y1, c1 = norm(x, r, None, "blocks", True, stream=side)
    assert torch.equal(s0, s1) and torch.equal(y0.view(torch.uint8), y1.view(torch.uint8)) and torch.equal(c0, c1)
    xd, rd = x.cuda(), r.cuda()
    s, y = torch.empty_like(xd), torch.empty(rows, cols, dtype=FP8, device="cuda")
    z, zs = torch.empty(rows, cols, dtype=FP8, device="cuda"), torch.empty(rows, 32, device="cuda")
    ys = torch.empty(rows, 32, device="cuda")
    dn, dq = dl.rms_norm_desc(rows, cols, EPS, "bf16", "fp8"), dl.quant_blocks_desc(rows, cols)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl.dlf_rms_norm(dn, xd, rd, None, s, y, ys)
        dl.dlf_quant_blocks(dq, s, z, zs)
    for i in range(3):
        xd.copy_(x.cuda() * (i + 1))
        for t in (s, y, z):
            t.view(torch.uint8).fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        s2, y2, c2 = norm((x * (i + 1)), r, None, "blocks", True)
        z2, zs2 = quant(s2)
        assert torch.equal(s.cpu(), s2) and torch.equal(y.cpu().view(torch.uint8), y2.view(torch.uint8))
        assert torch.equal(ys.cpu(), c2) and torch.equal(z.cpu().view(torch.uint8), z2.view(torch.uint8)) and torch.equal(zs.cpu(), zs2)


def test_two_streams_at_once():
    x, r = rows_of(2000, 4096, "bf16", 17).cuda(), rows_of(2000, 4096, "bf16", 18).cuda()
    import dl_fusion_amd as dl
    d = dl.rms_norm_desc(2000, 4096, EPS)
    outs = [(torch.empty_like(x), torch.empty_like(x)) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, (s, y) in enumerate(outs):
        dl.dlf_rms_norm(d, x, r, None, s, y, None, streams[i % 2])
    torch.cuda.synchronize()
    assert math.isfinite(float(outs[0][1].float().sum()))
    for s, y in outs[1:]:
        assert torch.equal(s, outs[0][0]) and torch.equal(y, outs[0][1])
