"""The norm and the block quantiser where their loads and stores are non-temporal (from 64 MB of them on), at each width of a
row's workgroup, types, parts, strides and in place.  Bounds: those that test_gpu_row_blocks.py derives."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from test_gpu_row_blocks import EPS, FP8, U, check_blocks, definition, dtype_of, guarded, q, untouched  # noqa: E402

STREAM = 64 << 20
WIDTHS = [5, 130, 512, 1000, 2047, 4096, 4099, 8192, 16380, 20003]      # threads a row: 64 .. 1024, and rows that are read twice


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def rows_of(rows, cols, dtype, seed, more=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + more, generator=g, device="cuda") * torch.exp(3 * torch.rand(rows, 1, generator=g, device="cuda"))
    x[:, ::13] *= 30
    return x.to(dtype_of(dtype))[:, :cols]


def rows_for(cols, dtype, out, tensors):
    size = (4 if dtype == "f32" else 2) * tensors + {"f32": 4, "bf16": 2}.get(out, 1)
    rows = -(-STREAM // (cols * size)) + 2
    assert rows * cols * size >= STREAM > (rows - 3) * cols * size
    return rows


def norm_check(cols, dtype, out, residual, want_sum, strides=(0, 0, 0, 0)):
    import dl_fusion_amd as dl
    rows = rows_for(cols, dtype, out, 1 + residual + want_sum)
    x = rows_of(rows, cols, dtype, 1, strides[0])
    r = rows_of(rows, cols, dtype, 2, strides[1]) if residual else None
    w = torch.randn(cols, generator=torch.Generator().manual_seed(3)).cuda()
    sbuf, s = guarded(rows, cols + strides[2], dtype_of(dtype))
    ybuf, y = guarded(rows, cols + strides[3], FP8 if out in ("static", "blocks") else dtype_of(out))
    blocks, stride = -(-cols // 128), dl.scale_stride(cols)
    cbuf, c = guarded(rows, stride, torch.float32)
    inv = 20.0
    d = dl.rms_norm_desc(rows, cols, EPS, dtype, "fp8" if out in ("static", "blocks") else out, inv, *[cols + m for m in strides], stride)
    dl.dlf_rms_norm(d, x, r, w, s[:, :cols] if want_sum else None, y[:, :cols], c if out == "blocks" else None)
    assert untouched(sbuf, s, cols if want_sum else 0) and untouched(ybuf, y, cols) and untouched(cbuf, c, blocks if out == "blocks" else 0)
    e = (cols / 64 / 2 + 20 + 9) * U
    for at in range(0, rows, 4096):         # 64 bits of a part of the rows
        part = slice(at, at + 4096)
        h, want = definition(x[part], r[part] if residual else None, w)
        if want_sum:
            assert ((s[part, :cols].double() - h).abs() <= (U + (2.0 ** -8 if dtype == "bf16" else 0)) * h.abs()).all()
        got = y[part, :cols]
        if out == "blocks":
            check_blocks(want, got, c[part, :blocks], e)
        elif out == "static":
            t, off = want * inv, e + 2 * U
            assert ((q(t - off * t.abs()) <= got.double()) & (got.double() <= q(t + off * t.abs()))).all()
        else:
            assert ((got.double() - want).abs() <= (e + (2.0 ** -8 if out == "bf16" else 0)) * want.abs()).all()


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype,out,residual,want_sum", [("bf16", "blocks", True, True), ("bf16", "bf16", False, False),
                                                         ("f32", "f32", True, False), ("bf16", "static", False, True)])
def test_norm(cols, dtype, out, residual, want_sum):
    norm_check(cols, dtype, out, residual, want_sum)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype,out", [("bf16", "blocks"), ("f32", "bf16")])
def test_norm_strides(cols, dtype, out):
    norm_check(cols, dtype, out, True, True, (1, 3, 5, 7))


@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_in_place(cols):
    import dl_fusion_amd as dl
    rows = rows_for(cols, "bf16", "bf16", 3)
    x, r = rows_of(rows, cols, "bf16", 4), rows_of(rows, cols, "bf16", 5)
    x0, r0 = x.clone(), r.clone()
    s0, y0 = torch.empty_like(x0), torch.empty_like(x0)
    d = dl.rms_norm_desc(rows, cols, EPS)
    dl.dlf_rms_norm(d, x0, r0, None, s0, y0, None)
    assert not torch.equal(s0, y0)
    for s, y in ((x, r), (r, x)):
        x.copy_(x0)
        r.copy_(r0)
        dl.dlf_rms_norm(d, x, r, None, s, y, None)
        assert torch.equal(s, s0) and torch.equal(y, y0)


def test_norm_gives_the_same_bits_as_of_few_rows():
    import dl_fusion_amd as dl
    for cols in WIDTHS:
        rows = rows_for(cols, "bf16", "blocks", 1)
        x = rows_of(rows, cols, "bf16", 6)
        y, c = torch.empty(rows, cols, dtype=FP8, device="cuda"), torch.empty(rows, dl.scale_stride(cols), device="cuda")
        dl.dlf_rms_norm(dl.rms_norm_desc(rows, cols, EPS, "bf16", "fp8"), x, None, None, None, y, c)
        few = [0, rows // 2, rows - 1]
        y1, c1 = torch.empty(3, cols, dtype=FP8, device="cuda"), torch.empty(3, dl.scale_stride(cols), device="cuda")
        dl.dlf_rms_norm(dl.rms_norm_desc(3, cols, EPS, "bf16", "fp8"), x[few].contiguous(), None, None, None, y1, c1)
        blocks = -(-cols // 128)
        assert torch.equal(y[few].view(torch.uint8), y1.view(torch.uint8)) and torch.equal(c[few][:, :blocks], c1[:, :blocks])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [(0, 0, 0), (1, 3, 4)])
@pytest.mark.parametrize("cols", [8, 100, 128, 129, 1000, 4096, 11008, 65537])
def test_quant(cols, more, dtype):
    import dl_fusion_amd as dl
    blocks = -(-cols // 128)
    rows = -(-STREAM // (blocks * 128 * (5 if dtype == "f32" else 3))) + 1
    x = rows_of(rows, cols, dtype, 7, more[0])
    ybuf, y = guarded(rows, cols + more[1], FP8)
    stride = dl.scale_stride(cols) + more[2]
    cbuf, c = guarded(rows, stride, torch.float32)
    dl.dlf_quant_blocks(dl.quant_blocks_desc(rows, cols, dtype, cols + more[0], cols + more[1], stride), x, y[:, :cols], c)
    assert untouched(ybuf, y, cols) and untouched(cbuf, c, blocks)
    for at in range(0, rows, 4096):
        part = slice(at, at + 4096)
        check_blocks(x[part].double(), y[part, :cols], c[part, :blocks], 0.0)
