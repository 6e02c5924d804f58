"""CPU tests of the norm's, the block quantiser's and the block-scaled products' argument checks, and of the weights'
quantiser.  Nothing here launches a kernel: every device call is rejected, or is a zero-size no-op, before any HIP
call."""
import ctypes

import numpy as np
import pytest

dlf = pytest.importorskip("dl_fusion_amd", reason="libdlfusion.so not built")
torch = pytest.importorskip("torch")
from test_host_lib import fake_pointers  # noqa: E402

OK, INVALID, UNSUPPORTED, ALIAS = dlf.DLF_OK, dlf.DLF_ERR_INVALID_ARG, dlf.DLF_ERR_UNSUPPORTED, dlf.DLF_ERR_ALIAS
NAN, INF = float("nan"), float("inf")


def addr(i, off=0):
    """Fake device addresses, 64 GB apart, never dereferenced."""
    return (i + 1) * (64 << 30) + off


def ref(d):
    return None if d is None else ctypes.byref(d)


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------
def call_norm(x=addr(0), residual=addr(1), weight=addr(2), sum=addr(3), y=addr(4), y_scale=None, desc=True, **kw):
    args = dict(rows=4, cols=256)
    args.update(kw)
    d = dlf.rms_norm_desc(**args) if desc else None
    return dlf.raw().dlf_rms_norm(ref(d), x, residual, weight, sum, y, y_scale, None)


@fake_pointers
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=-8), INVALID), (dict(dtype=7), INVALID),
    (dict(out_dtype=-1), INVALID), (dict(dtype="fp8"), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=7e-31), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(x_stride=255), INVALID), (dict(residual_stride=255), INVALID),
    (dict(sum_stride=0), INVALID), (dict(y_stride=-256), INVALID), (dict(x_stride=(1 << 31) + 1), UNSUPPORTED),
    (dict(y_stride=(1 << 31) + 1), UNSUPPORTED), (dict(cols=(1 << 23) + 1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(out_dtype="fp8", out_inv_scale=0.0), INVALID), (dict(out_dtype="fp8", out_inv_scale=NAN), INVALID),
    (dict(out_dtype="fp8", out_inv_scale=INF), INVALID), (dict(y_scale=addr(5)), INVALID),
    (dict(y_scale=addr(5), out_dtype="fp8", y_scale_stride=1), INVALID),
    (dict(y_scale=addr(5), out_dtype="fp8", y_scale_stride=6), UNSUPPORTED),
    (dict(y_scale=addr(5), out_dtype="fp8", y_scale_stride=(1 << 20) + 4), UNSUPPORTED),
])
def test_norm_refuses_bad_descriptors(kw, status):
    assert call_norm(**kw) == status


@fake_pointers
def test_norm_refusals():
    assert call_norm(desc=False) == INVALID
    assert call_norm(x=None) == INVALID and call_norm(y=None) == INVALID
    for n in ("x", "residual", "weight", "sum", "y"):
        assert call_norm(**{n: addr(40, 8)}) == INVALID, n
        assert "aligned" in dlf.dlf_last_error()
    assert call_norm(y_scale=addr(40, 4), out_dtype="fp8") == INVALID
    # nothing to do: no tensor is looked at
    assert call_norm(rows=0, x=None, y=None) == OK
    # strides of tensors that are not there
    assert call_norm(rows=0, residual=None, sum=None, residual_stride=0, sum_stride=0) == OK
    size = 4 * 256 * 2
    assert call_norm(y=addr(0, size - 16)) == ALIAS
    assert call_norm(sum=addr(1, 16)) == ALIAS
    assert call_norm(y=addr(2)) == ALIAS
    assert call_norm(sum=addr(4, size - 16)) == ALIAS
    # an input in place: with another stride, or another type
    assert call_norm(sum=addr(0), sum_stride=264) == ALIAS
    assert call_norm(y=addr(0), out_dtype="f32") == ALIAS
    # both outputs in one input
    assert call_norm(sum=addr(0), y=addr(0)) == ALIAS
    assert call_norm(y_scale=addr(0), out_dtype="fp8") == ALIAS
    assert call_norm(y_scale=addr(4, 16), out_dtype="fp8") == ALIAS
    # in place of x, whose rows the residual overlaps in another way
    assert call_norm(sum=addr(0), residual=addr(0, 512)) == ALIAS


def test_norm_binding_checks_tensors():
    d = dlf.rms_norm_desc(4, 256)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256)
    for bad in (x.float(), x[:3], x[:, :128], torch.zeros(4, 264, dtype=torch.bfloat16)[:, :256], x.t(), x.view(-1),
                torch.zeros(4, 512, dtype=torch.bfloat16)[:, ::2]):
        for at in range(4):
            args = [x, x, x, x]
            args[at] = bad
            with pytest.raises(ValueError):
                dlf.dlf_rms_norm(d, args[0], args[1], w, args[2], args[3], None, stream=0)
    for bad in (w[:255], w.bfloat16()):
        with pytest.raises(ValueError):
            dlf.dlf_rms_norm(d, x, None, bad, None, x, None, stream=0)
    e = dlf.rms_norm_desc(4, 256, out_dtype="fp8")
    y = torch.zeros(4, 256, dtype=torch.uint8)
    for bad in (torch.zeros(13), torch.zeros(4, 4, dtype=torch.float64)):
        with pytest.raises(ValueError):
            dlf.dlf_rms_norm(e, x, None, w, None, y, bad, stream=0)


# ---------------------------------------------------------------------------
# Quantiser
# ---------------------------------------------------------------------------
def call_quant(x=addr(0), codes=addr(1), scale=addr(2), desc=True, **kw):
    args = dict(rows=4, cols=256)
    args.update(kw)
    return dlf.raw().dlf_quant_blocks(ref(dlf.quant_blocks_desc(**args) if desc else None), x, codes, scale, None)


@fake_pointers
def test_quant_refusals():
    assert call_quant(desc=False) == INVALID
    for kw in (dict(rows=-1), dict(cols=0), dict(dtype=9), dict(x_stride=255), dict(codes_stride=1), dict(row_scale_stride=1),
               dict(x=None), dict(codes=None), dict(scale=None), dict(x=addr(9, 2)), dict(codes=addr(9, 8)), dict(scale=addr(9, 4))):
        assert call_quant(**kw) == INVALID, kw
    for kw in (dict(dtype="fp8"), dict(cols=(1 << 23) + 1), dict(rows=1 << 31), dict(x_stride=(1 << 31) + 8),
               dict(row_scale_stride=7), dict(row_scale_stride=(1 << 20) + 4), dict(rows=1 << 28, cols=1024)):
        assert call_quant(**kw) == UNSUPPORTED, kw
    assert call_quant(rows=0, x=None, codes=None, scale=None) == OK
    assert call_quant(codes=addr(0, 2032)) == ALIAS
    assert call_quant(codes=addr(0)) == ALIAS
    assert call_quant(scale=addr(0, 16)) == ALIAS
    assert call_quant(scale=addr(1, 1008)) == ALIAS


def test_quant_binding_checks_tensors():
    d = dlf.quant_blocks_desc(4, 256)
    x, y, s = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 4)
    for args in ((x.float(), y, s), (x[:2], y, s), (x, x, s), (x, y[:, :128], s), (x, y, s[:3]), (x, y, s.double())):
        with pytest.raises(ValueError):
            dlf.dlf_quant_blocks(d, *args, stream=0)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------
PTRS = ("a", "a_scale", "b", "b_scale", "shift", "residual", "c")


def call_gemm(gate=None, desc=True, workspace=addr(20), workspace_bytes=1 << 40, **kw):
    p = {n: addr(i) for i, n in enumerate(PTRS)}
    p.update({n: kw.pop(n) for n in PTRS if n in kw})
    args = dict(m=4, n=256, k=512)
    args.update(kw)
    d = dlf.gemm_blocks_desc(**args) if desc else None
    if gate is None:
        return dlf.raw().dlf_gemm_blocks(ref(d), *[p[n] for n in PTRS], workspace, workspace_bytes, None)
    return dlf.raw().dlf_gemm_blocks_gated(ref(d), *[p[n] for n in PTRS[:5]], gate, p["c"], workspace, workspace_bytes, None)


BAD_GEMMS = [
    (dict(m=-1), INVALID), (dict(n=-2), INVALID), (dict(k=-16), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(k=520), UNSUPPORTED), (dict(k=8), UNSUPPORTED),
    (dict(n=(1 << 23) + 2), UNSUPPORTED), (dict(k=(1 << 23) + 16), UNSUPPORTED), (dict(m=(1 << 24) + 1), UNSUPPORTED),
    (dict(m=1 << 20, n=1 << 17), UNSUPPORTED), (dict(a_scale_stride=3), INVALID), (dict(b_scale_stride=0), INVALID),
    (dict(a_scale_stride=5), UNSUPPORTED), (dict(b_scale_stride=6), UNSUPPORTED),
    (dict(a_scale_stride=(1 << 20) + 4), UNSUPPORTED), (dict(b_scale_stride=(1 << 20) + 4), UNSUPPORTED),
]


@fake_pointers
@pytest.mark.parametrize("kw,status", BAD_GEMMS)
def test_products_refuse_bad_descriptors(kw, status):
    assert call_gemm(**kw) == status
    assert call_gemm(gate=0, **kw) == status
    size = ctypes.c_size_t(7)
    assert dlf.raw().dlf_gemm_blocks_workspace_bytes(ref(dlf.gemm_blocks_desc(**{**dict(m=4, n=256, k=512), **kw})),
                                                     ctypes.byref(size)) == status
    assert size.value == 0


@fake_pointers
def test_product_refusals():
    assert call_gemm(desc=False) == INVALID
    assert dlf.raw().dlf_gemm_blocks_workspace_bytes(ref(dlf.gemm_blocks_desc(4, 256, 512)), None) == INVALID
    for n in ("a", "a_scale", "b", "b_scale", "c"):
        assert call_gemm(**{n: None}) == INVALID, n
        assert call_gemm(gate=1, **{n: None}) == INVALID, n
    for n in PTRS:
        assert call_gemm(**{n: addr(40, 8)}) == INVALID, n
    assert call_gemm(workspace=addr(40, 8)) == INVALID
    assert call_gemm(m=0, a=None, c=None) == OK and call_gemm(n=0, b=None, c=None) == OK
    assert call_gemm(c=addr(0, 4 * 512 - 16)) == ALIAS
    assert call_gemm(c=addr(2, 256 * 512 - 16)) == ALIAS
    assert call_gemm(c=addr(1)) == ALIAS and call_gemm(c=addr(3, 16)) == ALIAS and call_gemm(c=addr(4)) == ALIAS
    assert call_gemm(c=addr(5)) == ALIAS
    # gated: two rows of scales a 256 rows
    assert call_gemm(gate=0, c=addr(3, 16)) == ALIAS
    for gate in (-1, 3):
        assert call_gemm(gate=gate) == INVALID
    assert call_gemm(gate=0, n=255) == INVALID
    assert call_gemm(gate=0, act="relu") == INVALID


@pytest.mark.parametrize("m", [0, 1, 16, 17, 32, 33, 64, 65, 200, 777, 4096, 1 << 24])
def test_workspace_sizes(m):
    """Whole fp32 outputs, rows rounded up to 4 columns, at most 8 of them; none where nothing is summed."""
    for n in (0, 1, 2, 5, 64, 300, 1024, 4096, 22016):
        for k in (0, 16, 128, 1024, 4096, 11008, 1 << 23):
            if m * n >= 1 << 37:
                continue
            size = dlf.dlf_gemm_blocks_workspace_bytes(dlf.gemm_blocks_desc(m, n, k))
            one = m * (-(-n // 4) * 4) * 4
            assert size == 0 if one == 0 else size % one == 0 and size // one <= 8 and size // one != 1
            assert size == 0 or k > 128
    assert dlf.dlf_gemm_blocks_workspace_bytes(dlf.gemm_blocks_desc(64, 4096, 11008)) > 0
    assert dlf.dlf_gemm_blocks_workspace_bytes(dlf.gemm_blocks_desc(1, 4096, 4096)) == 0


@fake_pointers
def test_product_refuses_a_bad_workspace():
    size = dlf.dlf_gemm_blocks_workspace_bytes(dlf.gemm_blocks_desc(64, 4096, 11008))
    big = dict(m=64, n=4096, k=11008)
    assert call_gemm(workspace=None, **big) == INVALID and call_gemm(workspace_bytes=size - 1, **big) == INVALID
    assert call_gemm(gate=0, workspace=None, **big) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6):
        assert call_gemm(workspace=addr(i, 256), **big) == ALIAS, i


def test_product_binding_checks_tensors():
    m, n, k = 4, 256, 512
    d = dlf.gemm_blocks_desc(m, n, k)
    fp8 = torch.float8_e4m3fn
    good = dict(a=torch.zeros(m, k, dtype=fp8), a_scale=torch.zeros(m, 4), b=torch.zeros(n, k, dtype=fp8), b_scale=torch.zeros(2, 4),
                shift=torch.zeros(n), residual=torch.zeros(m, n, dtype=torch.bfloat16), c=torch.zeros(m, n, dtype=torch.bfloat16),
                ws=None)
    bad = dict(a=[good["a"][:3], good["a"].float(), good["a"][:, :256], torch.zeros(m, 528, dtype=fp8)[:, :k]],
               a_scale=[good["a_scale"][:3], good["a_scale"].double()], b=[good["b"][:255], good["b"].bfloat16()],
               b_scale=[good["b_scale"][:1]], shift=[good["shift"][:9]], residual=[good["residual"].float(), good["residual"][:, :9]],
               c=[good["c"].float(), good["c"][:3]], ws=[torch.zeros(2, dtype=torch.uint8)])
    for name, tensors in bad.items():
        for t in tensors:
            p = dict(good, **{name: t})
            with pytest.raises(ValueError):
                dlf.dlf_gemm_blocks(d, *[p[x] for x in PTRS], p["ws"], 64, stream=0)
            if name == "residual":
                continue
            with pytest.raises(ValueError):
                dlf.dlf_gemm_blocks_gated(d, *[p[x] for x in PTRS[:5]], "silu", t if name == "c" else p["c"][:, :128].contiguous(),
                                          p["ws"], 64, stream=0)


# ---------------------------------------------------------------------------
# Weights
# ---------------------------------------------------------------------------
def definition(w, gated):
    """Codes' values and scales: every e4m3 value is looked at, the nearest taken, the even one of two."""
    values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    n, k = w.shape
    row = np.arange(n)
    slab = 2 * (row // 256) + row % 2 if gated else row // 128
    codes, scale = np.zeros((n, k), np.uint8), np.zeros((slab.max() + 1, dlf.scale_stride(k)), np.float32)
    for s in range(slab.max() + 1):
        at = np.nonzero(slab == s)[0]
        for t in range(-(-k // 128)):
            block = w[at, 128 * t:128 * t + 128].astype(np.float64)
            scale[s, t] = np.float32(max(np.abs(block).max(), 2.0 ** -110) / 448)
            v = np.minimum(np.abs(block) / np.float64(scale[s, t]), 448)
            off = np.abs(v[..., None] - values)
            near = off.min(-1, keepdims=True) == off
            best = np.where(near & (np.arange(127) % 2 == 0), 0, np.where(near, 1, 2)).argmin(-1)
            codes[at[:, None], 128 * t + np.arange(block.shape[1])] = best + 128 * np.signbit(block)
    return codes, scale


@pytest.mark.parametrize("n,k,gated", [(1, 1, False), (3, 130, False), (130, 64, False), (129, 257, False), (2, 16, True),
                                       (258, 40, True), (512, 130, True)])
def test_weights(n, k, gated):
    w = (np.random.RandomState(n + k).randn(n, k) * np.exp(np.random.RandomState(5).randn(n, 1))).astype(np.float32)
    w[0, 0] = 0.0
    codes, scale = dlf.dlf_quant_blocks_weights(w, gated)
    want_codes, want_scale = definition(w, gated)
    assert np.array_equal(scale, want_scale)
    assert np.array_equal(codes, want_codes)


def test_weights_at_every_code_and_between():
    """A block whose scale is 1: every e4m3 value comes back as itself, halfway points go to the even code."""
    values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    half = (values[:-1] + values[1:]) / 2
    w = np.zeros((2, 256), np.float32)
    w[0, :127], w[1, :127] = values, -values
    w[0, 128:254], w[1, 128:254] = half, -half
    w[0, 255] = 448
    codes, scale = dlf.dlf_quant_blocks_weights(w)
    assert (scale[0, :2] == 1).all()
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(126) + 1)
    assert np.array_equal(codes[0, :127], np.arange(127)) and np.array_equal(codes[0, 128:254], even)
    assert np.array_equal(codes[1, 128:254], even + 128) and np.array_equal(codes[1, 1:127], np.arange(1, 127) + 128)


def test_weights_refusals():
    raw = dlf.raw().dlf_quant_blocks_weights
    w = np.ones((4, 256), np.float32)
    codes, scale = np.full((4, 256), 7, np.uint8), np.full((1, 4), 7.0, np.float32)
    p = [x.ctypes.data for x in (w, codes, scale)]
    for args in ((-1, 256, p[0], 0, 4), (4, -1, p[0], 0, 4), (4, 256, None, 0, 4), (4, 256, p[0], 2, 4), (3, 256, p[0], 1, 4),
                 (4, 256, p[0], 0, 1), (4, 256, p[0], 0, 6)):
        assert raw(*args, p[1], p[2]) == INVALID, args
    assert raw(4, 256, p[0], 0, 4, None, p[2]) == INVALID and raw(4, 256, p[0], 0, 4, p[1], None) == INVALID
    assert raw(4, 256, p[0], 0, 4, p[0], p[2]) == ALIAS and raw(4, 256, p[0], 0, 4, p[1], p[1]) == ALIAS
    for bad in (NAN, INF, -INF):
        w[3, 255] = bad
        assert raw(4, 256, p[0], 0, 4, p[1], p[2]) == INVALID
    assert (codes == 7).all() and (scale == 7).all()
    assert raw(0, 256, None, 0, 4, None, None) == OK


def test_weights_of_zeros():
    codes, scale = dlf.dlf_quant_blocks_weights(np.zeros((2, 16), np.float32))
    assert (codes == 0).all() and scale[0, 0] == np.float32(2.0 ** -110 / 448) and (scale[0, 1:] == 0).all()


# ---------------------------------------------------------------------------
# The feed-forward block's weights
# ---------------------------------------------------------------------------
def test_feed_forward_packs_and_refuses():
    from dl_fusion_amd.feed_forward import GatedFeedForward, pack, pack_gate_up
    r = np.random.RandomState(0)
    gate, up, down = (r.randn(*s).astype(np.float32) for s in ((300, 256), (300, 256), (256, 304)))
    codes, scale = pack_gate_up(gate, up, "cpu")
    # row j of the gate is row 2j, of the up weight row 2j + 1, each with the scale that it has alone
    for w, first in ((gate, 0), (up, 1)):
        c, s = dlf.dlf_quant_blocks_weights(w)
        assert torch.equal(codes.view(torch.uint8)[first::2], torch.from_numpy(c)) and torch.equal(scale[first::2], torch.from_numpy(s))
    with pytest.raises(ValueError):
        pack_gate_up(gate, up[:299], "cpu")
    down = pack(down[:, :300 // 16 * 16], "cpu")
    small = pack_gate_up(gate[:288], up[:288], "cpu")
    GatedFeedForward(small, down)
    for bad in (dict(gate_up=down), dict(down=small), dict(norm=torch.ones(255)), dict(norm=torch.ones(256).double()),
                dict(gate_up=(small[0], small[1][:1])), dict(gate_up=(small[0].view(torch.uint8), small[1]))):
        with pytest.raises(ValueError):
            GatedFeedForward(**{**dict(gate_up=small, down=down), **bad})
