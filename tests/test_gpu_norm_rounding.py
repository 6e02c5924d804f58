"""How often the root-mean-square norm rounds, on rows whose sums of squares are exact: whole numbers, at most 2^24 in all.

With u = 2^-24: the mean and eps are added in 64 bits, their root's reciprocal is rounded to fp32 once (u of it, and less than
2^-40 from 64 bits), and so is the product by a value (u), none where the value is a power of two.  Bounds, derived before any
run: u (1 + 2^-10) for those, 2 u (1 + 2^-10) for all."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24 * (1 + 2.0 ** -10)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("eps", [2.0 ** -100, 1e-5, 0.375])
@pytest.mark.parametrize("rows,cols", [(4000, 5), (4000, 64), (3000, 1000), (2000, 2048), (1000, 4100), (300, 9000), (100, 20000)])
def test_the_root_and_its_reciprocal_are_rounded_once(rows, cols, eps):
    import dl_fusion_amd as dl
    g = torch.Generator().manual_seed(cols)
    x = torch.randint(-9, 10, (rows, cols), generator=g).float() * torch.randint(0, 2, (rows, 1), generator=g).mul(2).add(1)
    x[:, 0] = 1
    x = x.cuda()
    y = torch.empty_like(x)
    d = dl.rms_norm_desc(rows, cols, eps, "f32", "f32")
    dl.dlf_rms_norm(d, x, None, None, None, y, None)
    v = x.double()
    want = v / (v.square().mean(1, keepdim=True) + d.eps).sqrt()
    off = (y - want).abs()
    power = v.abs().log2().frac() == 0
    assert power[:, 0].all()
    assert (off <= U * want.abs())[power].all()
    assert (off <= 2 * U * want.abs()).all()


@pytest.mark.parametrize("cols", [1, 6, 40, 520, 4096, 20000])
@pytest.mark.parametrize("eps", [1e30, 1e37, 3e38])
def test_an_eps_beside_squares_past_the_range(cols, eps):
    """Rows of sums up to and past fp32's range, and an eps that counts beside their mean.  A sum is a chain of at most cols / 64
    + 40 additions, which the root halves; 3 u for its rounding, the product and the squares."""
    import dl_fusion_amd as dl
    g = torch.Generator().manual_seed(cols)
    x = (torch.rand(12, cols, generator=g) + 1) * torch.logspace(14, 20, 12)[:, None]
    x = x.cuda()
    y = torch.empty_like(x)
    d = dl.rms_norm_desc(12, cols, eps, "f32", "f32")
    dl.dlf_rms_norm(d, x, None, None, None, y, None)
    v = x.double()
    want = v / (v.square().mean(1, keepdim=True) + d.eps).sqrt()
    assert ((y - want).abs() <= ((cols / 64 + 40) / 2 + 3) * U * want).all(), (y / want - 1).abs().max(1).values.tolist()


@pytest.mark.parametrize("cols", [16392, 131080, (1 << 20) + 5, 1 << 23])
@pytest.mark.parametrize("value", [1.1, 0.7, 1e16])
def test_rows_of_one_value_however_long(cols, value):
    """Sums that round the same way again and again.  A chunk of 8 squares is off by 8 u at most, a thread's sum of chunks
    by u, the joins of 64 lanes and 16 waves by 22 u, the root halves it; 3 u for its rounding and the product.  (1e16: the longest
    rows pass fp32's range, and are taken 2^-80 times as large, which is exact.)"""
    import dl_fusion_amd as dl
    x = torch.full((2, cols), value, device="cuda")
    y = torch.empty_like(x)
    d = dl.rms_norm_desc(2, cols, 1e-5, "f32", "f32")
    dl.dlf_rms_norm(d, x, None, None, None, y, None)
    v = float(x[0, 0])
    want = v / (v * v + d.eps) ** 0.5
    off = float((y.double() - want).abs().max()) / want
    assert off <= (31 / 2 + 3) * U, off * 2 ** 24
