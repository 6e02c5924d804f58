"""Tensors of the host among those of the GPU are refused before anything is launched, whichever of a call's they are, on the
current stream, another one and a raw handle; the same call without them gives what it gave."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from test_devices_host import GATED, PRODUCT, QUANT, ROWS, gated, norm, product, quant  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("call,tensors,out", [(norm, ROWS, "y"), (quant, QUANT, "codes"), (product, PRODUCT, "c"), (gated, GATED, "c")])
def test_one_tensor_on_the_host(call, tensors, out):
    g = torch.Generator().manual_seed(1)
    here = {n: (torch.rand(t.shape, generator=g) + 0.5).to(t.dtype).cuda() for n, t in tensors.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for stream in (None, side, side.cuda_stream, 0):
        for name in tensors:
            with pytest.raises(ValueError, match=f"{name} is on cpu"):
                call(stream, dict(here, **{name: here[name].cpu()}))
        here[out].view(torch.uint8).fill_(0)
        torch.cuda.synchronize()
        call(stream, here)
        torch.cuda.synchronize()
        got.append(here[out].clone())
    assert got[0].float().abs().sum() > 0
    assert all(torch.equal(g.view(torch.uint8), got[0].view(torch.uint8)) for g in got)
