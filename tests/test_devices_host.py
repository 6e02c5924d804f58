"""CPU tests of the binding's check that all tensors of a call are on the device that the call runs on.  The tensor in question
is on the host, all others are raw addresses that nothing reads: the call has to end before it reaches the library."""
import pytest

dlf = pytest.importorskip("dl_fusion_amd", reason="libdlfusion.so not built")
torch = pytest.importorskip("torch")

FP8, BF16 = torch.float8_e4m3fn, torch.bfloat16
M, N, K = 4, 256, 512
ROWS = dict(x=torch.zeros(M, K, dtype=BF16), residual=torch.zeros(M, K, dtype=BF16), weight=torch.zeros(K),
            sum=torch.zeros(M, K, dtype=BF16), y=torch.zeros(M, K, dtype=FP8), y_scale=torch.zeros(M, 4))
QUANT = dict(x=ROWS["x"], codes=ROWS["y"], scale=ROWS["y_scale"])
PRODUCT = dict(a=torch.zeros(M, K, dtype=FP8), a_scale=torch.zeros(M, 4), b=torch.zeros(N, K, dtype=FP8), b_scale=torch.zeros(2, 4),
               col_shift=torch.zeros(N), residual=torch.zeros(M, N, dtype=BF16), c=torch.zeros(M, N, dtype=BF16),
               workspace=torch.zeros(64, dtype=torch.uint8))
GATED = {n: t for n, t in PRODUCT.items() if n != "residual"}
GATED["c"] = torch.zeros(M, N // 2, dtype=BF16)


def norm(stream, p):
    d = dlf.rms_norm_desc(M, K, out_dtype="fp8")
    dlf.dlf_rms_norm(d, p["x"], p["residual"], p["weight"], p["sum"], p["y"], p["y_scale"], stream=stream)


def quant(stream, p):
    dlf.dlf_quant_blocks(dlf.quant_blocks_desc(M, K), p["x"], p["codes"], p["scale"], stream=stream)


def product(stream, p):
    dlf.dlf_gemm_blocks(dlf.gemm_blocks_desc(M, N, K), *[p[n] for n in PRODUCT], 64, stream=stream)


def gated(stream, p):
    dlf.dlf_gemm_blocks_gated(dlf.gemm_blocks_desc(M, N, K), *[p[n] for n in ("a", "a_scale", "b", "b_scale", "col_shift")], "silu",
                              p["c"], p["workspace"], 64, stream=stream)


class Stream:
    """What torch.cuda.Stream has."""
    device, cuda_stream = torch.device("cuda", 0), 0


class Reached(Exception):
    pass


@pytest.fixture
def library(monkeypatch):
    def reached(*_):
        raise Reached
    for n in ("dlf_rms_norm", "dlf_quant_blocks", "dlf_gemm_blocks", "dlf_gemm_blocks_gated"):
        monkeypatch.setattr(dlf._lib, n, reached)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda _: 0, raising=False)


CASES = [(f, n, t) for f, ts in ((norm, ROWS), (quant, QUANT), (product, PRODUCT), (gated, GATED)) for n, t in ts.items()]


@pytest.mark.parametrize("stream", [None, 0, Stream()], ids=["current", "handle", "stream"])
@pytest.mark.parametrize("call,name,tensor", CASES, ids=[f"{f.__name__}-{n}" for f, n, _ in CASES])
def test_a_tensor_of_the_host_is_refused(library, call, name, tensor, stream):
    names = {norm: ROWS, quant: QUANT, product: PRODUCT, gated: GATED}[call]
    raw = {n: 4096 * (i + 1) for i, n in enumerate(names)}
    with pytest.raises(Reached):
        call(stream, raw)
    with pytest.raises(ValueError, match=f"{name} is on cpu"):
        call(stream, dict(raw, **{name: tensor}))


class OnDevice:
    """A tensor as the binding looks at one, on a device of our choice."""

    def __init__(self, t, device):
        self._t, self._device = t, device
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("stream", [None, 0, Stream()], ids=["current", "handle", "stream"])
@pytest.mark.parametrize("call,name,tensor", CASES, ids=[f"{f.__name__}-{n}" for f, n, _ in CASES])
def test_a_tensor_of_another_device_is_refused(library, call, name, tensor, stream):
    names = {norm: ROWS, quant: QUANT, product: PRODUCT, gated: GATED}[call]
    here = {n: OnDevice(t, 0) for n, t in names.items()}
    with pytest.raises(Reached):
        call(stream, here)
    with pytest.raises(ValueError, match="is on cuda:"):
        call(stream, dict(here, **{name: OnDevice(tensor, 1)}))


@pytest.mark.parametrize("call", [norm, quant, product, gated])
def test_all_tensors_on_another_device_than_the_stream_s(library, call):
    names = {norm: ROWS, quant: QUANT, product: PRODUCT, gated: GATED}[call]
    there = {n: OnDevice(t, 1) for n, t in names.items()}
    for stream in (None, Stream()):
        with pytest.raises(ValueError, match="is on cuda:1, the call runs on cuda:0"):
            call(stream, there)
    with pytest.raises(Reached):            # a handle may be any device's
        call(0, there)


@pytest.mark.parametrize("part", ["gate and up codes", "gate and up scales", "down scales", "norm"])
def test_a_feed_forward_block_s_weights_are_on_one_device(part):
    from dl_fusion_amd.feed_forward import GatedFeedForward, pack, pack_gate_up
    w = torch.ones(32, 16).numpy()
    gate_up, down, norm = pack_gate_up(w, w, "cpu"), pack(w.T.copy(), "cpu"), torch.ones(16)
    GatedFeedForward(gate_up, down, norm)
    off = lambda t: t.to("meta")  # noqa: E731
    bad = {"gate and up codes": dict(gate_up=(off(gate_up[0]), gate_up[1])), "gate and up scales": dict(gate_up=(gate_up[0], off(gate_up[1]))),
           "down scales": dict(down=(down[0], off(down[1]))), "norm": dict(norm=off(norm))}[part]
    with pytest.raises(ValueError, match=part):
        GatedFeedForward(**{**dict(gate_up=gate_up, down=down, norm=norm), **bad})
