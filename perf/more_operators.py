"""The operators of an 8-bit transformer layer with block scales, as cases that can be timed and compared.

Three operators: the root-mean-square norm with the residual's addition and an output in bf16, fp32 or e4m3, the
quantiser of rows into e4m3 with a scale for each 128 values, and the product of matrices that are held so (weights
with a scale for each 128 x 128 values), with its epilogue.

``run`` computes them in plain torch operations where ``own`` is false, and by the package's entry points
where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
BLOCK = 128
LEAST = 2.0 ** -110                 # a block's largest magnitude is taken as at least this
EPS = 1e-5
Y_SCALE = 0.0625                    # static scale of a norm's e4m3 output


# ----------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's token before a bf16 projection: the smallest call, all latency
        dict(name="norm one token", op="norm", rows=1, cols=4096, wide=0, dtype="bf16", residual=True, out="bf16"),
        # a decode batch before an 8-bit projection
        dict(name="norm decode batch 8-bit", op="norm", rows=64, cols=4096, wide=0, dtype="bf16", residual=True,
             out="blocks"),
        # prompts before an 8-bit projection
        dict(name="norm prompts 8-bit", op="norm", rows=8192, cols=4096, wide=0, dtype="bf16", residual=True,
             out="blocks"),
        # an fp32 stream of odd width, whose rows start at any address
        dict(name="norm odd width fp32", op="norm", rows=4099, cols=1023, wide=0, dtype="f32", residual=False, out="f32"),
        # a decode batch's activations before the second product of a feed-forward block
        dict(name="quantise decode batch", op="quant", rows=64, cols=11008, wide=0, dtype="bf16"),
        # the same of prompts
        dict(name="quantise prompts", op="quant", rows=8192, cols=11008, wide=0, dtype="bf16"),
        # one user's token through an output projection: the weights are read once
        dict(name="product one token", op="product", m=1, n=4096, k=4096, gate="none", act="none", shift=False,
             residual=True),
        # a decode batch through gate and up projections
        dict(name="product decode gated", op="product", m=64, n=22016, k=4096, gate="silu", act="none", shift=False,
             residual=False),
        # and back through the down projection: few columns, a long sum
        dict(name="product decode down", op="product", m=64, n=4096, k=11008, gate="none", act="none", shift=False,
             residual=True),
        # a short prompt, sizes that end inside tiles and blocks, bias and GELU
        dict(name="product ragged", op="product", m=777, n=5000, k=4112, gate="none", act="gelu_tanh", shift=True,
             residual=False),
        # prompts through gate and up projections: the matrix cores' rate
        dict(name="product prompts gated", op="product", m=8192, n=22016, k=4096, gate="silu", act="none", shift=False,
             residual=False),
        # and back
        dict(name="product prompts down", op="product", m=8192, n=4096, k=11008, gate="none", act="none", shift=False,
             residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "product", "product", "product"])
    if op != "product":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # heads of 64 to streams of 16384, some of odd width; at most 2^26 values
        cols = rng.choice([8 * _log(rng, 8, 2048), 128 * _log(rng, 1, 128), _log(rng, 64, 16384)])
        rows = _log(rng, 1, min(65536, (1 << 26) // cols))
        wide = cols + 8 * _log(rng, 1, 512) if rng.random() < 0.25 and rows * cols <= (1 << 25) else 0
        if op == "quant":
            return dict(op=op, rows=rows, cols=cols, wide=wide, dtype=dtype)
        return dict(op=op, rows=rows, cols=cols, wide=wide, dtype=dtype, residual=rng.random() < 0.7,
                    out=rng.choice([dtype, "bf16", "static", "blocks", "blocks"]))
    gate = rng.choice(["none", "none", "none", "silu", "gelu_tanh", "gelu_erf"])
    k = rng.choice([16 * _log(rng, 1, 1024), 128 * _log(rng, 1, 128)])
    n = rng.choice([2 * _log(rng, 1, 11008), 128 * _log(rng, 1, 172)])
    m = rng.choice([_log(rng, 1, 64), _log(rng, 1, 8192)])
    while m * n * k > (1 << 38) or n * k > (1 << 27):
        m, n = max(1, m * 3 // 4), max(2, n * 3 // 8 * 2)
    plain = gate == "none"
    return dict(op=op, m=m, n=n, k=k, gate=gate, act=rng.choice(["none", "none", "relu", "gelu_tanh", "gelu_erf"]) if plain
                else "none", shift=rng.random() < 0.4, residual=plain and rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
def _blocks(cols):
    return -(-cols // BLOCK)


def _stride(cols):
    return -(-_blocks(cols) // 4) * 4       # a row of scales is a whole number of 16 bytes


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _stream(rows, cols, wide, dtype, g):
    """Values as a residual stream has them: normal, every 97th channel 20 times as large, and rows of
    different size; as a column block of rows of `wide` values where that is given."""
    x = torch.randn((rows, wide or cols), generator=g, device=DEV)
    x *= torch.rand((rows, 1), generator=g, device=DEV).mul_(3).exp_()
    x[:, 13::97] *= 20
    x = x.to(_dtype(dtype))
    return x[:, 8:8 + cols] if wide else x


def _codes(x, scale):
    return (x / scale).clamp_(-448, 448).to(FP8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] != "product":
        rows, cols = case["rows"], case["cols"]
        s = dict(case, x=_stream(rows, cols, case["wide"], case["dtype"], g))
        out = case.get("out", "blocks")
        s["scale"] = torch.zeros((rows, _stride(cols)), device=DEV) if out == "blocks" else None
        s["y"] = torch.empty((rows, cols), dtype=FP8 if out in ("blocks", "static") else _dtype(out), device=DEV)
        if case["op"] == "norm":
            s["residual"] = _stream(rows, cols, 0, case["dtype"], g) if case["residual"] else None
            s["sum"] = torch.empty((rows, cols), dtype=_dtype(case["dtype"]), device=DEV) if case["residual"] else None
            s["weight"] = torch.randn(cols, generator=g, device=DEV).mul_(0.2).add_(1)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    gated = case["gate"] != "none"
    # activations and weights as their quantisers leave them: the largest value of a block is 448 scales
    a = torch.zeros((m, _blocks(k) * BLOCK), device=DEV)
    a[:, :k] = torch.randn((m, k), generator=g, device=DEV) * torch.rand((1, k), generator=g, device=DEV).mul_(2).exp_()
    a = a.view(m, -1, BLOCK)
    sa = a.abs().amax(2).clamp_(min=LEAST) / 448
    a_scale = torch.zeros((m, _stride(k)), device=DEV)
    a_scale[:, :_blocks(k)] = sa
    codes = _codes(a, sa[:, :, None]).view(m, -1)[:, :k].contiguous()
    # rows of one scale: 128 neighbours, or every second one of 256 where gate and up alternate
    tall = _blocks(n) * BLOCK if not gated else -(-n // (2 * BLOCK)) * 2 * BLOCK
    b = torch.zeros((tall, _blocks(k) * BLOCK), device=DEV)
    b[:n, :k] = torch.randn((n, k), generator=g, device=DEV).mul_(k ** -0.5)
    b = b.view((-1, 1, BLOCK) + (_blocks(k), BLOCK)) if not gated else b.view((-1, BLOCK, 2) + (_blocks(k), BLOCK)).transpose(1, 2)
    sb = b.abs().amax((2, 4)).clamp_(min=LEAST) / 448
    b = _codes(b, sb[:, :, None, :, None])
    b = b.view(torch.uint8)
    b = (b.transpose(1, 2) if gated else b).reshape(tall, -1)[:n, :k].contiguous().view(FP8)
    b_scale = torch.zeros((tall // BLOCK, _stride(k)), device=DEV)
    b_scale[:, :_blocks(k)] = sb.reshape(tall // BLOCK, -1)
    width = n // 2 if gated else n
    return dict(case, a=codes, a_scale=a_scale, b=b, b_scale=b_scale,
                bias=torch.randn(n, generator=g, device=DEV) if case["shift"] else None,
                residual=torch.randn((m, n), generator=g, device=DEV).to(torch.bfloat16) if case["residual"] else None,
                c=torch.empty((m, width), dtype=torch.bfloat16, device=DEV))


# ----------------------------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------------------------
def _plain_store(s, y):
    """y into the output: rounded, by the static scale, or by each block's own."""
    out = s.get("out", "blocks")
    if out == "static":
        s["y"].copy_((y * (1 / Y_SCALE)).clamp(-448, 448).to(FP8))
    elif out != "blocks":
        s["y"].copy_(y)
    else:
        rows, cols = y.shape
        wide = torch.nn.functional.pad(y, (0, _blocks(cols) * BLOCK - cols)).view(rows, -1, BLOCK)
        amax = wide.abs().amax(2).clamp(min=LEAST)
        s["scale"][:, :_blocks(cols)] = amax / 448
        s["y"].copy_((wide * (448 / amax)[:, :, None]).clamp(-448, 448).view(rows, -1)[:, :cols].to(FP8))


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
        s["sum"].copy_(h)
    _plain_store(s, h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"])


def _plain_quant(s):
    _plain_store(s, s["x"].float())


def _plain_act(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "gelu_erf":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v


def _plain_product(s):
    n, k = s["n"], s["k"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    r = torch.arange(n, device=DEV)
    row = r // BLOCK if s["gate"] == "none" else 2 * (r // (2 * BLOCK)) + r % 2
    b = s["b"].float() * s["b_scale"].repeat_interleave(BLOCK, 1)[row, :k]
    v = a @ b.t()
    if s["bias"] is not None:
        v = v + s["bias"]
    if s["gate"] != "none":
        s["c"].copy_(_plain_act(s["gate"], v[:, 0::2]) * v[:, 1::2])
        return
    if s["residual"] is not None:
        v = v + s["residual"].float()
    s["c"].copy_(_plain_act(s["act"], v))


# ----------------------------------------------------------------------------------------------
# The package's entry points
# ----------------------------------------------------------------------------------------------
def _own(s):
    import dl_fusion_amd as dlf
    d = s.get("desc")                       # descriptors and workspaces are kept, as a program keeps them
    if s["op"] == "norm":
        if d is None:
            out = "fp8" if s["out"] in ("static", "blocks") else s["out"]
            d = s["desc"] = dlf.rms_norm_desc(s["rows"], s["cols"], EPS, s["dtype"], out, out_inv_scale=1 / Y_SCALE,
                                              x_stride=s["x"].stride(0))
        dlf.dlf_rms_norm(d, s["x"], s["residual"], s["weight"], s["sum"], s["y"], s["scale"])
        return
    if s["op"] == "quant":
        if d is None:
            d = s["desc"] = dlf.quant_blocks_desc(s["rows"], s["cols"], s["dtype"], x_stride=s["x"].stride(0))
        dlf.dlf_quant_blocks(d, s["x"], s["y"], s["scale"])
        return
    if d is None:
        d = s["desc"] = dlf.gemm_blocks_desc(s["m"], s["n"], s["k"], s["act"])
        s["ws"] = torch.empty(dlf.dlf_gemm_blocks_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    if s["gate"] != "none":
        dlf.dlf_gemm_blocks_gated(d, s["a"], s["a_scale"], s["b"], s["b_scale"], s["bias"], s["gate"], s["c"], s["ws"],
                                  s["ws"].numel())
    else:
        dlf.dlf_gemm_blocks(d, s["a"], s["a_scale"], s["b"], s["b_scale"], s["bias"], s["residual"], s["c"], s["ws"],
                            s["ws"].numel())


_PLAIN = {"norm": _plain_norm, "quant": _plain_quant, "product": _plain_product}


def run(state):
    (_own if own else _PLAIN[state["op"]])(state)
    if state["op"] == "product":
        return state["c"]
    got = {"y": state["y"]}
    if state["scale"] is not None:
        got["scale"] = state["scale"][:, :_blocks(state["cols"])]
    if state.get("sum") is not None:
        got["sum"] = state["sum"]
    return got


# ----------------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------------
def work(case):
    if case["op"] != "product":
        rows, cols = case["rows"], case["cols"]
        size = 4 if case["dtype"] == "f32" else 2
        out = case.get("out", "blocks")
        moved = rows * cols * (size * (3 if case.get("residual") else 1) + {"f32": 4, "bf16": 2}.get(out, 1))
        moved += 4 * rows * _blocks(cols) if out == "blocks" else 0
        return {"bytes": moved + (4 * cols if case["op"] == "norm" else 0),
                "flops": rows * cols * (5 if case["op"] == "norm" else 2)}
    m, n, k = case["m"], case["n"], case["k"]
    width = n if case["gate"] == "none" else n // 2
    return {"bytes": (m + n) * k + 4 * (m + _blocks(n)) * _blocks(k) + 2 * m * width
            + (2 * m * n if case["residual"] else 0) + (4 * n if case["shift"] else 0), "flops": 2 * m * n * k}


# ----------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------------------------
def _exact_blocks(v):
    """Codes and scales of rows in 64 bits; the last block may be short."""
    codes, scales = [], []
    for block in v.split(BLOCK, 1):
        top = block.abs().max(1, keepdim=True).values.clamp(min=LEAST)
        scales.append(top / 448)
        codes.append((block / top * 448).clamp(-448, 448).to(FP8).double())
    return torch.cat(codes, 1), torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] != "product":
        v, got = s["x"].to(f64), {}
        if case["op"] == "norm":
            if s["residual"] is not None:
                v = got["sum"] = v + s["residual"].to(f64)
            v = v / ((v * v).sum(1, keepdim=True) / case["cols"] + EPS).sqrt() * s["weight"].to(f64)
        out = case.get("out", "blocks")
        if out == "blocks":
            got["y"], got["scale"] = _exact_blocks(v)
        else:
            got["y"] = (v / Y_SCALE).clamp(-448, 448).to(FP8).double() if out == "static" else v
        return got
    m, n, k = case["m"], case["n"], case["k"]
    v = torch.zeros((m, n), dtype=f64, device=DEV)
    rows = torch.arange(n, device=DEV)
    rows = rows // BLOCK if case["gate"] == "none" else rows // (2 * BLOCK) * 2 + rows % 2
    for j in range(_blocks(k)):
        at = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
        a = s["a"][:, at].to(f64) * s["a_scale"][:, j, None].to(f64)
        v.addmm_(a, (s["b"][:, at].to(f64) * s["b_scale"][rows, j, None].to(f64)).t())
    if s["bias"] is not None:
        v += s["bias"].to(f64)
    if s["residual"] is not None:
        v += s["residual"].to(f64)
    name = case["act"] if case["gate"] == "none" else case["gate"]
    u = v if case["gate"] == "none" else v[:, 0::2]
    if name == "relu":
        u = torch.where(u > 0, u, 0.0)
    elif name == "silu":
        u = u * torch.sigmoid(u)
    elif name == "gelu_tanh":
        u = u * torch.sigmoid(2 * math.sqrt(2 / math.pi) * u * (1 + 0.044715 * u ** 2))
    elif name == "gelu_erf":
        u = u * torch.erfc(-u / math.sqrt(2)) / 2
    return u if case["gate"] == "none" else u * v[:, 1::2]
