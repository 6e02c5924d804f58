"""Attention over the paged cache on the GPU against its definition in 64 bits.

Bounds, derived before any run.  The inputs are exact in both.  With u = 2^-24 the fp32 rounding,
D the head's dims and S = scale sum |q_i k_i| the size of a score's terms, a score is off by at most
e_s = (D + 2) u S, plus 2 u |s| for the two scale products; a probability by the relative
2 e_s (its own score and the maximum, which cancels in the quotient but for the same bound) +
4 u for exp2 and the scale to base 2; sums of T terms add T u.  The probability enters the second
product as two bf16 values, off by 2^-17.  The output is then off by at most
    (2 e_s + 4 u + 2 T u + 2^-17) sum_j p_j |v_j|     and its one rounding 2^-8 |out|,
where 2^-8 is bf16's largest rounding relative to the value; lse by e_s + (T + 8) u (1 + |lse|).
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
K_SCALE, V_SCALE = 0.0625, 0.3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dl_fusion_amd  # noqa: F401  (loud failure if the library is missing)
    torch.cuda.set_device(0)


def make(lens, heads, kv_heads, dim, page, dtype="bf16", spare=3, cols=None, q_more=0, seed=0, garbage=True, peak=1.0):
    """A cache in which the requests' pages lie in random order, every slot past a request's length
    and every unused page holding NaN (a stale cache's worst), and the table's unused entries bad."""
    g = torch.Generator().manual_seed(seed + 13 * dim + heads)
    need = [-(-n // page) for n in lens]
    cols = max([1, *need]) + 1 if cols is None else cols
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    shape = (pages, kv_heads, page, dim)
    if dtype == "fp8":
        k, v = ((torch.randn(shape, generator=g) / s).to(torch.float8_e4m3fn).view(torch.uint8)
                for s in (K_SCALE, V_SCALE))
        bad = 0x7F
    else:
        k, v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        bad = float("nan")
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    table[:, -1] = 2 ** 31 - 1
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for r, n in enumerate(lens):
        mine = order[at:at + need[r]]
        at += need[r]
        table[r, :need[r]] = torch.tensor(mine, dtype=torch.int32)
        for i, p in enumerate(mine):
            used[p, :max(0, min(page, n - i * page))] = True
    if garbage:
        for c in (k, v):
            c.transpose(1, 2)[~used] = bad
    q = torch.randn(len(lens), heads * dim + q_more, generator=g).mul(peak).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32), heads=heads, dim=dim,
                kv_heads=kv_heads, page=page, dtype=dtype, pages=pages, cols=cols)


def definition(s, scale, window=0, skip=()):
    """out and lse in 64 bits on the CPU, with their bounds; `skip`: (request, page column) to leave out."""
    h, hk, d, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    ks, vs = (K_SCALE, V_SCALE) if s["dtype"] == "fp8" else (1.0, 1.0)
    wide = (lambda c: c.view(torch.float8_e4m3fn)) if s["dtype"] == "fp8" else (lambda c: c)
    k, v = wide(s["k"]).double() * ks, wide(s["v"]).double() * vs
    n_req = len(s["lens"])
    out, lse = torch.zeros(n_req, h, d, dtype=torch.float64), torch.full((n_req, h), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(n_req):
        n = int(s["lens"][r])
        keep = [t for t in range(max(0, n - window) if window else 0, n) if (r, t // page) not in skip]
        if not keep:
            continue
        t = torch.tensor(keep)
        pid = s["table"][r].long()[t // page]
        kk, vv = k[pid, :, t % page], v[pid, :, t % page]              # [T][hk][d]
        q = s["q"][r, :h * d].double().view(hk, h // hk, d)
        z = torch.einsum("hgd,thd->hgt", q, kk) * scale
        size = (torch.einsum("hgd,thd->hgt", q.abs(), kk.abs()) * abs(scale)).amax(-1)
        e_s = (d + 2) * U * size + 2 * U * z.abs().amax(-1)
        p = torch.softmax(z, -1)
        o = torch.einsum("hgt,thd->hgd", p, vv)
        spread = torch.einsum("hgt,thd->hgd", p, vv.abs())
        tol = (2 * e_s + 4 * U + 2 * len(keep) * U + 2.0 ** -17)[..., None] * spread + 2.0 ** -8 * o.abs()
        zl = torch.logsumexp(z, -1)
        out[r], out_tol[r] = o.reshape(h, d), tol.reshape(h, d)
        lse[r] = zl.reshape(h)
        lse_tol[r] = (e_s + (len(keep) + 8) * U * (1 + zl.abs())).reshape(h)
    return out, out_tol, lse, lse_tol


def device(s):
    import dl_fusion_amd as dl
    cache = dl.kv_cache_desc(s["pages"], s["kv_heads"], s["page"], s["dim"], s["dtype"], K_SCALE, V_SCALE)
    dev = {n: s[n].cuda() for n in ("q", "k", "v", "table", "lens")}
    dev["q3"] = dev["q"][:, :s["heads"] * s["dim"]].unflatten(1, (s["heads"], s["dim"]))
    return cache, dev


def attend(s, scale, window=0, max_len=0, want_lse=True, dev=None, stream=None):
    import dl_fusion_amd as dl
    cache, dev = device(s) if dev is None else dev
    n, h, d = len(s["lens"]), s["heads"], s["dim"]
    desc = dl.paged_attn_desc(cache, n, h, s["cols"], scale, window, max_len, q_stride=s["q"].shape[1])
    size = dl.dlf_paged_attention_workspace_bytes(desc)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((n * h * d + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n * h + 64,), -7.0, dtype=torch.float32, device="cuda")
    dl.dlf_paged_attention(desc, dev["q3"], dev["k"], dev["v"], dev["table"], dev["lens"], out, lse if want_lse else None,
                           ws, size, stream)
    torch.cuda.synchronize()
    assert (out[n * h * d:] == -7).all() and (ws[size:] == 0xA5).all(), "store beyond an output or the workspace"
    assert (lse[n * h if want_lse else 0:] == -7).all()
    return out[:n * h * d].view(n, h, d).cpu(), lse[:n * h].view(n, h).cpu()


def check(s, scale, window=0, max_len=0, skip=()):
    out, lse = attend(s, scale, window, max_len)
    ref, tol, ref_lse, tol_lse = definition(s, scale, window, skip)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out.double()).all()
    assert (err <= tol).all(), float((err - tol).max())
    gone = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, gone) and (out[gone] == 0).all()
    err = (lse.double() - ref_lse).abs()[~gone]
    assert (err <= tol_lse[~gone]).all(), float((err - tol_lse[~gone]).max())


# lengths at every edge: none, one token, around a half tile, a tile, a page, several waves' tiles
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 100, 127, 128, 129, 160, 255, 257, 511, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_lengths(dim, page, dtype):
    print(f"attention lengths dim={dim} page={page} {dtype}", flush=True)
    check(make(EDGES, 6, 2, dim, page, dtype), dim ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (2, 1), (5, 1), (16, 1), (17, 1), (24, 2), (40, 1), (256, 1),
                                            (32, 8), (35, 5)])
def test_head_layouts(heads, kv_heads, dtype):
    print(f"attention heads={heads}/{kv_heads} {dtype}", flush=True)
    check(make([130, 0, 77, 1], heads, kv_heads, 64, 32, dtype, q_more=40), 0.2)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 100, 128, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("dim", [64, 128])
def test_windows(dim, window):
    print(f"attention window={window} dim={dim}", flush=True)
    check(make(EDGES, 4, 2, dim, 32), dim ** -0.5, window=window)


@pytest.mark.parametrize("max_len", [0, 1, 300, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("fp8", 64), ("bf16", 256)])
def test_long_and_short_together(dtype, dim, max_len):
    """Lengths far apart, whatever bound the caller gives (a wrong one too): same result."""
    print(f"attention ragged dim={dim} {dtype} max_len={max_len}", flush=True)
    check(make([4999, 3, 0, 2050, 1, 700], 8, 2, dim, 16, dtype), dim ** -0.5, max_len=max_len)


@pytest.mark.parametrize("requests", [1, 3, 67, 300])
def test_many_requests(requests):
    print(f"attention requests={requests}", flush=True)
    lens = [(37 * i * i + 11) % 190 for i in range(requests)]
    check(make(lens, 4, 4, 64, 16), 0.125)


def test_one_long_request_over_one_head():
    print("attention 40000 tokens, one kv head", flush=True)
    check(make([40000], 2, 1, 64, 64), 0.125)


def test_sharp_scores():
    """Scores of some hundreds: one token holds all the weight, the maximum moves from tile to tile."""
    for dtype in ("bf16", "fp8"):
        check(make([700, 65, 1], 8, 2, 128, 16, dtype, peak=40.0), 0.25)
        check(make([700, 65, 1], 8, 2, 128, 16, dtype, peak=40.0), -0.25)


def test_lengths_are_clipped_and_bad_pages_left_out():
    s = make([100, 64, 33, 20, 90], 4, 2, 64, 16, cols=9)
    s["lens"][3] = -4                       # none
    s["table"][0, 2] = -1                   # a page missing inside
    s["table"][0, 4] = s["pages"]           # and one past the pool
    s["table"][1, :] = -9                   # every page missing
    s["table"][4, 0] = -2 ** 31
    skip = {(0, 2), (0, 4), (4, 0)} | {(1, c) for c in range(9)}
    print("attention bad pages", flush=True)
    check(s, 0.125, skip=skip)
    # a length beyond the table reads the whole table and nothing past it
    s = make([144, 144], 4, 2, 64, 16, cols=9)
    s["table"][:, -1] = s["table"][:, 0]
    ref = definition(s, 0.125)
    s["lens"][:] = torch.tensor([2 ** 31 - 1, 1000], dtype=torch.int32)
    out, lse = attend(s, 0.125)
    assert ((out.double() - ref[0]).abs() <= ref[1]).all() and ((lse.double() - ref[2]).abs() <= ref[3]).all()


def test_without_lse_and_on_another_stream():
    s = make([300, 5, 0, 77], 8, 2, 128, 32)
    ref = definition(s, 0.1)
    dev = device(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a, _ = attend(s, 0.1, want_lse=False, dev=dev)
    b, lse = attend(s, 0.1, dev=dev, stream=side)
    assert torch.equal(a, b)
    assert ((b.double() - ref[0]).abs() <= ref[1]).all()


def test_values_not_finite_within_reach_reach_the_output():
    s = make([50, 50], 2, 2, 64, 16)
    s["v"][s["table"][0, 1].long(), 0, 3, 5] = float("nan")
    s["k"][s["table"][1, 2].long(), 1, 4, 9] = float("nan")
    out, lse = attend(s, 0.125)
    assert out[0, 0, 5].isnan() and out[1, 1].isnan().all() and lse[1, 1].isnan()
    assert torch.isfinite(out[0, 1]).all() and torch.isfinite(out[1, 0]).all()


def test_graph_replays_follow_the_lengths():
    """Captured once, replayed with the lengths, table and queries of later steps."""
    import dl_fusion_amd as dl
    steps = [make(lens, 8, 2, 128, 16, seed=i, cols=90, spare=200 - sum(-(-n // 16) for n in lens))
             for i, lens in enumerate([[5, 900, 0, 70], [1400, 2, 33, 64], [0, 0, 1, 0]])]
    cache, dev = device(steps[0])
    desc = dl.paged_attn_desc(cache, 4, 8, 90, 0.1)
    size = dl.dlf_paged_attention_workspace_bytes(desc)
    ws = torch.empty(size + 16, dtype=torch.uint8, device="cuda")
    out = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            dl.dlf_paged_attention(desc, dev["q3"], dev["k"], dev["v"], dev["table"], dev["lens"], out, None, ws, size)
    torch.cuda.current_stream().wait_stream(side)
    other = torch.randn(1 << 20, device="cuda")
    for s in steps + steps:
        assert s["pages"] == steps[0]["pages"]
        for n in ("q", "k", "v", "table", "lens"):
            dev[n].copy_(s[n])
        out.zero_()
        float(other.sum())                  # eager work and a synchronisation between replays
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu()
        eager, _ = attend(s, 0.1)
        assert torch.equal(got, eager)
        ref, tol, _, _ = definition(s, 0.1)
        assert ((got.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("requests,kv_heads", [(63, 2), (65, 2), (300, 3), (1100, 2), (4200, 1)])
def test_many_requests_of_which_few_are_long(requests, kv_heads):
    """Pieces are cut over any number of requests (a table of 101 pages lets any be long); past 4096
    items none is cut."""
    print(f"attention requests={requests} kv_heads={kv_heads}, two long", flush=True)
    lens = [(5 * i * i) % 23 for i in range(requests)]
    lens[requests // 2], lens[-1] = 1600, 777
    check(make(lens, 2 * kv_heads, kv_heads, 64, 16, cols=101), 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [513, 600, 5000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_over_pieces(dim, window, dtype):
    print(f"attention window={window} dim={dim} {dtype}, pieces", flush=True)
    check(make([6000, 512, 513, 0, 5001, 601, 1], 6, 2, dim, 48, dtype), dim ** -0.5, window=window)


@pytest.mark.parametrize("heads,kv_heads", [(16, 1), (17, 1), (40, 2), (5, 5)])
def test_head_layouts_over_pieces(heads, kv_heads):
    print(f"attention heads={heads}/{kv_heads}, pieces", flush=True)
    check(make([3000, 0, 1, 700], heads, kv_heads, 128, 32), 0.1)


def test_a_piece_without_a_page():
    """A long request whose pages are missing over whole pieces of it, and one without any."""
    s = make([20000, 3000, 40], 4, 2, 64, 16, cols=1300)
    s["table"][0, 100:1100] = -1
    s["table"][1, :] = -1
    skip = {(0, c) for c in range(100, 1100)} | {(1, c) for c in range(1300)}
    print("attention pieces without pages", flush=True)
    check(s, 0.125, skip=skip)


def test_repeats_give_the_same_bits():
    s = make([9000, 3, 0, 2050, 1, 700], 8, 2, 128, 16)
    dev = device(s)
    a, la = attend(s, 0.1, dev=dev)
    for _ in range(3):
        b, lb = attend(s, 0.1, dev=dev)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_offsets_beyond_32_bits():
    """The same pages at the far end of caches of more than 4 GB give the same bits."""
    import dl_fusion_amd as dl
    s = make([700, 33, 0, 1500], 16, 8, 128, 16)
    cache, dev = device(s)
    pages = (1 << 32) // (8 * 16 * 128 * 2) + 1000
    if torch.cuda.mem_get_info()[0] < 2 * pages * 8 * 16 * 128 * 2 + (1 << 30):
        pytest.skip("not enough memory")
    print("attention cache of 4.03 GB each", flush=True)
    far = dict(dev, k=torch.empty(pages, 8, 16, 128, dtype=torch.bfloat16, device="cuda"),
               v=torch.empty(pages, 8, 16, 128, dtype=torch.bfloat16, device="cuda"))
    shift = pages - s["pages"]
    far["k"][shift:], far["v"][shift:] = dev["k"], dev["v"]
    far["table"] = torch.where((dev["table"] >= 0) & (dev["table"] < s["pages"]), dev["table"] + shift, dev["table"])
    near = attend(s, 0.09, dev=(cache, dev))
    big = dl.kv_cache_desc(pages, 8, 16, 128)
    got = attend(s, 0.09, dev=(big, far))
    assert torch.equal(near[0], got[0]) and torch.equal(near[1], got[1])
    # and the store reaches there
    x = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * 16 - 1, -1, pages * 16 - 18], device="cuda")
    dl.dlf_paged_store(big, x, -x, slots, far["k"], far["v"])
    torch.cuda.synchronize()
    assert torch.equal(far["k"][-1, :, 15], x[0]) and torch.equal(far["v"][-1, :, 15], -x[0])
    assert torch.equal(far["k"][-2, :, 14], x[2]) and torch.equal(far["v"][-2, :, 14], -x[2])


def check_extended(s, scale, window=0):
    """Infinities and NaN where the definition has them, the bounds elsewhere."""
    out, lse = attend(s, scale, window)
    out = out.double()
    ref, tol, ref_lse, tol_lse = definition(s, scale, window)
    assert torch.equal(out.isnan(), ref.isnan())
    wide = ref.isinf()
    assert torch.equal(out[wide], ref[wide])
    rest = ref.isfinite()
    assert ((out - ref).abs()[rest] <= tol[rest]).all()
    assert ((lse.double() - ref_lse).abs() <= tol_lse).all()
    return ref


def value_rows(s, r, token):
    """[kv_heads][dim] of a token's values, to be written."""
    return s["v"][int(s["table"][r, token // s["page"]]), :, token % s["page"]]


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_values_are_infinite_outputs(dim):
    """One infinite value in a dim gives that infinity, both signs give NaN, other dims and heads are as before:
    a request of one token, and tokens at every place of tiles, waves and pieces."""
    print(f"attention infinite values dim={dim}", flush=True)
    lens = [1, 50, 140, 700, 3000]
    s = make(lens, 6, 2, dim, 16)
    for r, n in enumerate(lens):
        for i, token in enumerate({0, n // 3, n // 2, n - 1}):
            value_rows(s, r, token)[0, 3 + i] = float("inf")
            value_rows(s, r, token)[1, 40 + i] = -float("inf")
        value_rows(s, r, 0)[1, 50] = float("inf")
        value_rows(s, r, n - 1)[1, 50] = -float("inf")      # the first token's where there is one
    ref = check_extended(s, dim ** -0.5)
    assert ref.isinf().any(-1).all() and ref[1:, 3:].isnan().any(-1).all()
    check_extended(s, dim ** -0.5, window=45)


@pytest.mark.parametrize("far", [60, 256])
def test_an_infinite_value_of_a_token_that_hardly_counts(far):
    """Its probability e^-far times infinity is infinity, also where the probability itself is below fp32's
    range: before and after the token that counts, in its tile, another one and another piece."""
    print(f"attention infinite values, {far} below the maximum", flush=True)
    lens = [40, 40, 900, 900, 5000, 5000]
    s = make(lens, 2, 2, 64, 16)
    s["q"].zero_()
    s["q"].view(6, 2, 64)[:, :, 0] = 16.0
    s["k"].nan_to_num_(0.0).zero_()
    for r, (top, other) in enumerate([(30, 2), (2, 30), (800, 3), (3, 800), (4900, 100), (100, 4900)]):
        s["k"][int(s["table"][r, top // 16]), :, top % 16, 0] = far / 16
        value_rows(s, r, other)[:, 7] = float("inf")
        value_rows(s, r, other)[0, 9] = -float("inf")
    ref = check_extended(s, 1.0)
    assert (ref[:, :, 7] == float("inf")).all() and (ref[:, 0, 9] == -float("inf")).all()


def test_an_infinite_value_beside_one_that_is_not_a_number():
    s = make([600, 33], 2, 2, 128, 16)
    value_rows(s, 0, 17)[:, 5], value_rows(s, 0, 599)[:, 6] = float("inf"), float("nan")
    value_rows(s, 1, 32)[:, 5], value_rows(s, 1, 0)[:, 5] = float("inf"), float("nan")
    check_extended(s, 0.1)
