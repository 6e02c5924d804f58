"""Low-rank adapters on the GPU against their definition in 64 bits.

Bounds, derived before any run, with u = 2^-24 (fp32) and all inputs exact in both.  A value of
h = x A^T is a sum of k products: off by at most (k + 20) u H, H = sum |x| |A| (20 for the order
over waves and slices).  It is scaled (u), and enters the second product as two bf16 values
(2^-17), whose sum over the rank has (2 rank + 4) u more.  So before its rounding out is off by at most
    |scale| sum_r ((k + 2 rank + 26) u H_r + 2^-17 |h_r|) |B_nr|  +  2 u |out|
and by 2^-8 |out| in it (bf16's largest rounding relative to the value).
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dl_fusion_amd  # noqa: F401  (loud failure if the library is missing)
    torch.cuda.set_device(0)


def make(m, n, k, rank, adapters, ids, base=True, scales=True, seed=0, more=(0, 0, 0)):
    """`more`: elements between the rows of x, base and out beyond their width."""
    g = torch.Generator().manual_seed(seed + 31 * m + n)
    bf = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16)  # noqa: E731
    return dict(x=bf(m, k + more[0]), a=bf(adapters, rank, k), b=bf(adapters, n, rank) * 0.25,
                scale=torch.rand(adapters, generator=g) * 2 - 0.5 if scales else None, ids=ids.to(torch.int32),
                base=bf(m, n + more[1]) * 8 if base else None, n=n, k=k, rank=rank, adapters=adapters, more=more)


def definition(s, ids):
    m, n, k = s["x"].shape[0], s["n"], s["k"]
    x = s["x"][:, :k].double()
    out = torch.zeros(m, n, dtype=torch.float64) if s["base"] is None else s["base"][:, :n].double()
    tol = torch.zeros(m, n, dtype=torch.float64)
    for i in range(s["adapters"]):
        rows = (ids == i).nonzero().flatten()
        if not rows.numel():
            continue
        f = 1.0 if s["scale"] is None else float(s["scale"][i])
        a, b = s["a"][i].double(), s["b"][i].double()
        h, size = x[rows] @ a.t(), x[rows].abs() @ a.abs().t()
        out[rows] += f * (h @ b.t())
        tol[rows] = abs(f) * (((k + 2 * s["rank"] + 26) * U * size + 2.0 ** -17 * h.abs()) @ b.abs().t())
    return out, tol + (2 * U + 2.0 ** -8) * out.abs()


def add(s, row_map=None, in_place=False, stream=None, dev=None):
    import dl_fusion_amd as dl
    m, n, k = s["x"].shape[0], s["n"], s["k"]
    mx, my, mo = s["more"]
    dev = dev or {t: None if s[t] is None else s[t].cuda() for t in ("x", "a", "b", "scale", "ids", "base")}
    if in_place:
        buf = torch.full((m * (n + my) + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
        buf[:m * (n + my)].view(m, n + my).copy_(dev["base"])
        base = out = buf[:m * (n + my)].view(m, n + my)[:, :n]
        mo = my
    else:
        buf = torch.full((m * (n + mo) + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:m * (n + mo)].view(m, n + mo)[:, :n]
        base = None if dev["base"] is None else dev["base"][:, :n]
    before = buf.clone()
    d = dl.lora_desc(m, n, k, s["rank"], s["adapters"], 0 if row_map is None else s["ids"].numel(), k + mx, n + my, n + mo)
    size = dl.dlf_lora_workspace_bytes(d)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:size].view(torch.float32).fill_(float("nan"))       # scratch: read only where it was written
    torch.cuda.synchronize()
    dl.dlf_lora_add(d, dev["x"][:, :k], dev["a"], dev["b"], dev["scale"], dev["ids"], row_map, base, out, ws, size, stream)
    torch.cuda.synchronize()
    got = out.cpu()
    assert (ws[size:] == 0xA5).all(), "store beyond the workspace"
    out.copy_(before[:m * (n + mo)].view(m, n + mo)[:, :n])
    assert torch.equal(buf, before), "store beyond the output"
    return got


def check(s, ids=None, **kw):
    got = add(s, **kw)
    ref, tol = definition(s, s["ids"] if ids is None else ids)
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


def mixed(m, adapters, seed=1):
    """Any adapter on any row, with rows that have none (-1) and bad ids."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, adapters, (m,), generator=g)
    if m > 6:
        ids[2], ids[5] = adapters, -2 ** 31
    return ids


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("m", [1, 17, 65])
def test_ranks(m, rank):
    print(f"adapters m={m} rank={rank}", flush=True)
    check(make(m, 136, 264, rank, 5, mixed(m, 5)))


@pytest.mark.parametrize("n,k", [(8, 8), (64, 64), (72, 40), (256, 512), (264, 1000), (1032, 2056), (16, 4096), (2048, 24)])
@pytest.mark.parametrize("m", [3, 130])
def test_sizes(m, n, k):
    print(f"adapters m={m} n={n} k={k}", flush=True)
    check(make(m, n, k, 16, 3, mixed(m, 3)))


@pytest.mark.parametrize("adapters", [1, 2, 64, 65, 300])
def test_adapter_counts_and_orders(adapters):
    print(f"adapters {adapters}", flush=True)
    for m in (64, 150):
        check(make(m, 128, 128, 8, adapters, mixed(m, adapters)))
        check(make(m, 128, 128, 8, adapters, torch.arange(m) % adapters))
        check(make(m, 128, 128, 8, adapters, torch.arange(m) * adapters // m))
        check(make(m, 128, 128, 8, adapters, torch.full((m,), adapters - 1)))


def test_runs_of_one_adapter():
    """Prompts: long runs whose ends fall inside a tile."""
    ids = torch.cat([torch.full((n,), i) for i, n in enumerate([700, 1, 333, 64, 90, 2000])])
    print("adapters runs", flush=True)
    for rank in (16, 64, 128):
        check(make(ids.numel(), 320, 512, rank, 6, ids))


def test_no_adapter_at_all():
    s = make(70, 64, 64, 16, 2, torch.full((70,), -1))
    assert torch.equal(add(s), s["base"])
    s = make(70, 64, 64, 16, 2, torch.full((70,), -1), base=False)
    assert (add(s) == 0).all()


def test_an_empty_pool_and_an_empty_inner_dimension():
    import dl_fusion_amd as dl
    base = torch.randn(5, 64, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(base)
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    for k, adapters in ((64, 0), (0, 2)):
        d = dl.lora_desc(5, 64, k, 16, adapters)
        ws = torch.empty(dl.dlf_lora_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        x = torch.randn(5, 64, device="cuda").to(torch.bfloat16)
        b = torch.randn(2, 64, 16, device="cuda").to(torch.bfloat16)
        dl.dlf_lora_add(d, x.data_ptr(), b, b, None, ids, None, base, out.zero_(), ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(out, base)


@pytest.mark.parametrize("more", [(8, 0, 0), (0, 64, 0), (0, 0, 128), (40, 72, 8)])
def test_strides(more):
    print(f"adapters strides {more}", flush=True)
    check(make(70, 192, 128, 16, 4, mixed(70, 4), more=more))


def test_without_base_or_scales_and_in_place():
    check(make(70, 192, 128, 16, 4, mixed(70, 4), base=False))
    check(make(70, 192, 128, 16, 4, mixed(70, 4), scales=False))
    check(make(70, 192, 128, 16, 4, mixed(70, 4), base=False, scales=False))
    check(make(70, 192, 128, 16, 4, mixed(70, 4), more=(0, 64, 0)), in_place=True)
    check(make(300, 192, 128, 64, 4, mixed(300, 4)), in_place=True)


def test_row_map():
    """Rows name a request, requests an adapter: bad and missing requests have none."""
    g = torch.Generator().manual_seed(4)
    s = make(200, 64, 96, 8, 5, torch.tensor([3, -1, 0, 4, 4, 9, 1]))
    rows = torch.randint(-2, 9, (200,), generator=g)
    of = torch.tensor([int(s["ids"][r]) if 0 <= r < 7 else -1 for r in rows.tolist()])
    check(s, ids=of, row_map=rows.to(torch.int32).cuda())


def test_a_row_not_finite_stays_alone():
    s = make(40, 64, 64, 16, 2, torch.arange(40) % 2)
    s["x"][7, 3] = float("nan")
    s["x"][8, 9] = float("inf")
    got = add(s)
    assert got[7].isnan().all()
    rest = [i for i in range(40) if i not in (7, 8)]
    ref, tol = definition(s, s["ids"])
    assert ((got.double() - ref).abs()[rest] <= tol[rest]).all()


def test_stream_and_repeats():
    """On another stream, and twice: the same bits (the sums' order is fixed)."""
    s = make(130, 512, 1024, 32, 7, mixed(130, 7))
    dev = {t: s[t].cuda() for t in ("x", "a", "b", "scale", "ids", "base")}
    torch.cuda.synchronize()
    a = add(s, dev=dev)
    assert torch.equal(a, add(s, dev=dev, stream=torch.cuda.Stream()))
    assert torch.equal(a, add(s, dev=dev))


def test_graph_replays():
    import dl_fusion_amd as dl
    s = make(40, 256, 512, 16, 6, mixed(40, 6))
    dev = {t: s[t].cuda() for t in ("x", "a", "b", "scale", "ids", "base")}
    out = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    d = dl.lora_desc(40, 256, 512, 16, 6)
    ws = torch.empty(dl.dlf_lora_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            dl.dlf_lora_add(d, dev["x"], dev["a"], dev["b"], dev["scale"], dev["ids"], None, dev["base"], out, ws, ws.numel())
    torch.cuda.current_stream().wait_stream(side)
    other = torch.randn(1 << 20, device="cuda")
    for i in range(3):
        s["ids"] = mixed(40, 6, seed=20 + i).to(torch.int32)
        dev["ids"].copy_(s["ids"])
        out.zero_()
        float(other.sum())                  # eager work and a synchronisation between replays
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = definition(s, s["ids"])
        assert ((out.cpu().double() - ref).abs() <= tol).all()
        assert torch.equal(out.cpu(), add(s))


@pytest.mark.parametrize("m", [1, 16, 17])
@pytest.mark.parametrize("k", [8, 56, 8192, 8200])
@pytest.mark.parametrize("rank", [8, 24, 32, 40])
def test_few_rows(m, k, rank):
    """Around the sizes at which one launch does both products."""
    print(f"adapters m={m} k={k} rank={rank}", flush=True)
    check(make(m, 328, k, rank, 4, mixed(m, 4)))


@pytest.mark.parametrize("rank", [16, 72, 120])
@pytest.mark.parametrize("n,k", [(40, 136), (1000, 520), (4096, 264)])
def test_many_rows_of_one_adapter(n, k, rank):
    print(f"adapters many rows n={n} k={k} rank={rank}", flush=True)
    check(make(333, n, k, rank, 2, torch.arange(333) // 200))
    check(make(333, n, k, rank, 2, torch.arange(333) // 200, base=False, more=(8, 0, 16)))


@pytest.mark.parametrize("m", [256, 400])
def test_every_row_its_own_adapter(m):
    print(f"adapters m={m} all different", flush=True)
    check(make(m, 128, 128, 16, 64, mixed(m, 64)))
    check(make(m, 128, 128, 64, m, torch.arange(m)))


@pytest.mark.parametrize("rank", [8, 32, 40])
@pytest.mark.parametrize("k", [136, 6144, 6152])
def test_groups_of_one_adapter_in_a_small_batch(k, rank):
    """Groups of 15 to 48 rows among single ones, in any order, around the sizes at which one launch does both."""
    g = torch.Generator().manual_seed(3)
    ids = torch.cat([torch.full((n,), i) for i, n in enumerate([15, 16, 17, 33, 48, 1, 1, 5])] + [torch.full((9,), -1)])
    print(f"adapters groups k={k} rank={rank}", flush=True)
    check(make(ids.numel(), 200, k, rank, 8, ids))
    check(make(ids.numel(), 200, k, rank, 8, ids[torch.randperm(ids.numel(), generator=g)]))
    check(make(256, 200, k, rank, 1, torch.zeros(256)))
    check(make(257, 200, k, rank, 70, torch.arange(257) % 70))


# Batches whose number of tiles is a multiple of 16 and one off it, with two workgroups a CU and one; runs
# that end inside a tile, at its end, and longer ones
@pytest.mark.parametrize("run", [64, 100, 5000])
@pytest.mark.parametrize("m,n", [(1024, 2056), (1025, 2056), (1024, 968), (960, 72), (2048, 1032)])
@pytest.mark.parametrize("rank", [16, 128])
def test_tiles_and_ranges(rank, m, n, run):
    ids = (torch.arange(m) // run) % 4 - 1
    check(make(m, n, 136, rank, 3, ids, seed=13))


# Short ranges of columns: few tiles, widths of one block and a few, all rows of one adapter or of several
@pytest.mark.parametrize("n", [8, 64, 200, 1544])
@pytest.mark.parametrize("m,adapters", [(1, 1), (18, 1), (64, 2), (257, 1), (330, 3)])
def test_short_ranges(m, adapters, n):
    check(make(m, n, 520, 64, adapters, mixed(m, adapters), seed=14))


# One row without an adapter among 63 of one, and pools whose groups of 16 rows end anywhere
@pytest.mark.parametrize("adapters", [1, 2, 5])
@pytest.mark.parametrize("m", [33, 49, 64, 200])
def test_groups_of_few_adapters(m, adapters):
    for ids in (mixed(m, adapters), torch.where(torch.arange(m) % 64 == 7, -1, 0), torch.arange(m) % (adapters + 1) - 1):
        check(make(m, 264, 264, 24, adapters, ids, seed=15))


def few_and_many(m=90):
    """Adapter 0 on 5 rows of a tile, adapter 1 on 40 of one, adapter 2 on the rest, a row without any."""
    return torch.cat([torch.zeros(5), torch.full((40,), 1.0), torch.full((m - 46,), 2.0), torch.tensor([-1.0])]).long()


# every rank that is admitted, up to 16 rows of an adapter and more
@pytest.mark.parametrize("rank", range(8, 136, 8))
def test_every_rank(rank):
    print(f"adapters rank={rank}", flush=True)
    ids = few_and_many()
    check(make(ids.numel(), 328, 264, rank, 3, ids))
    check(make(13, 328, 264, rank, 3, mixed(13, 3), base=False))
    check(make(300, 328, 264, rank, 3, torch.arange(300) // 110))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rank", [8, 24, 40, 56, 72, 80, 88, 96, 104, 120])
def test_a_weight_not_finite_stays_in_its_column(rank, bad):
    """Outputs of a column depend on that row of B alone."""
    cols = [0, 1, 17, 32, 63, 100, 135]
    for ids in (few_and_many(), mixed(9, 3)):
        s = make(ids.numel(), 136, 264, rank, 3, ids)
        s["b"][:, cols] = bad
        print(f"adapters rank={rank} bad={bad}", flush=True)
        got = add(s)
        ref, tol = definition(s, s["ids"])
        rest = [c for c in range(136) if c not in cols]
        assert ((got.double() - ref).abs()[:, rest] <= tol[:, rest]).all()


def check_extended(s):
    """Infinities and NaN where the definition has them, the bound elsewhere."""
    got = add(s).double()
    ref, tol = definition(s, s["ids"])
    assert torch.equal(got.isnan(), ref.isnan())
    wide = ref.isinf()
    assert torch.equal(got[wide], ref[wide])
    rest = ref.isfinite()
    assert ((got - ref).abs()[rest] <= tol[rest]).all()
    return ref


@pytest.mark.parametrize("rank", [8, 32, 40, 64, 80, 128])
def test_infinities_stay_infinities(rank):
    """An infinite input, an infinite weight of either product, and both: the formula's infinity, not NaN, but
    where infinities of both signs meet or one meets zero."""
    ids = few_and_many()
    for what in ("x", "a", "b", "x and b"):
        print(f"adapters rank={rank}, infinities in {what}", flush=True)
        s = make(ids.numel(), 136, 264, rank, 3, ids, seed=16)
        s["scale"] += 1
        if "x" in what:
            s["a"], s["b"] = s["a"].abs(), s["b"].abs()     # no two signs: the rows' outputs are infinities
            s["x"][3, 7], s["x"][20, 263], s["x"][60, 0] = float("inf"), -float("inf"), float("inf")
            s["b"][:, 9] = 0                                # but for this column
        if "a" in what:
            s["a"][1, rank - 1, 5] = float("inf")
        if "b" in what:
            s["b"][:, 40, 3], s["b"][:, 135, rank - 1] = float("inf"), -float("inf")
            s["b"][:, 70, :2] = float("inf")                # NaN where the two ranks' signs differ
        ref = check_extended(s)
        assert ref.isinf().any() and ref.isfinite().any()


@pytest.mark.parametrize("rank", [16, 64, 128])
def test_an_inner_vector_at_the_end_of_the_range(rank):
    """(2 - 2^-9) 2^127 is finite in fp32, and rounds to an infinity of bf16."""
    ids = few_and_many()
    s = make(ids.numel(), 136, 264, rank, 3, ids, scales=False, seed=17)
    s["x"].zero_()
    s["a"].zero_()
    s["x"][:, 0], s["a"][:, :, 0] = (2 - 2.0 ** -7) * 2.0 ** 63, 2.0 ** 64
    s["x"][:, 9], s["a"][:, :, 9] = 1.5 * 2.0 ** 60, 2.0 ** 59
    s["b"] *= 2.0 ** -100
    ref = check_extended(s)
    assert ref.isfinite().all()
