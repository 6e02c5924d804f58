"""The page plan and the cache store on the GPU against their definitions.

Both are exact: the plan gives whole numbers, the bf16 store copies, and the fp8 store's codes are
one fp32 product and one rounding to e4m3, which the CPU's cast repeats bit for bit.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dl_fusion_amd  # noqa: F401  (loud failure if the library is missing)
    torch.cuda.set_device(0)


# ---------------------------------------------------------------------------
# Page plan: a token-by-token walk over Python integers
# ---------------------------------------------------------------------------
def plan_by_hand(cached, fresh, free, head, table, page, cap_pages, token_cap):
    cap = cap_pages * page
    up = lambda n: -(-n // page)  # noqa: E731
    head = max(head, 0)
    want = head
    table = [list(r) for r in table]
    starts, lens, slots, rows = [], [], [], []
    for r, (c, f) in enumerate(zip(cached, fresh)):
        c, f = max(c, 0), max(f, 0)
        starts.append(len(slots))
        lens.append(min(c + f, cap))
        for col in range(up(min(c, cap)), up(lens[-1])):
            table[r][col] = free[want] if want < len(free) else -1
            want += 1
        for pos in range(c, c + f):
            p = table[r][pos // page] if pos < cap else -1
            slots.append(p * page + pos % page if p >= 0 else -1)
            rows.append(r)
    starts.append(len(slots))
    total = len(slots)
    fill = max(0, token_cap - total)
    counts = [total, min(want, len(free)), max(lens, default=0), max(0, want - max(head, len(free)))]
    return table, starts, lens, (slots + [-1] * fill)[:token_cap], (rows + [-1] * fill)[:token_cap], counts


# requests, page, columns, longest cached, longest fresh, free pages beyond (or short of) the need, head, token room
PLANS = [
    (0, 16, 4, 0, 0, 3, 0, 5),
    (1, 16, 4, 20, 1, 0, 0, 0),
    (1, 16, 300, 0, 4097, 2, 1, 3),
    (3, 1, 40, 9, 20, 5, 4, 1),
    (37, 48, 9, 200, 150, 9, 2, 11),          # 48 tokens a page; some tokens past the table
    (255, 16, 30, 100, 3, 1, 0, 0),
    (256, 16, 30, 400, 1, 0, 7, 64),
    (257, 16, 30, 400, 40, -9, 3, 9),          # the free list ends early
    (700, 32, 20, 500, 70, 20, 0, -333),       # room for fewer tokens than there are
    (1300, 64, 8, 300, 90, 0, 2, 100),
]


@pytest.mark.parametrize("spec", PLANS, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("rows_wanted", [True, False])
def test_page_plan(spec, rows_wanted):
    import dl_fusion_amd as d
    n, page, cols, max_c, max_f, spare, head, room = spec
    print(f"page plan {spec}", flush=True)
    g = torch.Generator().manual_seed(n * 7 + page)
    cached = torch.randint(0, max_c + 1, (n,), generator=g).tolist()
    fresh = torch.randint(0, max_f + 1, (n,), generator=g).tolist()
    if n > 20:
        cached[3], fresh[3] = -5, 4            # a negative count is none
        cached[5], fresh[5] = 6, -2
        fresh[9] = fresh[10] = 0
        cached[11], fresh[11] = 2 ** 31 - 1, 3     # nothing of it fits the table
    need = sum(max(0, -(-min(max(c, 0) + max(f, 0), cols * page) // page) - -(-min(max(c, 0), cols * page) // page))
               for c, f in zip(cached, fresh))
    free = torch.randperm(max(0, head + need + spare) + 1000, generator=g)[:max(0, head + need + spare)].tolist()
    table = torch.randint(0, 5000, (n, cols), generator=g)
    table[torch.rand(n, cols, generator=g) < 0.1] = -1       # pages that an earlier step did not get
    token_cap = max(0, sum(max(f, 0) for f in fresh) + room)
    ref = plan_by_hand(cached, fresh, free, head, table.tolist(), page, cols, token_cap)

    i32 = dict(dtype=torch.int32, device="cuda")
    dev = dict(cached=torch.tensor(cached, **i32), fresh=torch.tensor(fresh, **i32), free=torch.tensor(free, **i32),
               head=torch.tensor([head], **i32) if head else None)
    out = dict(table=table.to(**i32), starts=torch.full((n + 1,), -7, **i32), lens=torch.full((n,), -7, **i32),
               slots=torch.full((token_cap + 8,), -7, dtype=torch.int64, device="cuda"),
               rows=torch.full((token_cap + 8,), -7, **i32), counts=torch.full((4,), -7, **i32))
    desc = d.page_plan_desc(n, page, cols, token_cap, len(free))
    for _ in range(2):                          # a second call finds its own entries and gives the same
        d.dlf_page_plan(desc, dev["cached"], dev["fresh"], dev["free"], dev["head"], out["table"], out["starts"],
                        out["lens"], out["slots"], out["rows"] if rows_wanted else None, out["counts"])
        torch.cuda.synchronize()
        assert out["table"].tolist() == ref[0]
        assert out["starts"].tolist() == ref[1]
        assert out["lens"].tolist() == ref[2]
        assert out["slots"][:token_cap].tolist() == ref[3]
        assert out["rows"][:token_cap].tolist() == (ref[4] if rows_wanted else [-7] * token_cap)
        assert out["counts"].tolist() == ref[5]
        assert (out["slots"][token_cap:] == -7).all() and (out["rows"][token_cap:] == -7).all(), "store beyond the room"


def test_page_plan_negative_head_and_totals_beyond_32_bits():
    import dl_fusion_amd as d
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 300
    cached = torch.zeros(n, **i32)
    fresh = torch.full((n,), 2 ** 30, **i32)    # 300 x 2^30 tokens; 4 pages of 16 fit each table
    free = torch.arange(4 * n, **i32).flip(0).contiguous()
    head = torch.tensor([-3], **i32)
    table = torch.full((n, 4), -1, **i32)
    starts, lens, counts = torch.empty(n + 1, **i32), torch.empty(n, **i32), torch.empty(4, **i32)
    slots = torch.empty(200, dtype=torch.int64, device="cuda")
    rows = torch.empty(200, **i32)
    d.dlf_page_plan(d.page_plan_desc(n, 16, 4, 200, 4 * n), cached, fresh, free, head, table, starts, lens, slots,
                    rows, counts)
    torch.cuda.synchronize()
    top = 2 ** 31 - 1
    assert table.flatten().tolist() == free.tolist()
    assert starts.tolist() == [min(top, i << 30) for i in range(n + 1)]
    assert (lens == 64).all() and counts.tolist() == [top, 4 * n, 64, 0]
    assert rows.tolist() == [0] * 200
    assert slots.tolist() == [(4 * n - 1 - t // 16) * 16 + t % 16 for t in range(64)] + [-1] * 136


# ---------------------------------------------------------------------------
# Store
# ---------------------------------------------------------------------------
STORES = [
    # tokens, kv heads, head dim, page, elements between rows of k and v beyond their width
    (1, 1, 64, 16, 0, 0),
    (1, 8, 128, 16, 0, 4096),
    (7, 3, 64, 48, 8, 0),
    (33, 5, 256, 32, 64, 72),
    (130, 32, 128, 16, 0, 0),
    (1029, 2, 128, 64, 1024, 256),
]


@pytest.mark.parametrize("spec", STORES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_paged_store(spec, dtype):
    import dl_fusion_amd as d
    tokens, heads, dim, page, more_k, more_v = spec
    print(f"paged store {spec} {dtype}", flush=True)
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // page) + 3
    ks, vs = 0.0625, 0.3
    wide = [(torch.randn(tokens, heads * dim + m, generator=g) * 20).to(torch.bfloat16) for m in (more_k, more_v)]
    special = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 448 * ks, 3e38, 1e-40],
                           dtype=torch.bfloat16)
    for w in wide:
        w[-1, :8] = special
    new = [w[:, :heads * dim].unflatten(1, (heads, dim)) for w in wide]
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    if tokens > 5:
        slots[1], slots[2], slots[3] = -1, pages * page, -(2 ** 40)
    store = torch.uint8 if dtype == "fp8" else torch.int16
    top = 256 if dtype == "fp8" else 30000
    caches = [torch.randint(0, top, (pages, heads, page, dim), generator=g).to(store) for _ in range(2)]
    ref = []
    for x, c, s in zip(new, caches, (ks, vs)):
        c = c.clone()
        if dtype == "fp8":
            inv = torch.tensor(1.0) / torch.tensor(s, dtype=torch.float32)
            codes = (x.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            codes = x.contiguous().view(torch.int16)
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < pages * page:
                c[slot // page, :, slot % page] = codes[t]
        ref.append(c)
    k, v = (w.cuda()[:, :heads * dim].unflatten(1, (heads, dim)) for w in wide)
    dev = [c.cuda() for c in caches]
    desc = d.kv_cache_desc(pages, heads, page, dim, dtype, ks, vs)
    d.dlf_paged_store(desc, k, v, slots.cuda(), *dev)
    torch.cuda.synchronize()
    for got, want in zip(dev, ref):
        got = got.cpu()
        if dtype == "fp8":                      # a NaN's sign is not defined
            nan = (want & 127) == 127
            assert ((got & 127) == 127)[nan].all()
            got, want = got[~nan], want[~nan]
        assert torch.equal(got, want)
