"""The attention block over a paged cache (dl_fusion_amd/decode.py): its parts run together, step by step,
against their definitions in 64 bits, and captured in a graph.

Each stage is checked from the stage before it as the device has it.  The product with adapters is rounded
twice to bf16 (2^-8 of the product, of the sum), its own sums and the adapters' stay below a quarter of
that: |x| |W| sums of 256 terms of fp32 rounding 2^-24 are 2^-16, and the adapters' inner vector as two
bf16 values is off by 2^-17 of it.  The attended rows are off by 2^-8 of the value, and by 2^-8 of sum p |v|
for everything else (scores of 64 products and probabilities as two bf16 values are below 2^-12).  The
output is rounded once."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HIDDEN, HEADS, KV, DIM, PAGE, COLS, RANK = 256, 4, 2, 64, 16, 70, 16
WIDTH = (HEADS + 2 * KV) * DIM


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()


def build(requests, g, cache="bf16", adapters=3):
    from dl_fusion_amd.decode import PagedAttentionBlock
    ad = None
    if adapters:
        ad = (rand(g, adapters, RANK, HIDDEN, scale=HIDDEN ** -0.5), rand(g, adapters, WIDTH, RANK, scale=0.25),
              torch.rand(adapters, generator=g).add(0.5).cuda())
    return PagedAttentionBlock(rand(g, WIDTH, HIDDEN, scale=HIDDEN ** -0.5), rand(g, HIDDEN, HEADS * DIM, scale=0.06),
                               HEADS, KV, DIM, requests, requests * COLS, PAGE, COLS, ad, cache=cache, k_scale=0.0625,
                               v_scale=0.0625)


def projected(block, x, ids):
    """The product with adapters in 64 bits, and its bound."""
    y = x.double() @ block.w_qkv.double().t()
    tol = y.abs()
    if block.adapters is not None:
        a, b, scale = (t.double() for t in block.adapters)
        for i, k in enumerate(ids):
            if k >= 0:
                h = x[i].double() @ a[k].t()
                y[i] += scale[k] * (h @ b[k].t())
                tol[i] += 2.0 ** -7 * (scale[k] * (h.abs() @ b[k].abs().t()))
    size = x.double().abs() @ block.w_qkv.double().abs().t()
    return y, 2.0 ** -8 * (tol * 1.01 + y.abs()) + 2.0 ** -15 * size + 2.0 ** -12 * y.abs()


def held(block, r):
    """The keys and values that place r has, out of its pages."""
    n = int(block.lens[r])
    at = block.table[r, :-(-n // PAGE)].long()
    got = []
    for c in (block.k_cache, block.v_cache):
        c = c.view(torch.uint8)[at].view(c.dtype).double() * (0.0625 if c.dtype == torch.float8_e4m3fn else 1.0)
        got.append(c.transpose(1, 2).reshape(-1, KV, DIM)[:n])
    return got


def check_step(block, x, y, ids, fresh, lens, kv_rows):
    """After a step: `kv_rows` [place] -> the qkv rows stored so far, appended to here."""
    b = block._buffers(block.requests)
    ref, tol = projected(block, x, ids)
    qkv = b["qkv"].double()
    assert ((qkv - ref).abs() <= tol).all()
    assert block.lens.tolist() == lens
    attended = block.attended.double()
    for r in range(block.requests):
        if fresh[r]:
            kv_rows[r].append(b["qkv"][r, HEADS * DIM:].clone())
        if not lens[r]:
            assert (attended[r] == 0).all()
            continue
        k, v = held(block, r)
        rows = torch.stack(kv_rows[r]).double().view(-1, 2, KV, DIM)
        if block.k_cache.dtype == torch.bfloat16:
            assert torch.equal(k, rows[:, 0]) and torch.equal(v, rows[:, 1])
        else:
            # e4m3: half a step is 2^-4 of a value, 2^-10 below the smallest normal code
            for got, want in ((k, rows[:, 0]), (v, rows[:, 1])):
                assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 0.0625 * 2.0 ** -10).all()
        q = qkv[r, :HEADS * DIM].view(KV, HEADS // KV, DIM)
        p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * DIM ** -0.5, -1)
        o = torch.einsum("hgt,thd->hgd", p, v).reshape(HEADS, DIM)
        spread = torch.einsum("hgt,thd->hgd", p, v.abs()).reshape(HEADS, DIM)
        assert ((attended[r] - o).abs() <= 2.0 ** -8 * (o.abs() + spread)).all(), r
    out = x.double() + attended.view(block.requests, -1) @ block.w_o.double().t()
    size = attended.abs().view(block.requests, -1) @ block.w_o.double().abs().t()
    assert ((y.double() - out).abs() <= 2.0 ** -8 * out.abs() * 1.01 + 2.0 ** -15 * size).all()


@pytest.mark.parametrize("cache,adapters", [("bf16", 3), ("bf16", 0), ("fp8", 3)])
def test_prompts_then_steps(cache, adapters):
    g = torch.Generator().manual_seed(5)
    requests, prompts = 5, [37, 0, 700, 16, 1]
    block = build(requests, g, cache, adapters)
    ids = [0, 2, -1, 1, 2] if adapters else [-1] * 5
    block.ids.copy_(torch.tensor(ids))
    total = sum(prompts)
    x = rand(g, total + 3, HIDDEN)                      # three rows of padding
    block.admit(x, torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    qkv = block._buffers(total + 3)["qkv"].clone()
    owner = [r for r, n in enumerate(prompts) for _ in range(n)]
    ref, tol = projected(block, x[:total], [ids[r] for r in owner])
    assert ((qkv[:total].double() - ref).abs() <= tol).all()
    kv_rows = [[qkv[t, HEADS * DIM:] for t in range(total) if owner[t] == r] for r in range(requests)]
    lens = list(prompts)
    y = torch.empty(requests, HIDDEN, dtype=torch.bfloat16, device="cuda")
    for fresh in ([1, 1, 1, 1, 1], [1, 0, 1, 0, 1], [0, 0, 0, 1, 0], [1, 1, 1, 1, 1]):
        print(f"decode block step fresh={fresh}", flush=True)
        x = rand(g, requests, HIDDEN)
        block.step(x, torch.tensor(fresh, dtype=torch.int32, device="cuda"), y)
        torch.cuda.synchronize()
        lens = [n + f for n, f in zip(lens, fresh)]
        check_step(block, x, y, ids, fresh, lens, kv_rows)
    pages = [p for r in range(requests) for p in block.table[r, :-(-lens[r] // PAGE)].tolist()]
    assert len(set(pages)) == len(pages) == int(block.head) and min(pages) >= 0


def test_a_captured_step_follows_the_requests():
    """A graph replayed over steps, with eager work between, equals the same steps run eagerly."""
    g = torch.Generator().manual_seed(9)
    requests = 4
    a, b = build(requests, g), None
    b = build(requests, g)
    for name in ("w_qkv", "w_o", "adapters"):
        setattr(b, name, getattr(a, name))
    prompts = torch.tensor([30, 600, 15, 1], dtype=torch.int32, device="cuda")
    x = rand(g, int(prompts.sum()), HIDDEN)
    for block in (a, b):
        block.ids.copy_(torch.tensor([0, 1, 2, -1]))
        block.admit(x, prompts)
    xs, fresh = rand(g, requests, HIDDEN), torch.ones(requests, dtype=torch.int32, device="cuda")
    ya, yb = (torch.empty(requests, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for block, y in ((a, ya), (b, yb)):
        block.step(xs, fresh, y)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            a.step(xs, fresh, ya)
    torch.cuda.current_stream().wait_stream(side)
    for i, f in enumerate([[1, 1, 1, 1], [0, 1, 1, 0], [1, 1, 0, 1], [1, 0, 1, 1]]):
        xs.copy_(rand(g, requests, HIDDEN))
        fresh.copy_(torch.tensor(f))
        if i == 2:                                      # another adapter from here on
            for block in (a, b):
                block.ids.copy_(torch.tensor([2, 2, -1, 0]))
        graph.replay()
        torch.cuda.synchronize()
        b.step(xs, fresh, yb)
        torch.cuda.synchronize()
        for name in ("table", "lens", "cached", "head", "attended"):
            assert torch.equal(getattr(a, name), getattr(b, name)), (i, name)
        assert torch.equal(ya, yb), i


def captured(step):
    """`step` run once and captured."""
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    return graph


def same_block(a, requests, g):
    b = build(requests, g)
    for name in ("w_qkv", "w_o", "adapters"):
        setattr(b, name, getattr(a, name))
    return b


def test_prompts_of_growing_length_between_replays():
    """The prompts' buffers move as they grow, the captured step's do not."""
    g = torch.Generator().manual_seed(21)
    requests = 3
    a = build(requests, g)
    b = same_block(a, requests, g)
    for block in (a, b):
        block.ids.copy_(torch.tensor([0, -1, 2]))
    xs, one = rand(g, requests, HIDDEN), torch.ones(requests, dtype=torch.int32, device="cuda")
    ya, yb = (torch.empty(requests, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b.step(xs, one, yb)
    graph = captured(lambda: a.step(xs, one, ya))       # counts as one step: capturing runs nothing
    for lengths in ([5, 0, 1], [40, 33, 0], [1, 2, 4], [200, 100, 300]):
        print(f"decode block prompts {lengths} between replays", flush=True)
        x = rand(g, sum(lengths), HIDDEN)
        xs.copy_(rand(g, requests, HIDDEN))
        fresh = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for block in (a, b):
            block.admit(x, fresh)
        graph.replay()
        torch.cuda.synchronize()
        b.step(xs, one, yb)
        torch.cuda.synchronize()
        for name in ("table", "lens", "cached", "head", "attended"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        assert torch.equal(ya, yb)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_places_leave_and_run_out_of_pages_between_replays(cache):
    """A captured step over a pool of 12 pages against eager steps over one that never ends: places that find no
    page wait, places that leave give theirs back, and what is attended to is the same bits throughout."""
    from dl_fusion_amd.decode import PagedAttentionBlock
    g = torch.Generator().manual_seed(33)
    requests = 3
    b = build(requests, g, cache)
    a = PagedAttentionBlock(b.w_qkv, b.w_o, HEADS, KV, DIM, requests, 12, PAGE, COLS, b.adapters, cache=cache,
                            k_scale=0.0625, v_scale=0.0625)
    i32 = dict(dtype=torch.int32, device="cuda")
    for block in (a, b):
        block.ids.copy_(torch.tensor([0, -1, 2]))
    xs, fresh = rand(g, requests, HIDDEN), torch.zeros(requests, **i32)
    ya, yb = (torch.empty(requests, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    graph = captured(lambda: a.step(xs, fresh, ya))
    waited = 0

    def admit(lengths):
        x, n = rand(g, sum(lengths), HIDDEN), torch.tensor(lengths, **i32)
        for block in (a, b):
            block.admit(x, n)
        assert not a.short.any() and not b.short.any()

    def steps(count):
        nonlocal waited
        for _ in range(count):
            xs.copy_(rand(g, requests, HIDDEN))
            fresh.fill_(1)
            graph.replay()
            torch.cuda.synchronize()
            waited += int(a.short.sum())
            b.step(xs, fresh - a.short, yb)
            torch.cuda.synchronize()
            assert torch.equal(a.cached, b.cached) and not b.short.any()
            assert torch.equal(a.attended, b.attended) and torch.equal(ya, yb)
            held = [p for r in range(requests) for p in a.table[r, :-(-int(a.cached[r]) // PAGE)].tolist()]
            assert sorted(held + a.free[int(a.head):].tolist()) == list(range(12))

    print(f"decode block, 12 pages, {cache}", flush=True)
    admit([40, 16, 100])
    steps(10)                           # 3 + 1 + 7 pages, and then one more for place 1 and none for place 0
    assert waited and a.cached.tolist()[0] == 48
    for block in (a, b):
        block.release([2])
    steps(3)
    admit([0, 0, 33])
    steps(20)
    for block in (a, b):
        block.release(torch.tensor([True, True, False], device="cuda"))
    admit([70, 1, 0])
    steps(4)
    for block in (a, b):
        block.release(range(requests))
    assert int(a.head) == 0 and (a.table == -1).all() and not a.cached.any()
