"""CPU tests of the decode operators' argument checks.  Nothing here launches a kernel: every call
is rejected, or is a zero-size no-op, before any HIP call."""
import ctypes

import pytest

dlf = pytest.importorskip("dl_fusion_amd", reason="libdlfusion.so not built")
from test_host_lib import fake_pointers  # noqa: E402

INVALID, UNSUPPORTED, ALIAS = dlf.DLF_ERR_INVALID_ARG, dlf.DLF_ERR_UNSUPPORTED, dlf.DLF_ERR_ALIAS
MB = 1 << 20


def addr(i, off=0):
    """Fake device addresses, 64 GB apart, never dereferenced."""
    return (i + 1) * (64 << 30) + off


def ref(d):
    return None if d is None else ctypes.byref(d)


# ---------------------------------------------------------------------------
# Page plan
# ---------------------------------------------------------------------------
PLAN_PTRS = ("cached", "fresh", "free_pages", "free_head", "block_table", "starts", "lens", "slots", "rows", "counts")


def call_plan(desc=(8, 16, 4, 32, 64), **ptrs):
    p = {n: addr(i) for i, n in enumerate(PLAN_PTRS)}
    p.update(ptrs)
    d = None if desc is None else dlf.page_plan_desc(*desc)
    return dlf.raw().dlf_page_plan(ref(d), *[p[n] for n in PLAN_PTRS], None)


@fake_pointers
def test_page_plan_refusals():
    assert call_plan(None) == INVALID
    for bad in [(-1, 16, 4, 32, 64), (8, 0, 4, 32, 64), (8, 16, 0, 32, 64), (8, 16, 4, -1, 64), (8, 16, 4, 32, -1),
                (8, -16, 4, 32, 64)]:
        assert call_plan(bad) == INVALID, bad
    assert call_plan((65537, 16, 4, 32, 64)) == UNSUPPORTED
    assert call_plan((8, 1 << 16, 1 << 15, 32, 64)) == UNSUPPORTED
    for n in ("cached", "fresh", "free_pages", "block_table", "starts", "lens", "slots", "counts"):
        assert call_plan(**{n: None}) == INVALID, n
    for n in PLAN_PTRS:
        assert call_plan(**{n: addr(40, 2)}) == INVALID, n
    assert call_plan(slots=addr(40, 4)) == INVALID
    assert "aligned" in dlf.dlf_last_error()
    # an output over an input, two outputs over each other, an output over the free list's head
    assert call_plan(lens=addr(0, 28)) == ALIAS
    assert call_plan(rows=addr(7, 8 * 32 - 4)) == ALIAS
    assert call_plan(counts=addr(3)) == ALIAS


# ---------------------------------------------------------------------------
# Store
# ---------------------------------------------------------------------------
def cache(**kw):
    args = dict(pages=8, kv_heads=2, page_size=16, head_dim=64, dtype="bf16", k_scale=1.0, v_scale=1.0)
    args.update(kw)
    return dlf.kv_cache_desc(**args)


BAD_CACHES = [
    (dict(dtype=7), INVALID), (dict(dtype="f32"), UNSUPPORTED), (dict(pages=0), INVALID), (dict(pages=-3), INVALID),
    (dict(kv_heads=0), INVALID), (dict(page_size=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=65536), UNSUPPORTED), (dict(kv_heads=5000), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED), (dict(dtype="fp8", k_scale=0.0), INVALID),
    (dict(dtype="fp8", v_scale=-1.0), INVALID), (dict(dtype="fp8", k_scale=float("nan")), INVALID),
    (dict(dtype="fp8", v_scale=float("inf")), INVALID), (dict(dtype="fp8", k_scale=1e-45), INVALID),
]


def call_store(c, tokens=4, ks=128, vs=128, k=addr(0), v=addr(1), slots=addr(2), kc=addr(3), vc=addr(4)):
    return dlf.raw().dlf_paged_store(ref(c), tokens, k, ks, v, vs, slots, kc, vc, None)


@fake_pointers
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_store_refuses_bad_caches(kw, status):
    assert call_store(cache(**kw)) == status


@fake_pointers
def test_store_refusals():
    c = cache()
    assert call_store(None) == INVALID
    assert call_store(c, tokens=-1) == INVALID
    assert call_store(c, tokens=(1 << 30) + 1) == UNSUPPORTED
    assert call_store(c, tokens=0, k=None, kc=None) == dlf.DLF_OK
    assert call_store(c, ks=120) == INVALID
    assert call_store(c, vs=132) == UNSUPPORTED
    assert call_store(c, vs=(1 << 31) + 8) == UNSUPPORTED
    for n in ("k", "v", "slots", "kc", "vc"):
        assert call_store(c, **{n: None}) == INVALID, n
    for n in ("k", "v", "kc", "vc"):
        assert call_store(c, **{n: addr(40, 8)}) == INVALID, n
    assert call_store(c, slots=addr(40, 4)) == INVALID
    size = 8 * 2 * 16 * 64 * 2
    assert call_store(c, vc=addr(3, size - 16)) == ALIAS
    assert call_store(c, kc=addr(0, (3 * 128 + 128) * 2 - 16)) == ALIAS
    # with rows 256 apart the last row ends later
    assert call_store(c, ks=256, kc=addr(0, (3 * 256 + 128) * 2 - 16)) == ALIAS
    assert call_store(c, slots=addr(4, 64)) == ALIAS


def test_store_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    c = cache()
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    for bad in (k[:, :, ::2], k[:, :1], k.view(4, 128), k.transpose(0, 1)):
        with pytest.raises(ValueError):
            dlf.dlf_paged_store(c, bad, bad, slots, k, k, stream=0)
    with pytest.raises(ValueError):
        dlf.dlf_paged_store(c, k, k, slots[:3], k, k, stream=0)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
ATTN_PTRS = ("q", "k_cache", "v_cache", "block_table", "lens", "out", "lse", "workspace")


def attn(c=None, **kw):
    args = dict(requests=4, heads=8, max_pages=4, softmax_scale=0.125)
    args.update(kw)
    return dlf.paged_attn_desc(cache() if c is None else c, **args)


def call_attn(d, ws_bytes=1 << 30, **ptrs):
    p = {n: addr(i) for i, n in enumerate(ATTN_PTRS)}
    p.update(ptrs)
    return dlf.raw().dlf_paged_attention(ref(d), *[p[n] for n in ATTN_PTRS], ws_bytes, None)


def attn_bytes(d):
    n = ctypes.c_size_t(123)
    st = dlf.raw().dlf_paged_attention_workspace_bytes(ref(d), ctypes.byref(n))
    return st, n.value


BAD_ATTN = [
    (dict(requests=-1), INVALID), (dict(window=-1), INVALID), (dict(max_len=-1), INVALID), (dict(max_pages=0), INVALID),
    (dict(heads=0), INVALID), (dict(heads=7), INVALID), (dict(heads=-8), INVALID),
    (dict(softmax_scale=float("nan")), INVALID), (dict(softmax_scale=float("inf")), INVALID),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(heads=2 * 257), UNSUPPORTED), (dict(requests=65537), UNSUPPORTED),
    (dict(q_stride=8 * 64 - 8), INVALID), (dict(q_stride=8 * 64 + 4), UNSUPPORTED),
    (dict(q_stride=(1 << 31) + 8), UNSUPPORTED),
]


@fake_pointers
@pytest.mark.parametrize("kw,status", BAD_ATTN)
def test_attention_refuses_bad_descriptors(kw, status):
    assert call_attn(attn(**kw)) == status
    assert attn_bytes(attn(**kw)) == (status, 0)


@fake_pointers
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_attention_refuses_bad_caches(kw, status):
    heads = 8 if kw.get("kv_heads", 2) != 5000 else 5000
    assert call_attn(attn(cache(**kw), heads=heads)) == status


@fake_pointers
def test_attention_refusals():
    d = attn()
    assert call_attn(None) == INVALID
    assert attn_bytes(None) == (INVALID, 0)
    assert dlf.raw().dlf_paged_attention_workspace_bytes(ref(d), None) == INVALID
    assert call_attn(attn(requests=0), q=None, out=None, workspace=None) == dlf.DLF_OK
    for n in ("q", "k_cache", "v_cache", "block_table", "lens", "out"):
        assert call_attn(d, **{n: None}) == INVALID, n
    for n in ("q", "k_cache", "v_cache", "out"):
        assert call_attn(d, **{n: addr(40, 8)}) == INVALID, n
    for n in ("block_table", "lens", "lse"):
        assert call_attn(d, **{n: addr(40, 2)}) == INVALID, n
    rows = 4 * 8 * 64 * 2
    assert call_attn(d, out=addr(0, rows - 16)) == ALIAS
    assert call_attn(d, out=addr(1)) == ALIAS
    assert call_attn(d, lse=addr(4, 12)) == ALIAS
    assert call_attn(d, lse=addr(5, rows - 4)) == ALIAS
    assert call_attn(attn(q_stride=1024), out=addr(0, (3 * 1024 + 512) * 2 - 16)) == ALIAS


@fake_pointers
def test_attention_workspace():
    """Needed where a request may be long enough to be cut, whatever says how long it may be."""
    for kw in (dict(max_pages=4, page=16), dict(max_pages=1 << 16, max_len=512), dict(max_pages=1 << 16, window=512),
               dict(max_pages=1 << 16, requests=5000), dict(max_pages=1 << 16, requests=0)):
        page = kw.pop("page", 16)
        assert attn_bytes(attn(cache(page_size=page), **kw)) == (dlf.DLF_OK, 0), kw
    d = attn(max_pages=1 << 16)
    st, need = attn_bytes(d)
    assert st == dlf.DLF_OK and need > 0
    assert call_attn(d, workspace=None) == INVALID and "workspace" in dlf.dlf_last_error()
    assert call_attn(d, ws_bytes=need - 1) == INVALID
    assert call_attn(d, workspace=addr(40, 8)) == INVALID
    for i, n in enumerate(ATTN_PTRS):
        if n != "workspace":
            assert call_attn(d, workspace=addr(i)) == ALIAS, n


def test_attention_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    d = attn()
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    wide = torch.zeros(4, 1024, dtype=torch.bfloat16)[:, :512].unflatten(1, (8, 64))
    i = torch.zeros(4, 4, dtype=torch.int32)
    for bad in (q[:3], q[:, :4], q.transpose(0, 1), q[:, :, ::2], q.view(4, 512), wide):
        with pytest.raises(ValueError):
            dlf.dlf_paged_attention(d, bad, q, q, i, i[0], q, None, None, 0, stream=0)


# ---------------------------------------------------------------------------
# Adapters
# ---------------------------------------------------------------------------
LORA_PTRS = ("x", "a", "b", "scale", "ids", "row_map", "base", "out", "workspace")


def lora(**kw):
    args = dict(m=5, n=64, k=96, rank=16, adapters=3, requests=2)
    args.update(kw)
    return dlf.lora_desc(**args)


def call_lora(d, ws_bytes=1 << 30, **ptrs):
    p = {n: addr(i) for i, n in enumerate(LORA_PTRS)}
    p.update(ptrs)
    return dlf.raw().dlf_lora_add(ref(d), *[p[n] for n in LORA_PTRS], ws_bytes, None)


def lora_bytes(d):
    n = ctypes.c_size_t(123)
    st = dlf.raw().dlf_lora_workspace_bytes(ref(d), ctypes.byref(n))
    return st, n.value


BAD_LORA = [
    (dict(dtype="f32"), UNSUPPORTED), (dict(dtype="fp8"), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(m=-1), INVALID), (dict(n=-8), INVALID), (dict(k=-8), INVALID), (dict(rank=-8), INVALID),
    (dict(adapters=-1), INVALID), (dict(requests=-1), INVALID), (dict(rank=0), UNSUPPORTED), (dict(rank=12), UNSUPPORTED),
    (dict(rank=136), UNSUPPORTED), (dict(n=60), UNSUPPORTED), (dict(k=100), UNSUPPORTED),
    (dict(n=(1 << 23) + 8), UNSUPPORTED), (dict(k=(1 << 23) + 8), UNSUPPORTED), (dict(m=(1 << 24) + 1), UNSUPPORTED),
    (dict(x_stride=88), INVALID), (dict(base_stride=56), INVALID), (dict(out_stride=56), INVALID),
    (dict(x_stride=100), UNSUPPORTED), (dict(base_stride=68), UNSUPPORTED), (dict(out_stride=(1 << 31) + 8), UNSUPPORTED),
]


@fake_pointers
@pytest.mark.parametrize("kw,status", BAD_LORA)
def test_adapters_refuse_bad_descriptors(kw, status):
    assert call_lora(lora(**kw)) == status
    assert lora_bytes(lora(**kw)) == (status, 0)


@fake_pointers
def test_adapters_refusals():
    d = lora()
    st, need = lora_bytes(d)
    assert st == dlf.DLF_OK and need >= 5 * 16 * 4
    assert call_lora(None) == INVALID and lora_bytes(None) == (INVALID, 0)
    assert dlf.raw().dlf_lora_workspace_bytes(ref(d), None) == INVALID
    assert call_lora(lora(m=0), x=None, out=None, workspace=None) == dlf.DLF_OK
    assert call_lora(lora(n=0), out=None, workspace=None) == dlf.DLF_OK
    assert lora_bytes(lora(m=0)) == (dlf.DLF_OK, 0)
    for n in ("x", "a", "b", "ids", "out", "workspace"):
        assert call_lora(d, **{n: None}) == INVALID, n
    for n in ("x", "a", "b", "base", "out", "workspace"):
        assert call_lora(d, **{n: addr(40, 8)}) == INVALID, n
    for n in ("scale", "ids", "row_map"):
        assert call_lora(d, **{n: addr(40, 2)}) == INVALID, n
    assert call_lora(d, ws_bytes=need - 1) == INVALID
    assert "workspace" in dlf.dlf_last_error()
    for n, size in (("x", 5 * 96 * 2), ("a", 3 * 16 * 96 * 2), ("b", 3 * 16 * 64 * 2), ("scale", 12), ("ids", 8),
                    ("row_map", 20)):
        last = addr(LORA_PTRS.index(n), (size - 1) // 16 * 16)
        assert call_lora(d, out=last) == ALIAS, n
        assert call_lora(d, workspace=last) == ALIAS, n
    # base may be out itself, not part of it, nor with another stride
    base = addr(LORA_PTRS.index("base"))
    assert call_lora(d, out=base + 128) == ALIAS
    assert call_lora(lora(out_stride=128), out=base) == ALIAS
    assert call_lora(d, workspace=base) == ALIAS
    assert call_lora(d, workspace=addr(LORA_PTRS.index("out"))) == ALIAS


def test_adapters_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    d = lora()
    x, y = torch.zeros(5, 96, dtype=torch.bfloat16), torch.zeros(5, 64, dtype=torch.bfloat16)
    w = torch.zeros(4096, dtype=torch.uint8)
    wide = torch.zeros(5, 128, dtype=torch.bfloat16)[:, :96]
    for bx, by in ((x[:4], y), (wide, y), (x.t(), y), (x, y[:, :32]), (x, y.view(5, 8, 8))):
        with pytest.raises(ValueError):
            dlf.dlf_lora_add(d, bx, x, x, None, x, None, None, by, w, 4096, stream=0)


# ---------------------------------------------------------------------------
# Sizes that no launch can have: 2^24 workgroups of 256 threads
# ---------------------------------------------------------------------------
@fake_pointers
def test_sizes_beyond_a_launch_are_refused():
    wide = cache(kv_heads=256)
    assert attn_bytes(attn(wide, heads=256, requests=65535)) == (dlf.DLF_OK, 0)
    for d in (attn(wide, heads=256, requests=65536), attn(cache(kv_heads=128), heads=128 * 17, requests=65536),
              attn(cache(kv_heads=1), heads=256, requests=65536, max_pages=1 << 20)):
        refused = d.requests * d.cache.kv_heads * -(-d.heads // d.cache.kv_heads // 16) >= 1 << 24
        assert attn_bytes(d) == ((UNSUPPORTED, 0) if refused else (dlf.DLF_OK, 0)), (d.heads, refused)
        if refused:
            assert call_attn(d) == UNSUPPORTED and "2^24" in dlf.dlf_last_error()
    # 4 tokens a workgroup from 1032 values a token on, 128 at 64 values
    for heads, dim, first in ((32, 256, (1 << 26) - 3), (17, 64, (1 << 26) - 3), (16, 64, (1 << 27) - 7),
                              (4, 64, (1 << 29) - 31)):
        c, w = cache(kv_heads=heads, head_dim=dim), heads * dim
        assert call_store(c, tokens=first, ks=w, vs=w) == UNSUPPORTED, (heads, dim)
        assert "values must stay below %d" % first in dlf.dlf_last_error()
        # one less passes this check, and is refused for a pointer
        assert call_store(c, tokens=first - 1, ks=w, vs=w, k=None) == INVALID, (heads, dim)


# ---------------------------------------------------------------------------
# The binding compares its tensors with the descriptor
# ---------------------------------------------------------------------------
def _calls():
    """entry point -> (call of a dict of tensors, the tensors); all as they should be."""
    import torch
    i32, i64, bf16, f32 = torch.int32, torch.int64, torch.bfloat16, torch.float32
    z = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    c, c8 = cache(), cache(dtype="fp8")
    plan = dlf.page_plan_desc(8, 16, 4, 32, 64)
    pool = (8, 2, 16, 64)
    d = attn(max_pages=1 << 12)
    size = dlf.dlf_paged_attention_workspace_bytes(d)
    lo = lora()
    lsize = dlf.dlf_lora_workspace_bytes(lo)
    u8 = torch.uint8
    return {
        "plan": (lambda t: dlf.dlf_page_plan(plan, *t.values(), stream=0),
                 dict(cached=z(i32, 8), fresh=z(i32, 8), free_pages=z(i32, 64), free_head=z(i32, 1),
                      block_table=z(i32, 8, 4), starts=z(i32, 9), lens=z(i32, 8), slots=z(i64, 32), rows=z(i32, 32),
                      counts=z(i32, 4))),
        "store": (lambda t: dlf.dlf_paged_store(c, *t.values(), stream=0),
                  dict(k=z(bf16, 4, 2, 64), v=z(bf16, 4, 2, 64), slots=z(i64, 4), k_cache=z(bf16, *pool),
                       v_cache=z(bf16, *pool))),
        "store fp8": (lambda t: dlf.dlf_paged_store(c8, *t.values(), stream=0),
                      dict(k=z(bf16, 4, 2, 64), v=z(bf16, 4, 2, 64), slots=z(i64, 4),
                           k_cache=z(torch.float8_e4m3fn, *pool), v_cache=z(u8, *pool))),
        "attention": (lambda t: dlf.dlf_paged_attention(d, *t.values(), size, stream=0),
                      dict(q=z(bf16, 4, 8, 64), k_cache=z(bf16, *pool), v_cache=z(bf16, *pool),
                           block_table=z(i32, 4, 1 << 12), lens=z(i32, 4), out=z(bf16, 4, 8, 64), lse=z(f32, 4, 8),
                           workspace=z(u8, size))),
        "adapters": (lambda t: dlf.dlf_lora_add(lo, *t.values(), lsize, stream=0),
                     dict(x=z(bf16, 5, 96), a=z(bf16, 3, 16, 96), b=z(bf16, 3, 64, 16), scale=z(f32, 3), ids=z(i32, 2),
                          row_map=z(i32, 5), base=z(bf16, 5, 64), out=z(bf16, 5, 64), workspace=z(u8, lsize))),
    }


@fake_pointers
@pytest.mark.parametrize("name", ["plan", "store", "store fp8", "attention", "adapters"])
def test_binding_refuses_arrays_unlike_the_descriptor(name):
    """Short ones, another type's and ones with gaps; every operand in turn."""
    torch = pytest.importorskip("torch")
    call, good = _calls()[name]
    with pytest.raises(dlf.DlfError) as e:      # as they should be: it gets as far as the launch
        call(good)
    assert e.value.status == dlf.DLF_ERR_HIP
    for n, t in good.items():
        short = t.reshape(-1)[:-1]
        gaps = torch.zeros(2 * t.numel(), dtype=t.dtype).view(*t.shape[:-1], -1)[..., ::2]
        other = [] if n == "workspace" else [t.to({torch.int32: torch.int64, torch.int64: torch.int32}.get(t.dtype, torch.float16))]
        if n == "free_head":                    # one number: nothing can lie between
            gaps = short
        for bad in (short, gaps, *other):
            with pytest.raises(ValueError):
                call({**good, n: bad})
    if "block_table" in good:
        t = good["block_table"]
        for cols in (t.shape[1] - 1, t.shape[1] + 1):
            with pytest.raises(ValueError, match="max_pages"):
                call({**good, "block_table": torch.zeros(t.shape[0], cols, dtype=torch.int32)})


@fake_pointers
def test_binding_wants_an_id_for_every_row_or_request():
    torch = pytest.importorskip("torch")
    call, good = _calls()["adapters"]
    with pytest.raises(ValueError, match="ids"):        # without a row map there are m of them, not `requests`
        call({**good, "row_map": None})
    with pytest.raises(dlf.DlfError):
        call({**good, "row_map": None, "ids": torch.zeros(5, dtype=torch.int32)})


# ---------------------------------------------------------------------------
# The attention block (dl_fusion_amd/decode.py): its buffers, made on the CPU
# ---------------------------------------------------------------------------
def block_on_the_cpu(adapters=True, requests=4, pages=64):
    torch = pytest.importorskip("torch")
    from dl_fusion_amd.decode import PagedAttentionBlock
    w = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    ad = (w(3, 16, 128), w(3, 512, 16), None) if adapters else None
    return PagedAttentionBlock(w(512, 128), w(128, 256), 4, 2, 64, requests, pages, 16, 16, ad)


def tensor_bytes():
    import gc
    import torch
    gc.collect()
    stores = [o.untyped_storage() for o in gc.get_objects() if issubclass(type(o), torch.Tensor)]
    return sum({s.data_ptr(): s.nbytes() for s in stores}.values())


@pytest.mark.parametrize("adapters", [False, True])
def test_prompts_of_any_length_share_their_buffers(adapters):
    block = block_on_the_cpu(adapters)
    step = block._buffers(4)
    start = tensor_bytes()
    block._buffers(3000)
    longest = tensor_bytes() - start
    assert longest >= 3000 * 512 * 2
    for m in [*range(5, 700, 13), 2999, 3000, 1]:
        b = block._buffers(m)
        assert [b[n].shape[0] for n in ("slots", "rows", "qkv")] == [m, m, m] and b["qkv"].is_contiguous()
        if adapters:
            assert b["lora"].m == m and b["lora_ws"].numel() >= dlf.dlf_lora_workspace_bytes(b["lora"])
        assert b["plan"].token_cap == m
        del b
    assert tensor_bytes() - start <= longest * 1.5          # a short batch's workspace may be the larger one
    again = block._buffers(4)
    assert all(again[n].data_ptr() == step[n].data_ptr() for n in ("slots", "rows", "qkv", "lora_ws") if n in step)


# ---------------------------------------------------------------------------
# The block's bookkeeping, its kernels replaced by Python on the CPU: places join, grow, leave and run out of
# pages, and every place holds just the tokens that a plain list of them says
# ---------------------------------------------------------------------------
PAGE, COLS = 16, 4


def up(n):
    return -(-n // PAGE)


@pytest.fixture
def kernels_in_python(monkeypatch):
    from dl_fusion_amd import decode
    cells, attended = {}, {}

    def plan(desc, cached, fresh, free, head, table, starts, lens, slots, rows, counts):
        cap, want, at = desc.max_pages * PAGE, int(head), 0
        slots.fill_(-1)
        rows.fill_(-1)
        for r in range(desc.requests):
            c, f = int(cached[r]), max(int(fresh[r]), 0)
            starts[r], lens[r] = at, min(c + f, cap)
            for col in range(up(min(c, cap)), up(int(lens[r]))):
                table[r, col] = free[want] if want < desc.free_cap else -1
                want += 1
            for pos in range(c, c + f):
                page = int(table[r, pos // PAGE]) if pos < cap else -1
                if at < desc.token_cap:
                    slots[at], rows[at] = (page * PAGE + pos % PAGE if page >= 0 else -1), r
                at += 1
        starts[desc.requests] = at
        counts[0], counts[1], counts[2] = at, min(want, desc.free_cap), int(lens.max())
        counts[3] = max(0, want - desc.free_cap)

    def product(desc, a, b, scale, shift, residual, c):
        c.copy_(a[:, :1].expand_as(c))          # a row's token number in all its columns

    def store(cache, k, v, slots, k_cache, v_cache):
        taken = [s for s in slots.tolist() if s >= 0]
        assert len(set(taken)) == len(taken) and k.shape[0] == len(slots)
        cells.update({s: int(k[i, 0, 0]) for i, s in enumerate(slots.tolist()) if s >= 0})

    def attention(desc, q, k_cache, v_cache, table, lens, out, lse, ws, size):
        attended["lens"], attended["table"] = lens.tolist(), table.tolist()
        out.zero_()

    for name, fn in (("dlf_page_plan", plan), ("dlf_gemm_fused", product), ("dlf_paged_store", store),
                     ("dlf_paged_attention", attention)):
        monkeypatch.setattr(decode, name, fn)
    return cells, attended


class Places:
    """What the block should hold: a list of token numbers a place, and the number of pages."""

    def __init__(self, requests, pages):
        self.tokens, self.pages = [[] for _ in range(requests)], pages

    def bring(self, news, rows):
        """news: [place] -> token numbers; returns how many are not stored."""
        free, short = self.pages - sum(up(len(t)) for t in self.tokens), []
        for t, new in zip(self.tokens, news):
            given = new[:rows]
            rows -= len(given)
            most = up(len(t)) + min(max(0, free), COLS - up(len(t)))
            fits = given[:max(0, PAGE * most - len(t))]
            free -= up(len(t) + len(fits)) - up(len(t))
            t += fits
            short.append(len(new) - len(fits))
        return short


def check_places(block, places, cells):
    assert block.cached.tolist() == [len(t) for t in places.tokens]
    pages = []
    for r, t in enumerate(places.tokens):
        mine = block.table[r, :up(len(t))].tolist()
        assert [cells[mine[i // PAGE] * PAGE + i % PAGE] for i in range(len(t))] == t, r
        pages += mine
    assert int(block.head) == len(pages)
    assert sorted(pages + block.free[len(pages):].tolist()) == list(range(places.pages))


@pytest.mark.parametrize("seed", range(6))
def test_places_join_grow_leave_and_run_out(kernels_in_python, seed):
    import random
    torch = pytest.importorskip("torch")
    cells, attended = kernels_in_python
    rng = random.Random(seed)
    requests, pages = 5, [1, 9, 11, 13, 20, 0][seed] or 7
    from dl_fusion_amd.decode import PagedAttentionBlock
    w = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    block = PagedAttentionBlock(w(512, 128), w(128, 256), 4, 2, 64, requests, pages, PAGE, COLS)
    places, number = Places(requests, pages), 0
    y = w(requests, 128)

    def numbers(count):
        nonlocal number
        number += count
        return [(number - count + i) % 251 for i in range(count)]       # bf16 has integers to 256

    def rows(tokens):
        x = w(len(tokens), 128)
        x[:, 0] = torch.tensor(tokens, dtype=torch.float32)
        return x

    ran_out = left = 0
    for _ in range(120):
        what = rng.choice(["admit", "step", "step", "step", "release"])
        if what == "admit":
            lengths = [rng.choice([0, 0, 1, rng.randrange(80)]) for _ in range(requests)]
            news = [numbers(n) for n in lengths]
            flat = [t for n in news for t in n]
            m = max(1, len(flat) + rng.choice([0, 0, 3, -2, -30]))
            if m == requests:
                continue
            short = places.bring(news, m)
            block.admit(rows((flat + [250] * 3)[:m]), torch.tensor(lengths, dtype=torch.int32))
        elif what == "step":
            fresh = [rng.choice([0, 1, 1, 1, -3, 2]) for _ in range(requests)]
            tokens = numbers(requests)
            short = places.bring([[t] if f > 0 else [] for t, f in zip(tokens, fresh)], requests)
            block.step(rows(tokens), torch.tensor(fresh, dtype=torch.int32), y)
            assert attended["lens"] == [len(t) for t in places.tokens]
            for r, t in enumerate(places.tokens):
                assert min(attended["table"][r][:up(len(t))], default=0) >= 0
        else:
            leaving = [r for r in range(requests) if rng.random() < 0.3]
            for r in leaving:
                left += len(places.tokens[r])
                places.tokens[r] = []
            flags = torch.tensor([r in leaving for r in range(requests)])
            block.release(leaving if rng.random() < 0.5 else flags)
            short = [0 if r in leaving else n for r, n in enumerate(short)] if _ else [0] * requests
        check_places(block, places, cells)
        assert block.short.tolist() == short, what
        ran_out += sum(short) > 0
    assert ran_out and left


def test_block_refuses_tensors_of_other_shapes(kernels_in_python):
    torch = pytest.importorskip("torch")
    from dl_fusion_amd.decode import PagedAttentionBlock
    w = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    args = lambda **kw: {**dict(w_qkv=w(512, 128), w_o=w(128, 256), heads=4, kv_heads=2, head_dim=64, requests=3,  # noqa: E731
                                pages=9, page_size=PAGE, max_pages=COLS), **kw}
    PagedAttentionBlock(**args())
    for bad in (dict(w_qkv=w(448, 128)), dict(w_o=w(128, 512)), dict(w_o=w(64, 256)), dict(w_qkv=w(512, 128, dtype=torch.float32)),
                dict(adapters=(w(3, 16, 64), w(3, 512, 16), None)), dict(adapters=(w(3, 16, 128), w(2, 512, 16), None)),
                dict(adapters=(w(3, 16, 128), w(3, 512, 8), None)), dict(adapters=(w(3, 16, 128), w(3, 512, 16), w(3)))):
        with pytest.raises(ValueError):
            PagedAttentionBlock(**args(**bad))
    block = PagedAttentionBlock(**args())
    x, y, one = w(3, 128), w(3, 128), torch.ones(3, dtype=torch.int32)
    for call in (lambda: block.step(x[:2], one, y), lambda: block.step(x, one, y[:, :64]), lambda: block.step(x, one[:2], y),
                 lambda: block.step(x, one.long(), y), lambda: block.step(x, one, y.float()),
                 lambda: block.admit(w(7, 64), one), lambda: block.admit(w(7, 128), one[:2]),
                 lambda: block.admit(w(7, 128), one.bool())):
        with pytest.raises(ValueError):
            call()
    block.step(x, one, y)
    block.admit(w(7, 128), one)
