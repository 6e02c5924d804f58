"""One attention block of a decoding model over a paged key-value cache, run through the C ABI.

The block is  y = x + attention(x W_qkv^T [+ adapters]) W_o^T  for requests whose keys and values live in
pages of one pool.  A step enqueues, on the current stream and without reading anything back:

    dlf_page_plan        pages and slots for the step's tokens, from the lengths on the device
    dlf_gemm_fused       queries, keys and values in one product
    dlf_lora_add         each request's adapter on it, in place
    dlf_paged_store      the new keys and values into their slots, out of the product's columns
    dlf_paged_attention  each request's new token over its pages
    dlf_gemm_fused       the output projection with the residual

so that it can be captured in a graph and replayed while requests grow, join and leave: their lengths,
tokens, pages and adapters are read from device memory.  ``admit`` brings a request's prompt to a place,
``release`` gives a place's pages back.  Where the pool has no page left, a token is not stored, its
request stays as long as it was, and ``short`` says so.  ``python -m dl_fusion_amd.decode`` runs a batch.
"""
from __future__ import annotations

import torch

from . import (dlf_gemm_fused, dlf_lora_add, dlf_lora_workspace_bytes, dlf_page_plan, dlf_paged_attention,
               dlf_paged_attention_workspace_bytes, dlf_paged_store, gemm_desc, kv_cache_desc, lora_desc,
               page_plan_desc, paged_attn_desc)


def _shaped(t, shape, name, dtype=torch.bfloat16):
    """The products read as many values as their descriptors say, whatever the tensor holds."""
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


class PagedAttentionBlock:
    """``w_qkv`` [(heads + 2 kv_heads) * head_dim][hidden] (queries, keys, values) and ``w_o``
    [hidden][heads * head_dim], bf16 on the device.  ``adapters``: (a [count][rank][hidden],
    b [count][qkv columns][rank], scale [count] or None) or None.  A pool of ``pages`` pages is shared by
    ``requests`` places of up to ``max_pages`` pages each."""

    def __init__(self, w_qkv, w_o, heads, kv_heads, head_dim, requests, pages, page_size, max_pages, adapters=None,
                 cache="bf16", k_scale=1.0, v_scale=1.0, max_len=0):
        self.w_qkv, self.w_o, self.adapters = w_qkv, w_o, adapters
        self.heads, self.kv_heads, self.head_dim, self.requests = heads, kv_heads, head_dim, requests
        self.page_size, self.max_pages = page_size, max_pages
        self.width, self.hidden = w_qkv.shape
        _shaped(w_qkv, ((heads + 2 * kv_heads) * head_dim, self.hidden), "w_qkv")
        _shaped(w_o, (self.hidden, heads * head_dim), "w_o")
        if adapters is not None:
            a, b, scale = adapters
            count, rank, _ = a.shape
            _shaped(a, (count, rank, self.hidden), "the adapters' a")
            _shaped(b, (count, self.width, rank), "the adapters' b")
            if scale is not None:
                _shaped(scale, (count,), "the adapters' scale", torch.float32)
        device = w_qkv.device
        i32 = dict(dtype=torch.int32, device=device)
        self.cache = kv_cache_desc(pages, kv_heads, page_size, head_dim, cache, k_scale, v_scale)
        shape = (pages, kv_heads, page_size, head_dim)
        dtype = torch.float8_e4m3fn if cache == "fp8" else torch.bfloat16
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        # the requests' state: tokens stored, the pages that hold them, adapters; and the pool's free pages from `head`
        # on (one entry more, for release() to write to)
        self.cached = torch.zeros(requests, **i32)
        self.table = torch.full((requests, max_pages), -1, **i32)
        self.ids = torch.full((requests,), -1, **i32)
        self._free = torch.arange(pages + 1, **i32)
        self.free = self._free[:pages]
        self.head = torch.zeros(1, **i32)
        # fresh tokens of the last admit or step, and those of them that were stored; a step's slots, and one for nobody
        self._asked, self._stored = torch.zeros(requests, **i32), torch.zeros(requests, **i32)
        self._slots = torch.empty(requests + 1, dtype=torch.int64, device=device)
        # what a step plans
        self.starts, self.lens = torch.empty(requests + 1, **i32), torch.empty(requests, **i32)
        self.counts = torch.empty(4, **i32)
        self.attn = paged_attn_desc(self.cache, requests, heads, max_pages, softmax_scale=head_dim ** -0.5,
                                    max_len=max_len, q_stride=self.width)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.attended = torch.empty(requests, heads, head_dim, **bf16)
        self.attn_ws = torch.empty(dlf_paged_attention_workspace_bytes(self.attn), dtype=torch.uint8, device=device)
        self._step = self._prompts = None       # buffers, made when they are needed

    def _buffers(self, m):
        """What m rows need.  A step's buffers are its own and stay where they are, as a captured graph needs
        them; batches of prompts of any length share one set, which grows to the longest."""
        if m == self.requests:
            if self._step is None:
                self._step = self._views(m, self._allocate(m))
            return self._step
        if self._prompts is None or self._prompts["rows"].numel() < m or (
                self.adapters is not None and self._prompts["lora_ws"].numel() < self._lora(m)[1]):
            most, ws = (0, 0) if self._prompts is None else (self._prompts[n].numel() for n in ("rows", "lora_ws"))
            self._prompts = None            # before the next is made
            self._prompts = self._allocate(max(m, most), ws)
        return self._views(m, self._prompts)

    def _lora(self, m):
        count, rank, _ = self.adapters[0].shape
        # the rows of a batch of prompts name their requests, those of a step are the requests
        d = lora_desc(m, self.width, self.hidden, rank, count, self.requests)
        return d, dlf_lora_workspace_bytes(d)

    def _allocate(self, m, lora_ws=0):
        device = self.w_qkv.device
        if self.adapters is not None:
            lora_ws = max(lora_ws, self._lora(m)[1])
        return dict(slots=torch.empty(m, dtype=torch.int64, device=device),
                    rows=torch.empty(m, dtype=torch.int32, device=device),
                    qkv=torch.empty(m, self.width, dtype=torch.bfloat16, device=device),
                    lora_ws=torch.empty(lora_ws, dtype=torch.uint8, device=device))

    def _views(self, m, room):
        got = dict(plan=page_plan_desc(self.requests, self.page_size, self.max_pages, m, self.free.numel()),
                   product=gemm_desc(m, self.width, self.hidden), lora_ws=room["lora_ws"],
                   **{n: room[n][:m] for n in ("slots", "rows", "qkv")})
        if self.adapters is not None:
            got["lora"] = self._lora(m)[0]
        return got

    def _project(self, x, b, row_map):
        dlf_gemm_fused(b["product"], x, self.w_qkv, None, None, None, b["qkv"])
        if self.adapters is not None:
            a, up, scale = self.adapters
            dlf_lora_add(b["lora"], x, a, up, scale, self.ids, row_map, b["qkv"], b["qkv"], b["lora_ws"],
                         b["lora_ws"].numel())

    def _store(self, b, slots):
        q = self.heads * self.head_dim
        kv = b["qkv"][:, q:].unflatten(1, (2, self.kv_heads, self.head_dim))
        dlf_paged_store(self.cache, kv[:, 0], kv[:, 1], slots, self.k_cache, self.v_cache)

    def _plan(self, b, fresh):
        dlf_page_plan(b["plan"], self.cached, fresh, self.free, self.head, self.table, self.starts, self.lens,
                      b["slots"], b["rows"], self.counts)
        self.head.copy_(self.counts[1:2])

    @property
    def short(self):
        """[requests] int32: the fresh tokens of the last admit or step that were not stored."""
        return self._asked - self._stored

    def admit(self, x, fresh):
        """Keys and values of prompts into the cache: ``fresh`` [requests] int32, how many tokens each place
        brings, and their rows x [tokens][hidden], request by request (more rows than tokens are padding).  Tokens
        without a row, past the pool's last page or past the place's table are not stored, and counted in ``short``:
        they are the last ones of their place, and may be brought again later.  Not to be captured: a longer batch of
        prompts moves the buffers."""
        _shaped(x, (x.shape[0], self.hidden), "x")
        _shaped(fresh, (self.requests,), "fresh", torch.int32)
        b = self._buffers(x.shape[0])
        fresh = fresh.clamp(min=0)
        # pages for the tokens that have a row only, or they would be nobody's
        before = fresh.cumsum(0) - fresh
        self._plan(b, torch.minimum(fresh, (x.shape[0] - before).clamp(min=0)).to(torch.int32))
        self._project(x, b, b["rows"])
        self._store(b, b["slots"])
        # lengths grow by the tokens that have a slot: missing pages are asked for again by the next plan
        self._asked.copy_(fresh)
        self._stored.zero_().index_add_(0, b["rows"].clamp(min=0), (b["slots"] >= 0).to(torch.int32))
        self.cached.add_(self._stored)

    def step(self, x, fresh, y):
        """One token for every place whose ``fresh`` (int32, 0 or 1) is 1: its row of x [requests][hidden] gives
        its row of y.  Other places attend to what they have cached and store nothing; so does a place whose token
        finds no page, or whose table is full: its ``short`` is 1, its row of y not to be used, and the token may be
        brought again once there are pages."""
        for t, name in ((x, "x"), (y, "y")):
            _shaped(t, (self.requests, self.hidden), name)
        _shaped(fresh, (self.requests,), "fresh", torch.int32)
        b = self._buffers(self.requests)
        self._plan(b, torch.gt(fresh, 0, out=self._asked))
        self._project(x, b, None)
        # the plan numbers the tokens, row r of x is place r; rows that no token has are -1, the last entry
        self._slots.fill_(-1)[b["rows"]] = b["slots"]
        self._store(b, self._slots[:-1])
        self.cached.add_(torch.ge(self._slots[:-1], 0, out=self._stored))
        q = b["qkv"][:, :self.heads * self.head_dim].unflatten(1, (self.heads, self.head_dim))
        dlf_paged_attention(self.attn, q, self.k_cache, self.v_cache, self.table, self.cached, self.attended, None,
                            self.attn_ws, self.attn_ws.numel())
        dlf_gemm_fused(gemm_desc(self.requests, self.hidden, self.heads * self.head_dim),
                       self.attended.view(self.requests, -1), self.w_o, None, None, x, y)

    def release(self, leaving):
        """Gives the pages of the places ``leaving`` (bool [requests], or their numbers) back to the pool and
        empties the places.  Enqueued like a step, between steps or replays."""
        if not isinstance(leaving, torch.Tensor):
            gone = set(leaving)
            leaving = torch.tensor([r in gone for r in range(self.requests)], device=self.cached.device)
        cols = torch.arange(self.max_pages, device=self.cached.device)
        held = leaving[:, None] & (cols < -(-self.cached // self.page_size)[:, None])
        back = held.flatten().cumsum(0)
        # the list's entries before `head` are taken pages', so that those that come back fit there
        to = torch.where(held.flatten(), self.head - back[-1:] + back - 1, self.free.numel())
        self._free.scatter_(0, to, self.table.flatten())
        self.head.sub_(back[-1:])
        self.table.masked_fill_(leaving[:, None], -1)
        self.cached.masked_fill_(leaving, 0)
        self._asked.masked_fill_(leaving, 0)
        self._stored.masked_fill_(leaving, 0)


def main():
    import argparse
    ap = argparse.ArgumentParser(description="decode steps of one attention block over a paged cache")
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=["bf16", "fp8"], default="bf16")
    ap.add_argument("--adapters", type=int, default=8)
    a = ap.parse_args()
    hidden, heads, kv_heads, dim, page, rank = 4096, 32, 8, 128, 16, 16
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)

    width = (heads + 2 * kv_heads) * dim
    max_pages = -(-(a.prompt + a.steps + 8) // page)
    adapters = None
    if a.adapters:
        adapters = (rand(a.adapters, rank, hidden, scale=hidden ** -0.5), rand(a.adapters, width, rank, scale=0.1), None)
    block = PagedAttentionBlock(rand(width, hidden, scale=hidden ** -0.5), rand(hidden, heads * dim, scale=hidden ** -0.5),
                                heads, kv_heads, dim, a.requests, a.requests * max_pages, page, max_pages, adapters,
                                cache=a.cache, k_scale=0.0625, v_scale=0.0625, max_len=max_pages * page)
    if a.adapters:
        block.ids.copy_(torch.arange(a.requests) % a.adapters)
    prompts = [max(1, a.prompt * (i + 1) // a.requests) for i in range(a.requests)]
    fresh = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    block.admit(rand(sum(prompts), hidden), fresh)
    x, y = rand(a.requests, hidden), torch.empty(a.requests, hidden, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    block.step(x, one, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, one, y)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) / a.steps * 1e3
    print(f"{a.requests} requests, longest {int(block.counts[2])} tokens, {a.cache} cache, {a.adapters} adapters: "
          f"{us:.1f} us a step, {a.requests / us * 1e6:.0f} tokens/s")


if __name__ == "__main__":
    main()
