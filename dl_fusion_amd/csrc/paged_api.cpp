// C ABI of the paged key-value cache: the page plan, the store and the attention that reads it.  Every check happens before
// the first HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/dlfusion.h"
#include "checks.h"
#include "kernels.h"
#include "status.h"

namespace {

using dlf::aligned;
using dlf::any_overlap;
using dlf::fail;
using dlf::ok;
using dlf::rows_bytes;

constexpr int64_t kMaxStride = int64_t(1) << 31;

dlf_status check_cache(const dlf_kv_cache_desc* c) {
    if (c->dtype != DLF_BF16 && c->dtype != DLF_FP8_E4M3) {
        if (c->dtype != DLF_F32) return fail(DLF_ERR_INVALID_ARG, "unknown cache dtype %d", static_cast<int>(c->dtype));
        return fail(DLF_ERR_UNSUPPORTED, "a paged cache is bf16 or fp8");
    }
    if (c->pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->head_dim < 1)
        return fail(DLF_ERR_INVALID_ARG, "pages, kv_heads, page_size and head_dim must be positive");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(DLF_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", c->head_dim);
    if (c->page_size % 16 != 0 || c->page_size > 32768)
        return fail(DLF_ERR_UNSUPPORTED, "page_size must be a multiple of 16, at most 32768 (got %d)", c->page_size);
    if (c->kv_heads > 4096) return fail(DLF_ERR_UNSUPPORTED, "more than 4096 kv heads");
    if (static_cast<int64_t>(c->pages) * c->page_size >= (int64_t(1) << 31))
        return fail(DLF_ERR_UNSUPPORTED, "pages * page_size must stay below 2^31");
    if (c->dtype == DLF_FP8_E4M3 &&
        !(std::isfinite(c->k_scale) && std::isfinite(c->v_scale) && c->k_scale > 0 && c->v_scale > 0 &&
          std::isfinite(1.0f / c->k_scale) && std::isfinite(1.0f / c->v_scale)))
        return fail(DLF_ERR_INVALID_ARG, "the scales of an fp8 cache and their inverses must be finite and positive");
    return ok();
}

size_t cache_bytes(const dlf_kv_cache_desc* c) {
    return static_cast<size_t>(c->pages) * static_cast<size_t>(c->kv_heads) * static_cast<size_t>(c->page_size) *
           static_cast<size_t>(c->head_dim) * (c->dtype == DLF_BF16 ? 2 : 1);
}

}  // namespace

extern "C" dlf_status dlf_page_plan(const dlf_page_plan_desc* d, const int32_t* cached, const int32_t* fresh,
                                    const int32_t* free_pages, const int32_t* free_head, int32_t* block_table,
                                    int32_t* starts, int32_t* lens, int64_t* slots, int32_t* rows, int32_t* counts,
                                    void* stream) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "page plan descriptor is NULL");
    if (d->requests < 0 || d->token_cap < 0 || d->free_cap < 0) return fail(DLF_ERR_INVALID_ARG, "negative size");
    if (d->page_size < 1 || d->max_pages < 1)
        return fail(DLF_ERR_INVALID_ARG, "page_size and max_pages must be positive");
    if (d->requests > 65536) return fail(DLF_ERR_UNSUPPORTED, "more than 65536 requests");
    if (static_cast<int64_t>(d->max_pages) * d->page_size >= (int64_t(1) << 31))
        return fail(DLF_ERR_UNSUPPORTED, "max_pages * page_size must stay below 2^31");
    if (!starts || !counts || (d->requests > 0 && (!cached || !fresh || !block_table || !lens)) ||
        (d->token_cap > 0 && !slots) || (d->free_cap > 0 && !free_pages))
        return fail(DLF_ERR_INVALID_ARG, "cached, fresh, free_pages, block_table, starts, lens, slots and counts must "
                                         "be non-NULL");
    if (!aligned(cached, 4) || !aligned(fresh, 4) || !aligned(free_pages, 4) || !aligned(free_head, 4) ||
        !aligned(block_table, 4) || !aligned(starts, 4) || !aligned(lens, 4) || !aligned(rows, 4) ||
        !aligned(counts, 4) || !aligned(slots, 8))
        return fail(DLF_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned, slots 8-byte");
    const size_t r = static_cast<size_t>(d->requests), t = static_cast<size_t>(d->token_cap);
    if (any_overlap({{block_table, r * static_cast<size_t>(d->max_pages) * 4}, {starts, (r + 1) * 4}, {lens, r * 4},
                     {slots, t * 8}, {rows, t * 4}, {counts, 16}},
                    {{cached, r * 4}, {fresh, r * 4}, {free_pages, static_cast<size_t>(d->free_cap) * 4},
                     {free_head, 4}}))
        return fail(DLF_ERR_ALIAS, "an output overlaps an input or another output");
    dlf::PagePlanArgs a{};
    a.cached = cached; a.fresh = fresh; a.free_pages = free_pages; a.free_head = free_head;
    a.table = block_table; a.starts = starts; a.lens = lens; a.slots = slots; a.rows = rows; a.counts = counts;
    a.requests = d->requests; a.page_size = d->page_size; a.max_pages = d->max_pages;
    a.token_cap = d->token_cap; a.free_cap = d->free_cap;
    const hipError_t e = dlf::launch_page_plan(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DLF_ERR_HIP, "dlf_page_plan: %s", hipGetErrorString(e));
    return ok();
}

extern "C" dlf_status dlf_paged_store(const dlf_kv_cache_desc* c, int64_t tokens, const void* k, int64_t k_stride,
                                      const void* v, int64_t v_stride, const int64_t* slots, void* k_cache,
                                      void* v_cache, void* stream) {
    if (!c) return fail(DLF_ERR_INVALID_ARG, "cache descriptor is NULL");
    const dlf_status st = check_cache(c);
    if (st != DLF_OK) return st;
    if (tokens < 0) return fail(DLF_ERR_INVALID_ARG, "negative token count");
    if (tokens > (int64_t(1) << 30)) return fail(DLF_ERR_UNSUPPORTED, "more than 2^30 tokens");
    if (tokens == 0) return ok();
    const int64_t width = static_cast<int64_t>(c->kv_heads) * c->head_dim;
    if (k_stride < width || v_stride < width)
        return fail(DLF_ERR_INVALID_ARG, "a row stride is below kv_heads * head_dim");
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride > kMaxStride || v_stride > kMaxStride)
        return fail(DLF_ERR_UNSUPPORTED, "row strides must be multiples of 8, at most 2^31");
    const int64_t each = dlf::paged_store_tokens(c->kv_heads, c->head_dim);
    if ((tokens + each - 1) / each >= dlf::kMaxWorkgroups)
        return fail(DLF_ERR_UNSUPPORTED, "tokens of %lld values must stay below %lld", static_cast<long long>(width),
                    static_cast<long long>(each * (dlf::kMaxWorkgroups - 1) + 1));
    if (!k || !v || !slots || !k_cache || !v_cache)
        return fail(DLF_ERR_INVALID_ARG, "k, v, slots and the caches must be non-NULL");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 8))
        return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned (slots 8)");
    const size_t cb = cache_bytes(c);
    if (any_overlap({{k_cache, cb}, {v_cache, cb}},
                    {{k, rows_bytes(tokens, k_stride, width, 2)}, {v, rows_bytes(tokens, v_stride, width, 2)},
                     {slots, static_cast<size_t>(tokens) * 8}}))
        return fail(DLF_ERR_ALIAS, "a cache overlaps an input or the other cache");
    dlf::PagedStoreArgs a{};
    a.src[0] = static_cast<const uint16_t*>(k);
    a.src[1] = static_cast<const uint16_t*>(v);
    a.cache[0] = k_cache;
    a.cache[1] = v_cache;
    a.slots = slots;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.fp8 = c->dtype == DLF_FP8_E4M3;
    a.inv_scale[0] = a.fp8 ? 1.0f / c->k_scale : 1.0f;
    a.inv_scale[1] = a.fp8 ? 1.0f / c->v_scale : 1.0f;
    a.tokens = tokens;
    a.slot_count = static_cast<int64_t>(c->pages) * c->page_size;
    a.kv_heads = c->kv_heads;
    a.head_dim = c->head_dim;
    a.page_size = c->page_size;
    const hipError_t e = dlf::launch_paged_store(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DLF_ERR_HIP, "dlf_paged_store: %s", hipGetErrorString(e));
    return ok();
}

namespace {

// the descriptor's checks; fills the kernel's sizes
dlf_status check_attn_desc(const dlf_paged_attn_desc* d, dlf::PagedAttnArgs* a) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "attention descriptor is NULL");
    const dlf_kv_cache_desc* c = &d->cache;
    const dlf_status st = check_cache(c);
    if (st != DLF_OK) return st;
    if (d->requests < 0 || d->window < 0 || d->max_len < 0)
        return fail(DLF_ERR_INVALID_ARG, "requests, window and max_len must not be negative");
    if (d->max_pages < 1) return fail(DLF_ERR_INVALID_ARG, "max_pages must be positive");
    if (d->heads < 1 || d->heads % c->kv_heads != 0)
        return fail(DLF_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
    if (!std::isfinite(d->softmax_scale)) return fail(DLF_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (static_cast<int64_t>(d->max_pages) * c->page_size >= (int64_t(1) << 31))
        return fail(DLF_ERR_UNSUPPORTED, "max_pages * page_size must stay below 2^31");
    const int group = d->heads / c->kv_heads;
    if (group > 256) return fail(DLF_ERR_UNSUPPORTED, "more than 256 query heads to a kv head");
    if (d->requests > 65536) return fail(DLF_ERR_UNSUPPORTED, "more than 65536 requests");
    if (d->q_stride < static_cast<int64_t>(d->heads) * c->head_dim)
        return fail(DLF_ERR_INVALID_ARG, "q_stride is below heads * head_dim");
    if (d->q_stride % 8 != 0 || d->q_stride > kMaxStride)
        return fail(DLF_ERR_UNSUPPORTED, "q_stride must be a multiple of 8, at most 2^31");
    *a = dlf::PagedAttnArgs{};
    a->q_stride = d->q_stride;
    a->requests = d->requests;
    a->heads = d->heads;
    a->kv_heads = c->kv_heads;
    a->page_size = c->page_size;
    a->pages = c->pages;
    a->max_pages = d->max_pages;
    a->window = d->window;
    a->group = group;
    a->head_tiles = (group + 15) / 16;
    if (static_cast<int64_t>(d->requests) * c->kv_heads * a->head_tiles >= dlf::kMaxWorkgroups)
        return fail(DLF_ERR_UNSUPPORTED, "requests * kv_heads * ceil(heads / kv_heads / 16) must stay below 2^24");
    const bool fp8 = c->dtype == DLF_FP8_E4M3;
    a->score_scale = static_cast<float>(static_cast<double>(d->softmax_scale) * (fp8 ? c->k_scale : 1.0f) *
                                        1.4426950408889634074);
    a->v_scale = fp8 ? c->v_scale : 1.0f;
    dlf::plan_paged_attention(a, c->head_dim * (fp8 ? 1 : 2), d->max_len);
    return ok();
}

// rows of the pieces' sums, where items are cut
size_t attn_part_rows(const dlf::PagedAttnArgs& a) {
    if (a.aim == 0) return 0;
    const size_t items = static_cast<size_t>(a.requests) * static_cast<size_t>(a.kv_heads * a.head_tiles);
    return (items + static_cast<size_t>(a.aim)) * static_cast<size_t>(a.group < 16 ? a.group : 16);
}

size_t attn_ws_bytes(const dlf::PagedAttnArgs& a, int head_dim) {
    if (a.aim == 0) return 0;
    return attn_part_rows(a) * (static_cast<size_t>(head_dim) + 2) * 4 + static_cast<size_t>(a.requests) * 8;
}

}  // namespace

extern "C" dlf_status dlf_paged_attention_workspace_bytes(const dlf_paged_attn_desc* d, size_t* bytes) {
    if (!bytes) return fail(DLF_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    dlf::PagedAttnArgs a;
    const dlf_status st = check_attn_desc(d, &a);
    if (st != DLF_OK) return st;
    *bytes = d->requests > 0 ? attn_ws_bytes(a, d->cache.head_dim) : 0;
    return ok();
}

extern "C" dlf_status dlf_paged_attention(const dlf_paged_attn_desc* d, const void* q, const void* k_cache,
                                          const void* v_cache, const int32_t* block_table, const int32_t* lens,
                                          void* out, float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    dlf::PagedAttnArgs a;
    const dlf_status st = check_attn_desc(d, &a);
    if (st != DLF_OK || d->requests == 0) return st;
    if (!q || !k_cache || !v_cache || !block_table || !lens || !out)
        return fail(DLF_ERR_INVALID_ARG, "q, the caches, block_table, lens and out must be non-NULL");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned (int32 and fp32 arrays 4)");
    const size_t r = static_cast<size_t>(d->requests), rows = r * static_cast<size_t>(d->heads);
    const size_t width = static_cast<size_t>(d->cache.head_dim);
    const dlf::Span qs{q, rows_bytes(d->requests, d->q_stride, static_cast<int64_t>(d->heads) * d->cache.head_dim, 2)};
    const dlf::Span ks{k_cache, cache_bytes(&d->cache)}, vs{v_cache, cache_bytes(&d->cache)};
    const dlf::Span ts{block_table, r * static_cast<size_t>(d->max_pages) * 4}, ls{lens, r * 4};
    const dlf::Span os{out, rows * width * 2}, es{lse, rows * 4};
    const size_t part_rows = attn_part_rows(a), need = attn_ws_bytes(a, d->cache.head_dim);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(DLF_ERR_INVALID_ARG, "workspace of %zu bytes needed (dlf_paged_attention_workspace_bytes), got %zu",
                        need, workspace ? workspace_bytes : size_t(0));
        if (!aligned(workspace, 16)) return fail(DLF_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    }
    if (any_overlap({os, es, {workspace, need}}, {qs, ks, vs, ts, ls}))
        return fail(DLF_ERR_ALIAS, "an output or the workspace overlaps an operand");
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = need > 0 ? a.part_o + part_rows * width : nullptr;
    a.pieces = need > 0 ? reinterpret_cast<int32_t*>(a.part_ml + part_rows * 2) : nullptr;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint8_t*>(k_cache);
    a.v = static_cast<const uint8_t*>(v_cache);
    a.table = block_table;
    a.lens = lens;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    const hipError_t e = dlf::launch_paged_attention(a, d->cache.head_dim, d->cache.dtype == DLF_FP8_E4M3,
                                                     static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DLF_ERR_HIP, "dlf_paged_attention: %s", hipGetErrorString(e));
    return ok();
}
