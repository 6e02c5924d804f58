// The bookkeeping and the filling of a paged key-value cache: block tables and slot maps from
// request lengths, and the store of new keys and values into their slots.
#include "device_common.h"
#include "kernels.h"

namespace dlf {
namespace {

// ---------------------------------------------------------------------------------------------
// Page plan.  With c = min(cached, cap), n = min(cached + fresh, cap), a request needs
// ceil(n / page) - ceil(c / page) new pages; its first one's place in the free list and its first
// token's number are exclusive sums over the requests before it.
//
// One launch: workgroup (chunk, slice) owns 256 requests, sums those before its chunk again
// (8 bytes a request from L2; 1024 requests are three loads a thread) and scans its own in LDS.
// The alternative, a scan kernel and a fill kernel, costs a launch more.  The chunk's new table
// entries and tokens are then flat lists, found by a binary search over the LDS sums, so that a
// long prompt among short ones spreads over every thread of its chunk's slices.
// ---------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 256;

struct PlanRequest {
    int64_t cached, fresh, len;  // clipped as the entry point defines
    int32_t have, need;          // pages held, pages to take
};

__device__ __forceinline__ PlanRequest plan_request(const PagePlanArgs& p, int r) {
    PlanRequest q{};
    const uint32_t ps = static_cast<uint32_t>(p.page_size);
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;    // < 2^31
    const int64_t c = p.cached[r], f = p.fresh[r];
    q.cached = c > 0 ? c : 0;
    q.fresh = f > 0 ? f : 0;
    q.len = q.cached + q.fresh < cap ? q.cached + q.fresh : cap;
    const int64_t held = q.cached < cap ? q.cached : cap;
    q.have = static_cast<int32_t>((static_cast<uint32_t>(held) + ps - 1) / ps);
    q.need = static_cast<int32_t>((static_cast<uint32_t>(q.len) + ps - 1) / ps) - q.have;
    return q;
}

__device__ __forceinline__ int32_t hold_int32(int64_t v) {
    return v < INT32_MAX ? static_cast<int32_t>(v) : INT32_MAX;
}

// Inclusive sum over the workgroup's threads, in place in LDS.
__device__ __forceinline__ void block_scan(int64_t* a, int64_t* b, int tid) {
    for (int d = 1; d < kPlanThreads; d <<= 1) {
        __syncthreads();
        const int64_t x = tid >= d ? a[tid - d] : 0, y = tid >= d ? b[tid - d] : 0;
        __syncthreads();
        a[tid] += x;
        b[tid] += y;
    }
    __syncthreads();
}

// The number of entries of the ascending list a[0..n) that are <= v (n <= 256).
__device__ __forceinline__ int count_up_to(const int64_t* a, int n, int64_t v) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(const PagePlanArgs p) {
    __shared__ int64_t fresh_end[kPlanThreads], need_end[kPlanThreads];   // inclusive sums in the chunk
    __shared__ int64_t base[2];                                           // fresh and need before the chunk
    __shared__ int64_t cached_s[kPlanThreads];
    __shared__ int32_t have_s[kPlanThreads];
    __shared__ int longest;
    const int tid = static_cast<int>(threadIdx.x);
    const int r0 = static_cast<int>(blockIdx.x) * kPlanThreads;
    const int slice = static_cast<int>(blockIdx.y), slices = static_cast<int>(gridDim.y);
    const bool last = blockIdx.x + 1 == gridDim.x;
    const int n = p.requests - r0 < kPlanThreads ? p.requests - r0 : kPlanThreads;
    int64_t head = p.free_head ? *p.free_head : 0;
    head = head > 0 ? head : 0;

    // this chunk's own request, and the sums over the requests before the chunk
    PlanRequest q{};
    if (tid < n) q = plan_request(p, r0 + tid);
    int64_t f = 0, g = 0;
    int top = static_cast<int>(q.len);
    for (int r = tid; r < r0; r += kPlanThreads) {
        const PlanRequest o = plan_request(p, r);
        f += o.fresh;
        g += o.need;
        top = o.len > top ? static_cast<int>(o.len) : top;
    }
    if (tid == 0) longest = 0;
    fresh_end[tid] = f;
    need_end[tid] = g;
    block_scan(fresh_end, need_end, tid);
    if (tid == 0) {
        base[0] = fresh_end[kPlanThreads - 1];
        base[1] = need_end[kPlanThreads - 1];
    }
    atomicMax(&longest, top);       // LDS; a maximum does not depend on the order
    __syncthreads();
    fresh_end[tid] = q.fresh;
    need_end[tid] = q.need;
    cached_s[tid] = q.cached;
    have_s[tid] = q.have;
    block_scan(fresh_end, need_end, tid);
    const int64_t fresh0 = base[0], need0 = base[1];
    const int64_t fresh_n = fresh_end[kPlanThreads - 1], need_n = need_end[kPlanThreads - 1];

    if (slice == 0) {
        if (tid < n) {
            p.starts[r0 + tid] = hold_int32(fresh0 + fresh_end[tid] - q.fresh);
            p.lens[r0 + tid] = static_cast<int32_t>(q.len);
        }
        if (last && tid == 0) {
            const int64_t want = head + need0 + need_n;
            p.starts[p.requests] = hold_int32(fresh0 + fresh_n);
            p.counts[0] = hold_int32(fresh0 + fresh_n);
            p.counts[1] = static_cast<int32_t>(want < p.free_cap ? want : p.free_cap);
            p.counts[2] = longest;
            const int64_t have = head > p.free_cap ? head : p.free_cap;
            p.counts[3] = hold_int32(want > have ? want - have : 0);
        }
    }

    const int64_t step = static_cast<int64_t>(slices) * kPlanThreads;
    // new table entries
    for (int64_t e = static_cast<int64_t>(slice) * kPlanThreads + tid; e < need_n; e += step) {
        const int i = count_up_to(need_end, n, e);
        const int64_t first = i > 0 ? need_end[i - 1] : 0;
        const int64_t at = head + need0 + e;
        p.table[static_cast<int64_t>(r0 + i) * p.max_pages + have_s[i] + (e - first)] =
            at < p.free_cap ? p.free_pages[at] : -1;
    }
    // tokens; the last chunk also fills the places past the last token
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int64_t end = last ? p.token_cap - fresh0 : (fresh_n < p.token_cap - fresh0 ? fresh_n : p.token_cap - fresh0);
    for (int64_t e = static_cast<int64_t>(slice) * kPlanThreads + tid; e < end; e += step) {
        int64_t slot = -1;
        int32_t row = -1;
        if (e < fresh_n) {
            const int i = count_up_to(fresh_end, n, e);
            const int64_t first = i > 0 ? fresh_end[i - 1] : 0;
            const int64_t pos = cached_s[i] + (e - first);
            row = r0 + i;
            if (pos < cap) {
                const uint32_t col = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page_size);
                int32_t page = -1;
                if (static_cast<int32_t>(col) < have_s[i]) {
                    page = p.table[static_cast<int64_t>(row) * p.max_pages + col];
                } else {
                    // an entry that this launch writes: taken from the free list itself
                    const int64_t at = head + need0 + (i > 0 ? need_end[i - 1] : 0) + (static_cast<int32_t>(col) - have_s[i]);
                    if (at < p.free_cap) page = p.free_pages[at];
                }
                if (page >= 0)
                    slot = static_cast<int64_t>(page) * p.page_size + (static_cast<uint32_t>(pos) % static_cast<uint32_t>(p.page_size));
            }
        }
        p.slots[fresh0 + e] = slot;
        if (p.rows) p.rows[fresh0 + e] = row;
    }
}

// ---------------------------------------------------------------------------------------------
// Store.  A copy: 2 or 3 bytes moved per byte of bf16 input, nothing to compute.  A thread moves 8
// values (one 16-byte load); neighbouring threads take neighbouring chunks of a head and then the
// next head of the same token, so a token's row is read in whole lines and each head's run of
// head_dim values is written whole.
// ---------------------------------------------------------------------------------------------
constexpr int kStoreThreads = 256;

// Eight codes of fp32(v * inv); the clamp keeps NaN (both comparisons are false), which the
// conversion then encodes as the e4m3 NaN.
__device__ __forceinline__ float clamp_e4m3(float v) {
    v = v > 448.0f ? 448.0f : v;
    return v < -448.0f ? -448.0f : v;
}

__device__ __forceinline__ uint2 quant8(const u32x4_t x, float inv) {
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v[2 * e] = clamp_e4m3(__fmul_rn(__uint_as_float(x[2 * i + e] << 16), inv));
            v[2 * e + 1] = clamp_e4m3(__fmul_rn(__uint_as_float(x[2 * i + e] & 0xFFFF0000u), inv));
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
        out[i] = static_cast<uint32_t>(w);
    }
    return make_uint2(out[0], out[1]);
}

template <bool FP8>
__global__ __launch_bounds__(kStoreThreads) void paged_store_kernel(const PagedStoreArgs p) {
    const int which = static_cast<int>(blockIdx.y);     // 0 keys, 1 values
    const uint16_t* const src = p.src[which];
    uint8_t* const cache = static_cast<uint8_t*>(p.cache[which]);
    const int64_t stride = p.stride[which];
    const float inv = p.inv_scale[which];
    const int per_head = p.head_dim / 8;
    const int chunks = p.kv_heads * per_head;           // 16-byte chunks of a token's row
    const int tokens = chunks < kStoreThreads ? kStoreThreads / chunks : 1;   // tokens a workgroup
    const int t = static_cast<int>(threadIdx.x) / chunks;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * tokens + t;
    if (t >= tokens || token >= p.tokens) return;
    const int64_t slot = p.slots[token];
    if (slot < 0 || slot >= p.slot_count) return;
    const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
    const uint32_t off = static_cast<uint32_t>(slot) - page * static_cast<uint32_t>(p.page_size);
    for (int c = static_cast<int>(threadIdx.x) - t * chunks; c < chunks; c += kStoreThreads) {
        const int h = c / per_head, e = 8 * (c - h * per_head);
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(src + token * stride + 8 * c);
        const int64_t at = ((static_cast<int64_t>(page) * p.kv_heads + h) * p.page_size + off) * p.head_dim + e;
        if constexpr (FP8) *reinterpret_cast<uint2*>(cache + at) = quant8(x, inv);
        else *reinterpret_cast<u32x4_t*>(cache + 2 * at) = x;
    }
}

}  // namespace

hipError_t launch_page_plan(const PagePlanArgs& a, hipStream_t s) {
    const int chunks = a.requests > kPlanThreads ? (a.requests + kPlanThreads - 1) / kPlanThreads : 1;
    // slices: eight tokens a thread, at most 256 workgroups a chunk
    int64_t slices = (static_cast<int64_t>(a.token_cap) / chunks + 8 * kPlanThreads - 1) / (8 * kPlanThreads);
    slices = slices < 1 ? 1 : slices > 256 ? 256 : slices;
    page_plan_kernel<<<dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(slices)), kPlanThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_paged_store(const PagedStoreArgs& a, hipStream_t s) {
    const int chunks = a.kv_heads * (a.head_dim / 8);
    const int tokens = chunks < kStoreThreads ? kStoreThreads / chunks : 1;
    const dim3 grid(static_cast<unsigned>((a.tokens + tokens - 1) / tokens), 2);
    if (a.fp8) paged_store_kernel<true><<<grid, kStoreThreads, 0, s>>>(a);
    else paged_store_kernel<false><<<grid, kStoreThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dlf
