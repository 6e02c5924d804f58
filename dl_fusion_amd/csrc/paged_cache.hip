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
// (8 bytes a request from L2; 1024 requests are three loads a thread) and scans its own in
// registers and LDS.  The alternative, a scan kernel and a fill kernel, costs a launch more.  The
// chunk's new table entries and tokens are then flat lists, found by a binary search over the LDS
// sums, so that a long prompt among short ones spreads over every thread of its chunk's slices.
// What bounds it is the chain of dependent steps (lengths, sums, search, table or free list), not
// bytes: one request 3.9 us on the device, 1024 requests of a token each 6.0, 97 prompts of 133 000
// tokens in all 6.1 (1.6 MB of slots and rows), of which a launch is 2; the call takes 6 to 7 on the host.
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

// x of the lane that the DPP control names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t dpp64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(x), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(x >> 32), CTRL, ROWS, 0xF, false);
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Inclusive sum over the wave's lanes: shifts by 1, 2, 4 and 8 within rows of 16 lanes, then the rows'
// sums handed on.
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
    x += dpp64<0x111, 0xF>(x);
    x += dpp64<0x112, 0xF>(x);
    x += dpp64<0x114, 0xF>(x);
    x += dpp64<0x118, 0xF>(x);
    x += dpp64<0x142, 0xA>(x);
    x += dpp64<0x143, 0xC>(x);
    return x;
}

__device__ __forceinline__ int64_t last_lane(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(x), 63);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(x >> 32), 63);
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// The number of entries of the ascending list a[0..256) that are <= v, for v below the last one.
__device__ __forceinline__ int count_up_to(const int64_t* a, int64_t v) {
    int n = 0;
#pragma unroll
    for (int d = kPlanThreads / 2; d > 0; d >>= 1) n += a[n + d - 1] <= v ? d : 0;
    return n;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(const PagePlanArgs p) {
    __shared__ int64_t fresh_end[kPlanThreads], need_end[kPlanThreads];   // inclusive sums in the chunk
    __shared__ int64_t cached_s[kPlanThreads];
    __shared__ int32_t have_s[kPlanThreads];
    constexpr int kPlanWaves = kPlanThreads / 64;
    // of every wave: fresh and need of its requests before the chunk, of its part of the chunk, longest
    __shared__ int64_t sums[kPlanWaves][4];
    __shared__ int top_s[kPlanWaves];
    const int tid = static_cast<int>(threadIdx.x), wave = tid >> 6;
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
    int64_t fresh_to = wave_scan(q.fresh), need_to = wave_scan(q.need);
    f = wave_scan(f);
    g = wave_scan(g);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const int other = __shfl_xor(top, d);
        top = other > top ? other : top;
    }
    if ((tid & 63) == 63) {
        sums[wave][0] = f;
        sums[wave][1] = g;
        sums[wave][2] = fresh_to;
        sums[wave][3] = need_to;
        top_s[wave] = top;
    }
    __syncthreads();
    int64_t fresh0 = 0, need0 = 0, fresh_n = 0, need_n = 0;
    int longest = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        fresh0 += sums[w][0];
        need0 += sums[w][1];
        if (w == wave) {
            fresh_to += fresh_n;
            need_to += need_n;
        }
        fresh_n += sums[w][2];
        need_n += sums[w][3];
        longest = top_s[w] > longest ? top_s[w] : longest;
    }
    fresh_end[tid] = fresh_to;
    need_end[tid] = need_to;
    cached_s[tid] = q.cached;
    have_s[tid] = q.have;
    __syncthreads();

    if (slice == 0) {
        if (tid < n) {
            p.starts[r0 + tid] = hold_int32(fresh0 + fresh_to - q.fresh);
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
        const int i = count_up_to(need_end, e);
        const int64_t first = i > 0 ? need_end[i - 1] : 0;
        const int64_t at = head + need0 + e;
        p.table[static_cast<int64_t>(r0 + i) * p.max_pages + have_s[i] + (e - first)] =
            at < p.free_cap ? p.free_pages[at] : -1;
    }
    // tokens; the last chunk also fills the places past the last token
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int64_t end = last ? p.token_cap - fresh0 : (fresh_n < p.token_cap - fresh0 ? fresh_n : p.token_cap - fresh0);
    // four tokens a thread at a time, step by step together, since each is a chain of searches and loads
    constexpr int kTogether = 4;
    for (int64_t e0 = static_cast<int64_t>(slice) * kPlanThreads + tid; e0 < end; e0 += kTogether * step) {
        int i[kTogether];
        int64_t pos[kTogether];
        const int32_t* from[kTogether];
        int32_t page[kTogether];
        uint32_t col[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            const int64_t e = e0 + j * step;
            i[j] = count_up_to(fresh_end, e < fresh_n ? e : 0);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            const int64_t e = e0 + j * step;
            const int b = i[j] > 0 ? i[j] - 1 : 0;
            pos[j] = cached_s[i[j]] + e - (i[j] > 0 ? fresh_end[b] : 0);
            from[j] = nullptr;
            col[j] = static_cast<uint32_t>(pos[j]) / static_cast<uint32_t>(p.page_size);
            if (e < fresh_n && e < end && pos[j] < cap) {
                const int64_t more = static_cast<int64_t>(col[j]) - have_s[i[j]];
                // an entry that this launch writes is taken from the free list itself
                const int64_t at = head + need0 + (i[j] > 0 ? need_end[b] : 0) + more;
                if (more < 0) from[j] = p.table + static_cast<int64_t>(r0 + i[j]) * p.max_pages + col[j];
                else if (at < p.free_cap) from[j] = p.free_pages + at;
            }
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            page[j] = -1;
            if (from[j]) page[j] = *from[j];
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            const int64_t e = e0 + j * step;
            if (e >= end) continue;
            const uint32_t in = static_cast<uint32_t>(pos[j]) - col[j] * static_cast<uint32_t>(p.page_size);
            p.slots[fresh0 + e] = page[j] >= 0 ? static_cast<int64_t>(page[j]) * p.page_size + in : -1;
            if (p.rows) p.rows[fresh0 + e] = e < fresh_n ? r0 + i[j] : -1;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Store.  A copy: 2 or 3 bytes moved per byte of bf16 input, nothing to compute.  A thread moves 8
// values (one 16-byte load); neighbouring threads take neighbouring chunks of a head and then the
// next head of the same token, so a token's row is read in whole lines and each head's run of
// head_dim values is written whole.  Four tokens a thread are read before the first is stored, and
// before their slots are known.  16411 tokens of 8 heads of 128 to an e4m3 cache in random slots: 24 us
// for 101 MB, 4.2 TB/s (a copy of whole GB runs at 5.2); 64 tokens 3.5 us on the device.
// ---------------------------------------------------------------------------------------------
constexpr int kStoreThreads = 256;
constexpr int kStoreTogether = 4;      // tokens a thread has in flight

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
    if (t >= tokens) return;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (tokens * kStoreTogether) + t;
    int64_t slot[kStoreTogether];
#pragma unroll
    for (int j = 0; j < kStoreTogether; ++j) {
        const int64_t token = first + j * tokens;
        slot[j] = token < p.tokens ? p.slots[token] : -1;
    }
    for (int c = static_cast<int>(threadIdx.x) - t * chunks; c < chunks; c += kStoreThreads) {
        const int h = c / per_head, e = 8 * (c - h * per_head);
        u32x4_t x[kStoreTogether];
#pragma unroll
        for (int j = 0; j < kStoreTogether; ++j) {
            // a token past the last repeats the last: loaded, never stored
            const int64_t token = first + j * tokens < p.tokens ? first + j * tokens : p.tokens - 1;
            x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(src + token * stride + 8 * c));
        }
#pragma unroll
        for (int j = 0; j < kStoreTogether; ++j) {
            if (slot[j] < 0 || slot[j] >= p.slot_count) continue;
            const uint32_t page = static_cast<uint32_t>(slot[j]) / static_cast<uint32_t>(p.page_size);
            const uint32_t off = static_cast<uint32_t>(slot[j]) - page * static_cast<uint32_t>(p.page_size);
            const int64_t at = ((static_cast<int64_t>(page) * p.kv_heads + h) * p.page_size + off) * p.head_dim + e;
            if constexpr (FP8) *reinterpret_cast<uint2*>(cache + at) = quant8(x[j], inv);
            else *reinterpret_cast<u32x4_t*>(cache + 2 * at) = x[j];
        }
    }
}

}  // namespace

hipError_t launch_page_plan(const PagePlanArgs& a, hipStream_t s) {
    const int chunks = a.requests > kPlanThreads ? (a.requests + kPlanThreads - 1) / kPlanThreads : 1;
    // slices: four tokens a thread, at most 256 workgroups a chunk
    int64_t slices = (static_cast<int64_t>(a.token_cap) / chunks + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    slices = slices < 1 ? 1 : slices > 256 ? 256 : slices;
    page_plan_kernel<<<dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(slices)), kPlanThreads, 0, s>>>(a);
    return hipGetLastError();
}

int paged_store_tokens(int kv_heads, int head_dim) {
    const int chunks = kv_heads * (head_dim / 8);
    return kStoreTogether * (chunks < kStoreThreads ? kStoreThreads / chunks : 1);
}

hipError_t launch_paged_store(const PagedStoreArgs& a, hipStream_t s) {
    const int each = paged_store_tokens(a.kv_heads, a.head_dim);
    const dim3 grid(static_cast<unsigned>((a.tokens + each - 1) / each), 2);
    if (a.fp8) paged_store_kernel<true><<<grid, kStoreThreads, 0, s>>>(a);
    else paged_store_kernel<false><<<grid, kStoreThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dlf
