// Attention of one new token per request over a paged key-value cache.
//
// For a request, a kv head and the up to 16 query heads q of its group that share a tile:
//     s_j = scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j)
// in one pass over the tokens j, with the running maximum m and sum l of the softmax: a tile's new
// maximum m' rescales what is summed so far by exp(m - m').
//
// What bounds it is the read of the cache: 4 flops a value at bf16 and one query head, 64 at 16 of
// them, against the hundreds a byte that the matrix cores could do.  So the products need no tuning
// beyond keeping out of the way, and the layout is chosen so that little stands between a load and
// the MFMA that uses it: the keys pass through LDS, the values only through a byte permute.  64 uneven requests of up to 8191 tokens read
// 698 MB in 118 us, 5.9 TB/s; two of 32768 and 131072 tokens 671 MB in 113 us, 5.9 TB/s (8 kv heads of
// 128 dims); a loop of nothing but such loads reads 6.8 TB/s in random pages.
//  - scores are computed transposed, S^T = K Q^T (16 tokens x 16 queries an MFMA): a lane's key
//    operand is 16 contiguous bytes of one token's row;
//  - the 16x16 result leaves each lane with one query's scores of 4 tokens, which is just the
//    operand that the second product, O^T = V^T P^T, wants from that lane, if its 32 tokens are
//    numbered 4 (lane / 16) + 16 half + 0..3: the probabilities never move;
//  - a lane loads the value rows of those 8 tokens, 1/16 of a row each, and a byte permute of pairs of
//    tokens gives the 8 tokens of each of its dims: the order of the dims among the lanes is free, since
//    the result's rows come out in the same order.
// 16 query rows are computed whatever the group: the rest is zeros and costs nothing that bounds.  A group of
// more than 16 heads is several tiles, and each reads the cache: 64 requests of 8192 tokens on one kv head
// take 56, 99, 189 and 363 us with 16, 32, 64 and 128 query heads.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "mma_common.h"

namespace dlf {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kJoinThreads = 256;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;

// What is read of a request: tokens [lo, len), in tiles of 32 from t16 on, lo rounded down to a
// multiple of 16 so that 16 tokens share a page.
struct Reach {
    int len, lo, t16;
    uint32_t tiles;     // 0 where there is no token
};

__device__ __forceinline__ Reach reach_of(const PagedAttnArgs& p, int r) {
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;   // < 2^31
    int len = p.lens[r];
    len = len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
    const int lo = p.window > 0 && len > p.window ? len - p.window : 0;
    const int t16 = lo & ~15;
    return {len, lo, t16, (static_cast<uint32_t>(len - t16) + 31) / 32};
}

// Tiles that a request counts for in the split of the work: at least one, which writes its zeros.
__device__ __forceinline__ uint32_t share_of(const Reach& k) { return k.tiles > 0 ? k.tiles : 1; }

// The cache bytes of 32 tokens of one head, as a wave holds them: the keys in LDS, the values in
// registers.
//
// A lane's key operand is 16 bytes of one token's row, and the 16 lanes next to each other have 16
// tokens: loaded straight to registers that is 64 accesses of the cache to a load, and 58 GB/s a CU
// was all it gave.  So keys go to LDS by loads of whole lines, no register between, and come back with
// one 16-byte read a lane.  A row's 16-byte chunk c lies at place c ^ swizzle(row), so that the 16
// lanes' reads fall on all banks: the lanes of the load take their chunks in that order.
template <int D, bool FP8>
struct KvTile {
    static constexpr int kRow = D * (FP8 ? 1 : 2);      // bytes of a token's row
    static constexpr int kBytes = 32 * kRow;            // the keys of a tile
    static constexpr int kChunks = kRow / 16;
    static constexpr int kKeyReads = kRow / 64;         // 16-byte reads a lane and 16 tokens
    static constexpr int kKeyLoads = kRow / 64;         // 1 KB loads to LDS for 16 tokens
    static constexpr int kValWords = kRow / 64;         // 32-bit words of a lane's 1/16 of a row
    typedef uint32_t value_t __attribute__((ext_vector_type(kValWords < 4 ? kValWords : 4)));
    static constexpr int kValLoads = (kValWords + 3) / 4;
    value_t v[8][kValLoads];
    __device__ __forceinline__ uint32_t word(int token, int c) const { return v[token][c / 4][c & 3]; }
    static __device__ __forceinline__ int swizzle(int row) {
        return kChunks >= 16 ? row & 15 : (row / (16 / kChunks)) & (kChunks - 1);
    }
};

// Two bf16 values a word from two e4m3 codes (exact).
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8x2_to_bf16x2(uint32_t codes) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HIGH));
}

// Inclusive sum over the wave's lanes: shifts by 1, 2, 4 and 8 within rows of 16 lanes, then the
// rows' sums handed on; lanes without a source add 0.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    x += __builtin_amdgcn_update_dpp(0u, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0u, x, 0x143, 0xC, 0xF, false);
    return x;
}

// Where parts are joined to NaN, the factor of a part's sum o once more.  A part whose maximum is so far below the
// others' that f is 0 adds nothing, unless its sum is infinite: no probability is 0, so that the infinity stays.
__device__ __forceinline__ float weight_of(float f, float o) { return f == 0.0f && __builtin_isinf(o) ? 1.0f : f; }

// What a workgroup takes: tiles [tile, end) of request r, for one kv head and tile of its query heads.
struct Work {
    int r, head;
    uint32_t tile, end;
    int block, pieces;      // its number among the pieces of all requests, and those of its request
};

// Lengths are only known here, so the pieces are cut here: with `all` tiles in all items, an item is
// cut into pieces of at most max(all / aim, least) tiles, equal ones within a request.  There are at
// most aim + items of them, whatever the lengths.  Each wave adds the lengths up by itself: one load
// and two scans of 64 lanes for up to 64 requests.
__device__ __forceinline__ bool find_work(const PagedAttnArgs& p, int heads, int lane, Work* w) {
    const int per = (p.requests + 63) / 64;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int r = lane * per + i;
        if (r < p.requests) mine += share_of(reach_of(p, r));
    }
    const uint32_t all = __builtin_amdgcn_readlane(wave_scan(mine), 63);      // < 2^31
    const uint64_t even = (static_cast<uint64_t>(all) * static_cast<uint32_t>(heads) + static_cast<uint32_t>(p.aim) - 1) /
                          static_cast<uint32_t>(p.aim);
    uint32_t most = even < all ? static_cast<uint32_t>(even) : all;
    most = most > static_cast<uint32_t>(p.least) ? most : static_cast<uint32_t>(p.least);
    uint32_t cuts = 0;
    for (int i = 0; i < per; ++i) {
        const int r = lane * per + i;
        if (r < p.requests) cuts += (share_of(reach_of(p, r)) + most - 1) / most;
    }
    const uint32_t upto = wave_scan(cuts);
    const uint32_t at = blockIdx.x / static_cast<uint32_t>(heads);
    const int first = __popcll(__ballot(upto <= at));
    if (first == 64) return false;      // past the last piece
    uint32_t before = __builtin_amdgcn_readlane(upto, first) - __builtin_amdgcn_readlane(cuts, first);
    int r = first * per;
    uint32_t share = share_of(reach_of(p, r)), n = (share + most - 1) / most;
    while (before + n <= at) {
        before += n;
        share = share_of(reach_of(p, ++r));
        n = (share + most - 1) / most;
    }
    const uint32_t size = (share + n - 1) / n;      // size <= most, so that (n - 1) size < share
    w->r = r;
    w->head = static_cast<int>(blockIdx.x - at * static_cast<uint32_t>(heads));
    w->tile = (at - before) * size;
    w->end = w->tile + size < share ? w->tile + size : share;
    w->block = static_cast<int>(before);
    w->pieces = static_cast<int>(n);
    return true;
}

// CUT: items are cut into pieces, and those of more than one left to the join; else a workgroup
// takes an item.
template <int D, bool FP8, bool CUT>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : D == 128 ? 3 : 4) void paged_attention_kernel(const PagedAttnArgs p) {
    using Tile = KvTile<D, FP8>;
    constexpr int kRow = Tile::kRow;
    constexpr int kSteps = D / 32;          // MFMA steps over the head's dims
    constexpr int kFrag = D / 16;           // dims a lane's value chunk holds = output fragments
    constexpr int kPad = D + 4;             // floats of an LDS row: 16 rows in different banks
    // the waves' keys, and after them the waves' sums [kWaves][rows][kPad]
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    float* const o_s = reinterpret_cast<float*>(lds);
    __shared__ float m_s[kWaves][16], l_s[kWaves][16];

    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int qi = lane & 15, g = lane >> 4;
    const int heads = p.kv_heads * p.head_tiles, rows = p.group < 16 ? p.group : 16;
    const uint32_t per_page = static_cast<uint32_t>(p.page_size) / 16;
    // key loads: where lane's 16 bytes of the n-th KB of 16 tokens come from; key reads: where the chunks
    // 4 s + g of token qi lie
    uint32_t key_from[Tile::kKeyLoads], key_at[Tile::kKeyReads];
#pragma unroll
    for (int n = 0; n < Tile::kKeyLoads; ++n) {
        const int row = (1024 * n + 16 * lane) / kRow, place = lane & (Tile::kChunks < 64 ? Tile::kChunks - 1 : 63);
        key_from[n] = static_cast<uint32_t>(row * kRow + 16 * (place ^ Tile::swizzle(row)));
    }
#pragma unroll
    for (int s = 0; s < Tile::kKeyReads; ++s)
        key_at[s] = static_cast<uint32_t>(qi * kRow + 16 * ((4 * s + g) ^ Tile::swizzle(qi)));
    uint8_t* const keys = lds + wave * Tile::kBytes;
    const uint32_t value_lane = static_cast<uint32_t>(4 * g * kRow + qi * (kRow / 16));

    Work work;
    if constexpr (CUT) {
        if (!find_work(p, heads, lane, &work)) return;
    } else {
        work.r = static_cast<int>(blockIdx.x) / heads;
        work.head = static_cast<int>(blockIdx.x) - work.r * heads;
    }
    const int r = work.r, kvh = work.head / p.head_tiles, ht = work.head - kvh * p.head_tiles;
    const int head0 = kvh * p.group + 16 * ht;                          // first query head of the tile
    const int nq = p.group - 16 * ht < 16 ? p.group - 16 * ht : 16;     // query heads in it
    const Reach reach = reach_of(p, r);
    const int len = reach.len, lo = reach.lo, t16 = reach.t16;
    // this wave's tiles: first, first + kWaves, ..
    const uint32_t first = (CUT ? work.tile : 0u) + static_cast<uint32_t>(wave);
    const uint32_t end = CUT && work.end < reach.tiles ? work.end : reach.tiles;
    const uint32_t tiles = first < end ? (end - first + kWaves - 1) / kWaves : 0;

    // byte offsets of the cache runs of the next 64 half tiles (16 tokens), one a lane; -1: no page
    int64_t run = -1;
    auto find_runs = [&](uint32_t i) {
        const uint32_t at = 32 * (first + kWaves * (i + static_cast<uint32_t>(lane) / 2)) + 16u * (lane & 1);
        const uint32_t h16 = (static_cast<uint32_t>(t16) + at) / 16, col = h16 / per_page;
        run = -1;
        if (at < static_cast<uint32_t>(len - t16)) {
            const int32_t page = p.table[static_cast<int64_t>(r) * p.max_pages + col];
            if (page >= 0 && page < p.pages)
                run = ((static_cast<int64_t>(page) * p.kv_heads + kvh) * p.page_size + 16 * (h16 - col * per_page)) * kRow;
        }
    };
    if (tiles > 0) find_runs(0);

    // query fragments: query qi, the dims that the key loads bring this lane
    bf16x8_t qf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        // bf16 keys: dims 32 s + 8 g ..; e4m3 keys: 16 a load, the steps 2 i and 2 i + 1 of load i
        const int dim = FP8 ? 64 * (s / 2) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
        u32x4_t v{0u, 0u, 0u, 0u};
        if (qi < nq)
            v = *reinterpret_cast<const u32x4_t*>(p.q + r * p.q_stride + static_cast<int64_t>(head0 + qi) * D + dim);
        qf[s] = __builtin_bit_cast(bf16x8_t, v);
    }

    f32x4_t o[kFrag];
#pragma unroll
    for (int i = 0; i < kFrag; ++i) o[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;      // l: this lane's share of the sum

    // where the two halves of tile i lie; a half without a page is read from the pool's start and masked
    struct Where {
        int64_t off[2];
        bool there[2];
    };
    auto locate = [&](uint32_t i) {
        Where w;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int lo32 = __builtin_amdgcn_readlane(static_cast<int>(run), static_cast<int>(2 * (i & 31)) + hh);
            const int hi32 = __builtin_amdgcn_readlane(static_cast<int>(run >> 32), static_cast<int>(2 * (i & 31)) + hh);
            w.there[hh] = hi32 >= 0;
            w.off[hh] = w.there[hh] ? (static_cast<int64_t>(hi32) << 32) | static_cast<uint32_t>(lo32) : 0;
        }
        return w;
    };
    auto fetch_keys = [&](const Where& w) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const __amdgpu_buffer_rsrc_t rsrc = buffer_rsrc(p.k + w.off[hh], 16 * kRow);
#pragma unroll
            for (int n = 0; n < Tile::kKeyLoads; ++n)
                load_lds16_stream(rsrc, key_from[n], keys + (16 * hh * kRow + 1024 * n));
        }
    };
    auto fetch_values = [&](const Where& w, Tile& t) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* const vp = p.v + w.off[hh] + value_lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a load's lanes cover whole lines: non-temporal ones read 6.8 TB/s against 6.0
#pragma unroll
                for (int c = 0; c < Tile::kValLoads; ++c)
                    t.v[4 * hh + j][c] = __builtin_nontemporal_load(reinterpret_cast<const typename Tile::value_t*>(vp + j * kRow + 16 * c));
            }
        }
    };
    auto scores = [&](f32x4_t (&sc)[2]) {
        u32x4_t kw[Tile::kKeyReads][2];
#pragma unroll
        for (int s = 0; s < Tile::kKeyReads; ++s)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) kw[s][hh] = *reinterpret_cast<const u32x4_t*>(keys + 16 * hh * kRow + key_at[s]);
        // all reads on their way before the first is waited for, where there are registers for it
        if constexpr (Tile::kKeyReads <= 4) __builtin_amdgcn_sched_barrier(0);
        sc[0] = sc[1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                u32x4_t k;
                if constexpr (FP8) {
                    const uint32_t c0 = kw[s / 2][hh][2 * (s & 1)], c1 = kw[s / 2][hh][2 * (s & 1) + 1];
                    k = u32x4_t{fp8x2_to_bf16x2<false>(c0), fp8x2_to_bf16x2<true>(c0), fp8x2_to_bf16x2<false>(c1),
                                fp8x2_to_bf16x2<true>(c1)};
                } else {
                    k = kw[s][hh];
                }
                sc[hh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k), qf[s], sc[hh], 0, 0, 0);
            }
    };
    // EXTENDED: values that are not finite kept apart, as explained at the second pass below
    auto add_values = [&](auto extended_c, const Where& w, uint32_t at, Tile& t, const f32x4_t (&sc)[2]) {
        constexpr bool EXTENDED = decltype(extended_c)::value;
        // lane: query qi, tokens tok0 + 16 hh + 4 g + e
        const int tok0 = t16 + static_cast<int>(at);
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = sc[i / 4][i & 3] * p.score_scale;
        if (tok0 < lo || tok0 > len - 32 || !w.there[0] || !w.there[1]) {
            // masked tokens: the score is replaced, whatever it was, and the value row is cleared, since
            // 0 x NaN or 0 x inf of a stale slot would reach the sum
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t tok = static_cast<uint32_t>(tok0 + 4 * g) + 16 * (i / 4) + (i & 3);
                const bool seen = tok >= static_cast<uint32_t>(lo) && tok < static_cast<uint32_t>(len) && w.there[i / 4];
                z[i] = seen ? z[i] : -INFINITY;
#pragma unroll
                for (int c = 0; c < Tile::kValLoads; ++c) t.v[i][c] = seen ? t.v[i][c] : typename Tile::value_t(0u);
            }
        }
        float top = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top);
        const float base = mn == -INFINITY ? 0.0f : mn;     // nothing seen yet: every exp2 below is 0
        const float alpha = __builtin_amdgcn_exp2f(m - base);
        m = mn;
        // p = hi + lo in bf16: the 2^-8 of one rounding would reach the output as much as its own rounding
        float pr[8], lo_p[8], sum = 0.0f;
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            pr[i] = __builtin_amdgcn_exp2f(z[i] - base);
            sum += pr[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ph[i] = pack_bf16x2(pr[2 * i], pr[2 * i + 1]);
            lo_p[2 * i] = pr[2 * i] - __uint_as_float(ph[i] << 16);
            lo_p[2 * i + 1] = pr[2 * i + 1] - __uint_as_float(ph[i] & 0xFFFF0000u);
            pl[i] = pack_bf16x2(lo_p[2 * i], lo_p[2 * i + 1]);
        }
        l = l * alpha + sum;
        const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, u32x4_t{ph[0], ph[1], ph[2], ph[3]});
        const bf16x8_t pg = __builtin_bit_cast(bf16x8_t, u32x4_t{pl[0], pl[1], pl[2], pl[3]});
        // EXTENDED: 1 for every token that counts, however little; NaN and the 0 of a score of -inf stay
        uint32_t pc[4] = {};
        if constexpr (EXTENDED) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pc[i] = pack_bf16x2(z[2 * i] > -INFINITY ? 1.0f : pr[2 * i], z[2 * i + 1] > -INFINITY ? 1.0f : pr[2 * i + 1]);
        }
        auto add = [&](int i, u32x4_t vt) {
            if constexpr (EXTENDED) {
                u32x4_t apart;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t bad = not_finite_bf16x2(vt[e]);
                    apart[e] = vt[e] & bad;
                    vt[e] &= ~bad;
                    o[i][e] *= __builtin_isinf(o[i][e]) ? 1.0f : alpha;
                }
                const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vt);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf, o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pg, o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, apart),
                                                               __builtin_bit_cast(bf16x8_t, u32x4_t{pc[0], pc[1], pc[2], pc[3]}), o[i], 0, 0, 0);
                return;
            }
            const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vt);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf, o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pg, o[i], 0, 0, 0);
        };
        // dims of the lane's chunk, from one word of each of the 8 tokens: bytes of pairs of tokens are
        // brought together, an e4m3 pair of two dims at a time before the conversion
#pragma unroll
        for (int c = 0; c < Tile::kValWords; ++c) {
            if constexpr (FP8) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    u32x4_t even, odd;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = __builtin_amdgcn_perm(t.word(2 * i + 1, c), t.word(2 * i, c), half ? 0x07030602u : 0x05010400u);
                        even[i] = fp8x2_to_bf16x2<false>(y);
                        odd[i] = fp8x2_to_bf16x2<true>(y);
                    }
                    add(4 * c + 2 * half, even);
                    add(4 * c + 2 * half + 1, odd);
                }
            } else {
                u32x4_t even, odd;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    even[i] = __builtin_amdgcn_perm(t.word(2 * i + 1, c), t.word(2 * i, c), 0x05040100u);
                    odd[i] = __builtin_amdgcn_perm(t.word(2 * i + 1, c), t.word(2 * i, c), 0x07060302u);
                }
                add(2 * c, even);
                add(2 * c + 1, odd);
            }
        }
    };

    // A tile's LDS and registers are refilled as they fall free, the keys after its scores, the values
    // after the sums: something is always in flight.  The last tile is peeled so that every fetch in the
    // loop is unconditional, which keeps the waits exact: the keys have landed once at most the values'
    // loads, which were issued after them, are outstanding.
    constexpr int kValueLoads = 8 * Tile::kValLoads;
    if (tiles > 0) {
        Tile t;
        f32x4_t sc[2];
        Where w = locate(0);
        fetch_keys(w);
        __builtin_amdgcn_sched_barrier(0);
        fetch_values(w, t);
        __builtin_amdgcn_sched_barrier(0);
        uint32_t at = 32 * first;
        for (uint32_t i = 1; i < tiles; ++i) {
            if ((i & 31) == 0) find_runs(i);
            const Where next = locate(i);
            __builtin_amdgcn_sched_barrier(0);
            wait_vmcnt<kValueLoads>();
            scores(sc);
            __builtin_amdgcn_sched_barrier(0);      // the tile's reads are done
            fetch_keys(next);
            __builtin_amdgcn_sched_barrier(0);
            add_values(std::false_type{}, w, at, t, sc);
            __builtin_amdgcn_sched_barrier(0);
            fetch_values(next, t);
            __builtin_amdgcn_sched_barrier(0);
            w = next;
            at += 32 * kWaves;
        }
        wait_vmcnt<kValueLoads>();
        scores(sc);
        add_values(std::false_type{}, w, at, t, sc);
    }
    // A value of infinity has become NaN wherever hi or lo of its probability is 0, lo is below it, or a later
    // rescaling is by 0; every such mistake is a NaN.  So a wave that has one goes over its tiles once more, in no
    // hurry, with two products of the finite values and a third of the others by 1: an infinity in the sum, NaN where
    // both signs meet or a value is NaN.  e4m3 has no infinities.  The look for NaN takes 0.1 to 0.2 us of a call.
    if constexpr (!FP8) {
        f32x4_t any{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kFrag; ++i) any += o[i];
        if (__builtin_expect(__ballot(__builtin_isnan(any[0] + any[1] + any[2] + any[3]) && qi < nq) != 0, 0)) {
#pragma unroll
            for (int i = 0; i < kFrag; ++i) o[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            m = -INFINITY;
            l = 0.0f;
            for (uint32_t i = 0; i < tiles; ++i) {
                if ((i & 31) == 0) find_runs(i);
                const Where w = locate(i);
                Tile t;
                f32x4_t sc[2];
                fetch_keys(w);
                fetch_values(w, t);
                wait_vmcnt<0>();
                __builtin_amdgcn_sched_barrier(0);
                scores(sc);
                __builtin_amdgcn_sched_barrier(0);      // the tile's reads are done
                add_values(std::true_type{}, w, 32 * (first + kWaves * i), t, sc);
            }
        }
    }

    // ---- the waves' results joined through LDS ----
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();        // no wave reads keys any more
    if (qi < nq) {
        if (g == 0) {
            m_s[wave][qi] = m;
            l_s[wave][qi] = l;
        }
        // fragment i, element e: dim kFrag (4 g + e) + i of query qi
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < kFrag; ++i) o_s[(wave * rows + qi) * kPad + kFrag * (4 * g + e) + i] = o[i][e];
    }
    __syncthreads();
    if (CUT && threadIdx.x == 0 && work.head == 0 && work.tile == 0)
        *reinterpret_cast<int2*>(p.pieces + 2 * r) = make_int2(work.block, work.pieces);      // for the join
    for (int i = static_cast<int>(threadIdx.x); i < nq * D / 2; i += 64 * kWaves) {
        const int row = i / (D / 2), dim = 2 * (i % (D / 2));
        float top = m_s[0][row];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_s[w][row]);
        const float base = top == -INFINITY ? 0.0f : top;
        float x = 0.0f, y = 0.0f, sum = 0.0f;
        const float* const from = o_s + row * kPad + dim;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(m_s[w][row] - base);
            x += f * from[w * rows * kPad];
            y += f * from[w * rows * kPad + 1];
            sum += f * l_s[w][row];
        }
        if (__builtin_expect(__builtin_isunordered(x, y), 0)) {
            x = y = 0.0f;
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(m_s[w][row] - base), a = from[w * rows * kPad], b = from[w * rows * kPad + 1];
                x += weight_of(f, a) * a;
                y += weight_of(f, b) * b;
            }
        }
        if (CUT && work.pieces > 1) {
            const int64_t at = static_cast<int64_t>(blockIdx.x) * rows + row;
            *reinterpret_cast<f32x2_t*>(p.part_o + at * D + dim) = f32x2_t{x, y};
            if (dim == 0) *reinterpret_cast<f32x2_t*>(p.part_ml + 2 * at) = f32x2_t{top, sum};
            continue;
        }
        // no token left: zeros.  A sum of NaN is not 0 and goes through.
        const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
        const int64_t row_at = static_cast<int64_t>(r) * p.heads + head0 + row;
        *reinterpret_cast<uint32_t*>(p.out + row_at * D + dim) = pack_bf16x2(x * inv, y * inv);
        if (p.lse && dim == 0) p.lse[row_at] = sum == 0.0f ? -INFINITY : kLn2 * (base + __builtin_amdgcn_logf(sum));
    }
}

// The pieces of an item joined: a workgroup per request and query head, a thread 4 dims of every
// kJoinThreads * 4 / D-th piece.
template <int D>
__global__ __launch_bounds__(kJoinThreads) void paged_attention_join_kernel(const PagedAttnArgs p) {
    constexpr int kAcross = D / 4, kDown = kJoinThreads / kAcross;
    __shared__ f32x4_t o_s[kDown][kAcross];
    __shared__ float l_s[kDown], m_s[kJoinThreads / 64];
    const int r = static_cast<int>(blockIdx.x) / p.heads, h = static_cast<int>(blockIdx.x) - r * p.heads;
    const int2 held = *reinterpret_cast<const int2*>(p.pieces + 2 * r);
    const int mine = held.y;
    if (mine == 1) return;      // written by the one workgroup
    const int kvh = h / p.group, q = h - kvh * p.group;
    const int rows = p.group < 16 ? p.group : 16, heads = p.kv_heads * p.head_tiles;
    auto place = [&](int s) {
        return (static_cast<int64_t>(held.x + s) * heads + kvh * p.head_tiles + q / 16) * rows + q % 16;
    };
    const int tid = static_cast<int>(threadIdx.x);
    float top = -INFINITY;
    for (int s = tid; s < mine; s += kJoinThreads) top = fmaxf(top, p.part_ml[2 * place(s)]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63) == 0) m_s[tid / 64] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 64; ++w) top = fmaxf(top, m_s[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    const int c = tid % kAcross, down = tid / kAcross;
    f32x4_t o{0.0f, 0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
#pragma unroll 4
    for (int s = down; s < mine; s += kDown) {
        const int64_t at = place(s);
        const f32x2_t ml = *reinterpret_cast<const f32x2_t*>(p.part_ml + 2 * at);
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p.part_o + at * D + 4 * c);
        const float f = __builtin_amdgcn_exp2f(ml[0] - base);
        sum += f * ml[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += f * x[e];
    }
    if (__builtin_expect(__builtin_isunordered(o[0], o[1]) || __builtin_isunordered(o[2], o[3]), 0)) {
        o = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = down; s < mine; s += kDown) {
            const int64_t at = place(s);
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p.part_o + at * D + 4 * c);
            const float f = __builtin_amdgcn_exp2f(p.part_ml[2 * at] - base);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += weight_of(f, x[e]) * x[e];
        }
    }
    o_s[down][c] = o;
    if (c == 0) l_s[down] = sum;
    __syncthreads();
    if (tid >= kAcross) return;
    o = o_s[0][tid];
    sum = l_s[0];
#pragma unroll
    for (int w = 1; w < kDown; ++w) {
        const f32x4_t x = o_s[w][tid];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += x[e];
        sum += l_s[w];
    }
    const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
    const int64_t row_at = static_cast<int64_t>(r) * p.heads + h;
    *reinterpret_cast<uint2*>(p.out + row_at * D + 4 * tid) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (p.lse && tid == 0) p.lse[row_at] = sum == 0.0f ? -INFINITY : kLn2 * (base + __builtin_amdgcn_logf(sum));
}

template <int D, bool FP8>
hipError_t launch(const PagedAttnArgs& a, hipStream_t s) {
    const int rows = a.group < 16 ? a.group : 16;
    constexpr unsigned kKeys = kWaves * KvTile<D, FP8>::kBytes;
    const unsigned sums = static_cast<unsigned>(kWaves * rows * (D + 4) * 4), lds = kKeys > sums ? kKeys : sums;
    const unsigned items = static_cast<unsigned>(a.requests) * static_cast<unsigned>(a.kv_heads * a.head_tiles);
    if (a.aim == 0) {
        paged_attention_kernel<D, FP8, false><<<items, 64 * kWaves, lds, s>>>(a);
        return hipGetLastError();
    }
    paged_attention_kernel<D, FP8, true><<<items + static_cast<unsigned>(a.aim), 64 * kWaves, lds, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    paged_attention_join_kernel<D><<<static_cast<unsigned>(a.requests) * static_cast<unsigned>(a.heads), kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Items are cut where the longest may pass 176 KB of keys (704 tokens of 256 bytes) or 1024 tokens.
// Measured at 8 kv heads (us, whole | cut), one request of 256-byte rows: 400 tokens 7.4 | 10.0,
// 640 7.5 | 8.7, 777 9.3 | 9.0, 1024 10.5 | 9.0; 64 uneven ones of up to 640 tokens 16 | 20, 1280 29 | 28;
// 512-byte rows, 640 tokens: 19.6 | 12.4; 64-byte rows, 1024 tokens: 8.9 | 9.1.  Beyond 4096 items the
// items alone are several rounds of what the chip holds, which is enough where lengths are alike: 1024 requests of
// 300 to 700 tokens read 6.0 TB/s.  One long request among them is one workgroup's, though: 513 with one of 131072
// tokens take 1251 us, and 512, which are cut, 259.
// 1024 pieces, 4 a CU: 512 lost up to 9% (the last ones leave CUs idle), 2048 up to 7% where there are
// few kv heads and heads of 256 dims (beginnings and ends of pieces), and gained at most 4% elsewhere.
// A piece has at least a tile a wave.
void plan_paged_attention(PagedAttnArgs* a, int row_bytes, int max_len) {
    constexpr int kWholeBytes = 176 << 10, kWholeTokens = 1024, kMaxItems = 4096, kPieces = 1024;
    int64_t reach = static_cast<int64_t>(a->max_pages) * a->page_size;
    const int64_t tiles = a->requests * (reach / 32 + 1);
    if (max_len > 0 && max_len < reach) reach = max_len;
    if (a->window > 0 && a->window < reach) reach = a->window;
    const int64_t items = static_cast<int64_t>(a->requests) * a->kv_heads * a->head_tiles;
    const bool whole = reach <= kWholeTokens && reach * row_bytes <= kWholeBytes;
    a->least = kWaves;
    a->aim = whole || items > kMaxItems || tiles >= (int64_t(1) << 31) ? 0 : kPieces;
}

hipError_t launch_paged_attention(const PagedAttnArgs& a, int head_dim, bool fp8, hipStream_t s) {
    switch (head_dim) {
        case 64: return fp8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
        case 128: return fp8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
        default: return fp8 ? launch<256, true>(a, s) : launch<256, false>(a, s);
    }
}

}  // namespace dlf
