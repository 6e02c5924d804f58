// Attention of one new token per request over a paged key-value cache.
//
// For a request, a kv head and the up to 16 query heads q of its group that share a tile:
//     s_j = scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j)
// in one pass over the tokens j, with the running maximum m and sum l of the softmax: a tile's new
// maximum m' rescales what is summed so far by exp(m - m').
//
// What bounds it is the read of the cache: 4 flops a value at bf16 and one query head, 64 at 16 of
// them, against the hundreds a byte that the matrix cores could do.  So the products need no tuning
// beyond keeping out of the way, and the layout is chosen so that nothing stands between a load and
// the MFMA that uses it, no LDS and no lane exchange:
//  - scores are computed transposed, S^T = K Q^T (16 tokens x 16 queries an MFMA): a lane's key
//    operand is 16 contiguous bytes of one token's row;
//  - the 16x16 result leaves each lane with one query's scores of 4 tokens, which is just the
//    operand that the second product, O^T = V^T P^T, wants from that lane, if its 32 tokens are
//    numbered 4 (lane / 16) + 16 half + 0..3: the probabilities never move;
//  - a lane loads the value rows of those 8 tokens, 1/16 of a row each, and a byte permute of pairs of
//    tokens gives the 8 tokens of each of its dims: the order of the dims among the lanes is free, since
//    the result's rows come out in the same order.
// 16 query rows are computed whatever the group: the rest is zeros and costs nothing that bounds.
#include "device_common.h"
#include "kernels.h"
#include "mma_common.h"

namespace dlf {
namespace {

constexpr int kAttnWaves = 4;
constexpr float kLn2 = 0.693147180559945309f;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// The cache bytes of 32 tokens of one head as a wave holds them.
template <int D, bool FP8>
struct KvTile {
    static constexpr int kRow = D * (FP8 ? 1 : 2);      // bytes of a token's row
    static constexpr int kKeyLoads = kRow / 64;         // 16-byte loads a lane and 16 tokens
    static constexpr int kValWords = kRow / 64;         // 32-bit words of a lane's 1/16 of a row
    u32x4_t k[2][kKeyLoads];
    uint32_t v[8][kValWords];
};

// Two bf16 values a word from two e4m3 codes (exact).
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8x2_to_bf16x2(uint32_t codes) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HIGH));
}

template <int D, bool FP8>
__global__ __launch_bounds__(64 * kAttnWaves, D == 256 ? 1 : 2) void paged_attention_kernel(const PagedAttnArgs p) {
    using Tile = KvTile<D, FP8>;
    constexpr int kRow = Tile::kRow;
    constexpr int kSteps = D / 32;          // MFMA steps over the head's dims
    constexpr int kFrag = D / 16;           // dims a lane's value chunk holds = output fragments
    __shared__ float o_s[kAttnWaves][16][D];
    __shared__ float m_s[kAttnWaves][16], l_s[kAttnWaves][16];

    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int qi = lane & 15, g = lane >> 4;
    int item = static_cast<int>(blockIdx.x);
    const int ht = item % p.head_tiles;
    item /= p.head_tiles;
    const int kvh = item % p.kv_heads, r = item / p.kv_heads;
    const int head0 = kvh * p.group + 16 * ht;                          // first query head of the tile
    const int nq = p.group - 16 * ht < 16 ? p.group - 16 * ht : 16;     // query heads in it

    // the tokens attended to: [lo, len); tiles start at a multiple of 16 so that 16 tokens share a page
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;   // < 2^31
    int len = p.lens[r];
    len = len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
    const int lo = p.window > 0 && len > p.window ? len - p.window : 0;
    const int t16 = lo & ~15;
    const int tiles = (len - t16 + 31) / 32;
    const int a = tiles * wave / kAttnWaves, b = tiles * (wave + 1) / kAttnWaves;

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

    // byte offsets of the cache runs of the next 64 half tiles (16 tokens), one a lane; -1: no page
    const uint32_t per_page = static_cast<uint32_t>(p.page_size) / 16;
    int64_t run = -1;
    auto find_runs = [&](int tile) {
        const int tok = t16 + 32 * tile + 16 * lane;
        run = -1;
        if (tok < len) {
            const uint32_t h16 = static_cast<uint32_t>(tok) / 16, col = h16 / per_page;
            const int32_t page = p.table[static_cast<int64_t>(r) * p.max_pages + col];
            if (page >= 0 && page < p.pages)
                run = ((static_cast<int64_t>(page) * p.kv_heads + kvh) * p.page_size + 16 * (h16 - col * per_page)) * kRow;
        }
    };
    // tile `tile` (wave-uniform) into registers; runs without a page are read from page 0 and masked
    auto fetch = [&](int tile, Tile& t, bool (&there)[2]) {
        if (((tile - a) & 31) == 0) find_runs(tile);
        const int at = 2 * ((tile - a) & 31);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int lo32 = __builtin_amdgcn_readlane(static_cast<int>(run), at + hh);
            const int hi32 = __builtin_amdgcn_readlane(static_cast<int>(run >> 32), at + hh);
            there[hh] = hi32 >= 0;
            const int64_t off = there[hh] ? (static_cast<int64_t>(hi32) << 32) | static_cast<uint32_t>(lo32) : 0;
            const uint8_t* const kp = p.k + off + qi * kRow + 16 * g;
#pragma unroll
            for (int s = 0; s < Tile::kKeyLoads; ++s) t.k[hh][s] = *reinterpret_cast<const u32x4_t*>(kp + 64 * s);
            const uint8_t* const vp = p.v + off + 4 * g * kRow + qi * (kRow / 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t* const w = t.v[4 * hh + j];
                if constexpr (Tile::kValWords == 1) {
                    w[0] = *reinterpret_cast<const uint32_t*>(vp + j * kRow);
                } else if constexpr (Tile::kValWords == 2) {
                    const u32x2_t x = *reinterpret_cast<const u32x2_t*>(vp + j * kRow);
                    w[0] = x[0];
                    w[1] = x[1];
                } else {
#pragma unroll
                    for (int c = 0; c < Tile::kValWords / 4; ++c) {
                        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(vp + j * kRow + 16 * c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[4 * c + e] = x[e];
                    }
                }
            }
        }
    };
    auto attend = [&](int tile, Tile& t, const bool (&there)[2]) {
        f32x4_t sc[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            sc[hh] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                u32x4_t kw;
                if constexpr (FP8) {
                    const u32x4_t x = t.k[hh][s / 2];
                    const uint32_t c0 = x[2 * (s & 1)], c1 = x[2 * (s & 1) + 1];
                    kw = u32x4_t{fp8x2_to_bf16x2<false>(c0), fp8x2_to_bf16x2<true>(c0), fp8x2_to_bf16x2<false>(c1),
                                 fp8x2_to_bf16x2<true>(c1)};
                } else {
                    kw = t.k[hh][s];
                }
                sc[hh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kw), qf[s], sc[hh], 0, 0, 0);
            }
        }
        // lane: query qi, tokens first + 16 hh + e
        const int first = t16 + 32 * tile + 4 * g;
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = sc[i / 4][i & 3] * p.score_scale;
        const int tok0 = t16 + 32 * tile;
        if (tok0 < lo || tok0 + 32 > len || !there[0] || !there[1]) {
            // masked tokens: the score is replaced, whatever it was, and the value row is cleared, since
            // 0 x NaN or 0 x inf of a stale slot would reach the sum
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tok = first + 16 * (i / 4) + (i & 3);
                const bool seen = tok >= lo && tok < len && there[i / 4];
                z[i] = seen ? z[i] : -INFINITY;
#pragma unroll
                for (int w = 0; w < Tile::kValWords; ++w) t.v[i][w] = seen ? t.v[i][w] : 0u;
            }
        }
        float top = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top);
        const float base = mn == -INFINITY ? 0.0f : mn;     // nothing seen yet: every exp2 below is 0
        const float alpha = __builtin_amdgcn_exp2f(m - base);
        m = mn;
        // p = hi + lo in bf16: the 2^-9 of one rounding would reach the output as much as its own rounding
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
        auto add = [&](int i, u32x4_t vt) {
            const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vt);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf, o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pg, o[i], 0, 0, 0);
        };
        // dims 2 w and 2 w + 1 of the lane's chunk, from one word of bf16 pairs of each token
        auto pair = [&](int w, const uint32_t (&x)[8]) {
            u32x4_t even, odd;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                even[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
                odd[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
            }
            add(2 * w, even);
            add(2 * w + 1, odd);
        };
#pragma unroll
        for (int w = 0; w < Tile::kValWords; ++w) {
            uint32_t x[8];
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fp8x2_to_bf16x2<false>(t.v[i][w]);
                pair(2 * w, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fp8x2_to_bf16x2<true>(t.v[i][w]);
                pair(2 * w + 1, x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = t.v[i][w];
                pair(w, x);
            }
        }
    };

    Tile t;
    bool there[2];
    for (int tile = a; tile < b; ++tile) {
        fetch(tile, t, there);
        attend(tile, t, there);
    }

    // ---- the waves' results joined through LDS ----
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (qi < nq) {
        if (g == 0) {
            m_s[wave][qi] = m;
            l_s[wave][qi] = l;
        }
        // fragment i, element e: dim kFrag (4 g + e) + i of query qi
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < kFrag; ++i) o_s[wave][qi][kFrag * (4 * g + e) + i] = o[i][e];
    }
    __syncthreads();
    for (int i = static_cast<int>(threadIdx.x); i < nq * D / 2; i += 64 * kAttnWaves) {
        const int row = i / (D / 2), dim = 2 * (i % (D / 2));
        float top = m_s[0][row];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, m_s[w][row]);
        const float base = top == -INFINITY ? 0.0f : top;
        float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(m_s[w][row] - base);
            x += f * o_s[w][row][dim];
            y += f * o_s[w][row][dim + 1];
            sum += f * l_s[w][row];
        }
        // no token left: zeros.  A sum of NaN is not 0 and goes through.
        const float inv = sum == 0.0f ? 0.0f : p.v_scale / sum;
        const int64_t row_at = static_cast<int64_t>(r) * p.heads + head0 + row;
        *reinterpret_cast<uint32_t*>(p.out + row_at * D + dim) = pack_bf16x2(x * inv, y * inv);
        if (p.lse && dim == 0) p.lse[row_at] = sum == 0.0f ? -INFINITY : kLn2 * (base + __builtin_amdgcn_logf(sum));
    }
}

template <int D, bool FP8>
hipError_t launch(const PagedAttnArgs& a, hipStream_t s) {
    const int64_t items = static_cast<int64_t>(a.requests) * a.kv_heads * a.head_tiles;
    paged_attention_kernel<D, FP8><<<static_cast<unsigned>(items), 64 * kAttnWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attention(const PagedAttnArgs& a, int head_dim, bool fp8, hipStream_t s) {
    switch (head_dim) {
        case 64: return fp8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
        case 128: return fp8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
        default: return fp8 ? launch<256, true>(a, s) : launch<256, false>(a, s);
    }
}

}  // namespace dlf
