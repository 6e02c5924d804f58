// Product of e4m3 matrices with block scales:
//     acc[i][j] = sum_t a_scale[i][t] b_scale[j / 128][t] sum_{k in t} a[i][k] b[j][k],   t = blocks of 128 of k
//     c = act(acc + shift [+ residual]),  or gate(acc[2j]) * acc[2j + 1]
//
// v_mfma_f32_16x16x128_f8f6f4 sums just one block: its result, from a zero start, is scaled and added to
// the fp32 sum by one FMA a value.
#include "block_scale.h"
#include "kernels.h"
#include "mma_common.h"

namespace dlf {
namespace {

// the unscaled form, both operands e4m3
__device__ __forceinline__ f32x4_t mma_block(const i32x8_t& a, const i32x8_t& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// A workgroup's tile: WM x WN waves, each of FM x FN fragments of 16 rows of a and 16 of b.
template <int WM_, int WN_, int FM_, int FN_>
struct BlockTile {
    static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
    static constexpr int BM = 16 * WM * FM, BN = 16 * WN * FN;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;    // 1 KB loads a wave and block of k
    static constexpr int kStage = (BM + BN) * kScaleBlock;      // bytes of a block of k
    static constexpr int kScales = BM * 16 + 1024;              // of four blocks' scales: a's rows, and two rows of b's
    static constexpr int kOut = BM * BN * 2;                    // the staged output
    static constexpr int kLds = 2 * kStage + 2 * kScales > kOut ? 2 * kStage + 2 * kScales : kOut;
    static_assert(FM % 2 == 0, "two buffers in turn");
    static_assert(LA >= 1 && LB >= 1 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW % 2 == 0, "whole loads");
    static_assert(BM % 64 == 0 && (BN == 128 || BN == 256 || BN == 64), "scales of whole waves, at most two rows of b's");
};

// Tile of a linear workgroup number: see tile_coords of the other products.  Neighbouring numbers are dealt to the 8 XCDs
// in turn; each gets a contiguous range, in groups of G tile rows that sweep the columns.
template <int G>
__device__ __forceinline__ void xcd_tile(int tiles_m, int tiles_n, int bid, int& tm, int& tn) {
    const int nb = tiles_m * tiles_n, xcd = bid & 7, local = bid >> 3, q = nb >> 3, r = nb & 7;
    const int id = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + local;
    const int g = id / (G * tiles_n), first = g * G;
    const int rows = tiles_m - first < G ? tiles_m - first : G, in = id - g * G * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

template <class T, int ACT>
__global__ __launch_bounds__(T::NT, 2) void gemm_blocks_kernel(const GemmBlocksArgs p, const int tiles_m, const int tiles_n) {
    constexpr bool GATED = ACT >= kActSiluMul;
    constexpr int FM = T::FM, FN = T::FN;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / T::WN, wn = wave % T::WN;
    int tm, tn;
    xcd_tile<8>(tiles_m, tiles_n, static_cast<int>(blockIdx.x), tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * T::BM;
    const int n0 = tn * T::BN;
    const int k = p.k, blocks = (k + kScaleBlock - 1) / kScaleBlock;
    const int g = lane >> 4, row = lane & 15;

    // Loads: 8 rows of 128 bytes an instruction, whole lines.  Load j of a wave takes rows 8 (wave + NW j) + lane / 8;
    // chunk c of row r lies at place c ^ (r / 2 % 8), so that the 16 rows of a fragment's read fall on all banks.  r / 2 % 8
    // does not depend on j (NW is even): one offset a lane serves all loads.
    const int in_row = lane >> 3, chunk = (lane & 7) ^ ((4 * wave + (in_row >> 1)) & 7);
    const uint32_t from = static_cast<uint32_t>((8 * wave + in_row) * static_cast<int64_t>(k) + 16 * chunk);
    auto panel = [&](const uint8_t* base, int64_t first, int64_t rows, int j) {
        // rows 8 NW j .. of the panel, those past its end outside the buffer
        int64_t left = rows - first - 8 * T::NW * j;
        left = left < 0 ? 0 : left > 8 * T::NW ? 8 * T::NW : left;
        return buffer_rsrc(base + (first + 8 * T::NW * j) * k, static_cast<uint32_t>(left * k));
    };
    __amdgpu_buffer_rsrc_t ra[T::LA], rb[T::LB];
#pragma unroll
    for (int j = 0; j < T::LA; ++j) ra[j] = panel(p.a, m0, p.m, j);
#pragma unroll
    for (int j = 0; j < T::LB; ++j) rb[j] = panel(p.b, n0, p.n, j);
    const int64_t rows_left = p.m - m0 < T::BM ? p.m - m0 : T::BM;
    const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(p.a_scale + m0 * p.a_scale_stride, static_cast<uint32_t>(rows_left * p.a_scale_stride * 4));
    // the two rows of b's scales that the tile may use
    const int slab = GATED ? 2 * (n0 / (2 * kScaleBlock)) : n0 / kScaleBlock;
    const int slabs = GATED ? slab + 2 : (p.n + kScaleBlock - 1) / kScaleBlock;
    const __amdgpu_buffer_rsrc_t rsb = buffer_rsrc(p.b_scale + static_cast<int64_t>(slab) * p.b_scale_stride,
                                                   static_cast<uint32_t>((slabs - slab < 2 ? slabs - slab : 2) * p.b_scale_stride * 4));
    uint8_t* const scales = lds + 2 * T::kStage;
    auto load_block = [&](int t) {
        const uint32_t at = static_cast<uint32_t>(t) * kScaleBlock;
        const uint32_t off = static_cast<int>(at) + 16 * chunk < k ? from + at : kOutOfRange;
        uint8_t* const to = lds + (t & 1) * T::kStage + wave * 1024;
#pragma unroll
        for (int j = 0; j < T::LA; ++j) load_lds16_buf(ra[j], off, to + j * T::NW * 1024);
#pragma unroll
        for (int j = 0; j < T::LB; ++j) load_lds16_buf(rb[j], off, to + T::BM * kScaleBlock + j * T::NW * 1024);
    };
    // scales of blocks 4 u .. 4 u + 3, 16 bytes a row
    auto load_scales = [&](int u) {
        uint8_t* const to = scales + (u & 1) * T::kScales;
        for (int q = wave; q <= T::BM / 64; q += T::NW) {
            if (q < T::BM / 64)
                load_lds16_buf(rsa, static_cast<uint32_t>(64 * q + lane) * static_cast<uint32_t>(p.a_scale_stride) * 4u + 16u * u, to + q * 1024);
            else
                load_lds16_buf(rsb, lane < 2 ? static_cast<uint32_t>(lane) * static_cast<uint32_t>(p.b_scale_stride) * 4u + 16u * u : kOutOfRange,
                               to + T::BM * 16);
        }
    };
    // operand reads: chunks g and 4 + g of row `row` of a fragment (a and b alike: any order of k does)
    const uint32_t lo = static_cast<uint32_t>(row * kScaleBlock + 16 * (g ^ (row >> 1))), hi = lo ^ 64u;
    const uint8_t* const xa = lds + wm * FM * 16 * kScaleBlock;
    const uint8_t* const wb = lds + T::BM * kScaleBlock + wn * FN * 16 * kScaleBlock;
    auto read = [&](const uint8_t* base) {
        const u32x4_t a = *reinterpret_cast<const u32x4_t*>(base + lo), b = *reinterpret_cast<const u32x4_t*>(base + hi);
        return i32x8_t{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                       static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
    };

    f32x4_t acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    if (blocks > 0) {
        load_scales(0);
        load_block(0);
        load_block(1);
        wait_vmcnt<T::LA + T::LB>();
        barrier();
        i32x8_t w[FN], x[2];
        f32x4_t part[2][FN];
        float s0[2], s1[2], b0, b1;         // scales of a fragment's rows times those of its columns, even and odd
        // the scales' place of block t, and row `row` of fragment i of a's
        auto scale_at = [&](int t) { return reinterpret_cast<const float*>(scales + ((t >> 2) & 1) * T::kScales) + (t & 3); };
        const int srow = 4 * (wm * FM * 16 + row);
        const int sb0 = 4 * T::BM + (GATED ? 0 : 4 * (wn * FN * 16 / kScaleBlock)), sb1 = GATED ? sb0 + 4 : sb0;
        const float* sc = scale_at(0);
        b0 = sc[sb0];
        b1 = sc[sb1];
        float sa = sc[srow];
#pragma unroll
        for (int j = 0; j < FN; ++j) w[j] = read(wb + j * 2048);
        x[0] = read(xa);
#pragma unroll
        for (int j = 0; j < FN; ++j) part[(FM - 1) & 1][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        s0[(FM - 1) & 1] = s1[(FM - 1) & 1] = 0.0f;
        auto add = [&](int i) {             // fragment i's block, into its sum
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = fmaf(part[i & 1][j][e], e & 1 ? s1[i & 1] : s0[i & 1], acc[j][i][e]);
        };
        for (int t = 0; t < blocks;) {
            // the next four blocks' scales; those before last have been read by all.  (Outside the loop below, whose
            // body has to stay free of branches: the sums are moved past them otherwise, and their registers spilled.)
            load_scales((t >> 2) + 1);
            const int end = t + 4 < blocks ? t + 4 : blocks;
#pragma unroll 1
            for (; t < end; ++t) {
                const int stage = (t & 1) * T::kStage, next = T::kStage - stage;
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const float s = sa;
                    if (i + 1 < FM) {
                        x[(i + 1) & 1] = read(xa + stage + (i + 1) * 2048);
                        sa = sc[srow + (i + 1) * 64];
                    } else {
                        // every wave has read its last of this block, and has the next one's loads: refill this one
                        wait_vmcnt<0>();
                        barrier();
                        load_block(t + 2);
                        x[(i + 1) & 1] = read(xa + next);
                    }
                    s0[i & 1] = s * b0;
                    s1[i & 1] = GATED ? s * b1 : s0[i & 1];
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        part[i & 1][j] = mma_block(w[j], x[i & 1]);
                        if (i + 1 == FM) w[j] = read(wb + next + j * 2048);
                    }
                    add((i + FM - 1) % FM);
                    if (i + 1 == FM) {
                        sc = scale_at(t + 1);
                        sa = sc[srow];
                        b0 = sc[sb0];
                        b1 = sc[sb1];
                    }
                    // an MFMA, then what the vector ALU and LDS do beside it
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        if (i + 1 == FM) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
                        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        add(FM - 1);
    }

    // ---- epilogue: lane holds row m0 + 16 (wm FM + i) + lane % 16, columns n0 + 16 (wn FN + j) + 4 (lane / 16) + e.
    // The rounded tile goes through LDS, so that every output is written by a 16-byte store of whole lines. ----
    constexpr int kRow = (GATED ? T::BN / 2 : T::BN) * 2, kChunks = kRow / 16;
    constexpr int kMix = (kChunks < 16 ? kChunks : 16) - 1;      // chunk c of row r lies at c ^ (r & kMix)
    wait_vmcnt<0>();
    __syncthreads();
    const int64_t m_last = p.m - 1;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int nl = 16 * (wn * FN + j) + 4 * g, n = n0 + nl;
        float sh[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.shift) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sh[e] = p.shift[n + e < p.n ? n + e : p.n - 1];
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int ml = 16 * (wm * FM + i) + row;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[j][i][e] + sh[e];
            if constexpr (GATED) {
                const int at = nl;          // bytes: columns nl / 2 and nl / 2 + 1
                *reinterpret_cast<uint32_t*>(lds + ml * kRow + (((at >> 4) ^ (ml & kMix)) << 4) + (at & 15)) =
                    pack_bf16x2(gate_act<ACT>(v[0]) * v[1], gate_act<ACT>(v[2]) * v[3]);
            } else {
                if (p.residual) {
                    const int64_t mc = m0 + ml < m_last ? m0 + ml : m_last;
                    if ((p.n & 3) == 0) {
                        const uint2 r = *reinterpret_cast<const uint2*>(p.residual + mc * p.n + (n + 4 <= p.n ? n : p.n - 4));
                        v[0] += __uint_as_float(r.x << 16);
                        v[1] += __uint_as_float(r.x & 0xFFFF0000u);
                        v[2] += __uint_as_float(r.y << 16);
                        v[3] += __uint_as_float(r.y & 0xFFFF0000u);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] += bf16_to_f32(p.residual[mc * p.n + (n + e < p.n ? n + e : p.n - 1)]);
                    }
                }
                const int at = 2 * nl;
                *reinterpret_cast<uint2*>(lds + ml * kRow + (((at >> 4) ^ (ml & kMix)) << 4) + (at & 15)) =
                    make_uint2(pack_bf16x2(activate<ACT>(v[0]), activate<ACT>(v[1])), pack_bf16x2(activate<ACT>(v[2]), activate<ACT>(v[3])));
            }
        }
    }
    __syncthreads();
    const int width = GATED ? p.n / 2 : p.n, first = GATED ? n0 / 2 : n0;
    const bool whole = (width & 7) == 0;
    for (int q = tid; q < T::BM * kChunks; q += T::NT) {
        const int ml = q / kChunks, cc = q - ml * kChunks, n = first + 8 * cc;
        const int64_t m = m0 + ml;
        if (m >= p.m || n >= width) continue;
        const uint8_t* const src = lds + ml * kRow + ((cc ^ (ml & kMix)) << 4);
        uint16_t* const dst = p.c + m * width + n;
        if (whole) {
            *reinterpret_cast<u32x4_t*>(dst) = *reinterpret_cast<const u32x4_t*>(src);
        } else {
            const int count = width - n < 8 ? width - n : 8;
            for (int e = 0; e < count; ++e) dst[e] = reinterpret_cast<const uint16_t*>(src)[e];
        }
    }
}

using Tile256 = BlockTile<2, 4, 8, 4>;      // 256 x 256, a wave 128 x 64
using Tile128 = BlockTile<2, 2, 4, 4>;      // 128 x 128, a wave 64 x 64
using Tile64 = BlockTile<2, 2, 2, 2>;       // 64 x 64, a wave 32 x 32

template <class T, int ACT>
hipError_t launch_tile(const GemmBlocksArgs& a, hipStream_t s) {
    const int64_t tiles_m = (a.m + T::BM - 1) / T::BM, tiles_n = (a.n + T::BN - 1) / T::BN;
    if (tiles_m * tiles_n >= kMaxWorkgroups / 2) return hipErrorInvalidValue;
    gemm_blocks_kernel<T, ACT><<<static_cast<unsigned>(tiles_m * tiles_n), T::NT, 0, s>>>(a, static_cast<int>(tiles_m), static_cast<int>(tiles_n));
    return hipGetLastError();
}

template <int ACT>
hipError_t launch(const GemmBlocksArgs& a, hipStream_t s) {
    if (a.m > 512) return launch_tile<Tile256, ACT>(a, s);
    if (a.m > 64) return launch_tile<Tile128, ACT>(a, s);
    return launch_tile<Tile64, ACT>(a, s);
}

}  // namespace

hipError_t launch_gemm_blocks(const GemmBlocksArgs& a, int act, hipStream_t s) {
    switch (act) {
        case kActNone: return launch<kActNone>(a, s);
        case kActRelu: return launch<kActRelu>(a, s);
        case kActGelu: return launch<kActGelu>(a, s);
        case kActGeluErf: return launch<kActGeluErf>(a, s);
        case kActSiluMul: return launch<kActSiluMul>(a, s);
        case kActGeluMul: return launch<kActGeluMul>(a, s);
        default: return launch<kActGeluErfMul>(a, s);
    }
}

}  // namespace dlf
