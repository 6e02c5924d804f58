// Products with block scales: tiles of 64 x 64 to 256 x 256 outputs a workgroup, and the choice among the kernels.
//
// A wave's fragments of b stay in registers for a block of k, those of a pass by, one for each FN MFMAs; each MFMA's result is a
// block's whole sum, which the vector ALU scales and adds while the matrix cores do the next.  That keeps the sums in VGPRs
// (the vector ALU reads no AGPRs), and FN x FM fragments of 4 with the operands' rings are what 256 registers hold: 128 x 64
// a wave, eight waves a CU for 256 x 256 outputs.
//
// What bounds: many rows, the bytes into each CU.  8192 x 22016 x 4096 gated takes 615 to 641 us (2.4 PFLOP/s), 8192 x 4096 x 11008
// 295 to 309 (2.5): the matrix cores are busy 62 to 66% of the clocks at 1.7 to 1.8 GHz; a block's 64 KB come from L2 (80% hits) 330 to 355
// clocks after they are asked for, at 37 KB a us and CU; without the loads (a timing copy) the cores are busy 80%.
// The scaling costs 3.5% (against plain sums).  Smaller tiles take more bytes an output: 777 x 5000 x 4112 33 us in tiles of
// 128 x 128, of which 303 MB into the CUs are 27.  Few rows, the read of b: 64 x 22016 x 4096 gated 18.2 us on the device
// (5.0 TB/s of b), 64 x 4096 x 11008 14 us in four parts of the sum (3.3 TB/s) and 4 for their join.
#include "gemm_blocks.h"

namespace dlf {
namespace {

// A workgroup's tile: WM x WN waves, each of FM x FN fragments of 16 rows of a and 16 of b.
template <int WM_, int WN_, int FM_, int FN_, int STAGES_ = 2, int WAVES_ = 2>
struct BlockTile {
    static constexpr int STAGES = STAGES_;                      // blocks of k in LDS
    static constexpr int kWaves = WAVES_;                       // on a SIMD at least: its registers are shared by that many
    static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
    static constexpr int BM = 16 * WM * FM, BN = 16 * WN * FN;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;    // 1 KB loads a wave and block of k
    static constexpr int kStage = (BM + BN) * kScaleBlock;      // bytes of a block of k
    // scales in LDS, kGroup blocks of k at a time: of a's rows, in the order in which a lane wants them, the same row of
    // four fragments together; and of two rows of b's
    static constexpr int kGroup = 8;
    static constexpr int H = (FM + 3) / 4;
    static constexpr int kARow = WM * H * 64;                   // floats of a block
    static constexpr int kScales = (kGroup * kARow + 2 * kGroup) * 4;
    static constexpr int kOut = BM * BN * 2;                    // the staged output
    static constexpr int kRing = STAGES * kStage;
    static constexpr int kLds = kRing + 2 * kScales > kOut ? kRing + 2 * kScales : kOut;
    static_assert(FM % 4 == 0 && NW == FM && LA % 2 == 0 && (LA + LB) % FM == 0, "a load of a is half of a wave's rows; the loads go evenly into the groups");
    static_assert(LA >= 1 && LB >= 1 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW % 2 == 0, "whole loads");
    static_assert(BM % 64 == 0 && (BN == 128 || BN == 256 || BN == 64), "scales of whole waves, at most two rows of b's");
};

// Tile of a linear workgroup number.  Neighbouring numbers are dealt to the 8 XCDs in turn; each XCD gets a contiguous range, in
// groups of G tile rows that sweep the columns, so that the 32 tiles that run on it share panels in its L2.  (G = 4 and 16
// were not faster than 8.)
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
__global__ __launch_bounds__(T::NT, T::kWaves) void gemm_blocks_kernel(const GemmBlocksArgs p, const int tiles_m, const int tiles_n) {
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
    const int k = p.k;
    // this part's blocks of k: `blocks` from `begin` on, a multiple of 4
    const int begin = static_cast<int>(blockIdx.y) * p.part_blocks, all = (k + kScaleBlock - 1) / kScaleBlock;
    const int blocks = begin + p.part_blocks < all ? p.part_blocks : all - begin;
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
    float* const scales = reinterpret_cast<float*>(lds + T::kRing);
    constexpr int kLoads = T::LA + T::LB;
    auto load_off = [&](int t) {
        const uint32_t at = static_cast<uint32_t>(begin + t) * kScaleBlock;
        return static_cast<int>(at) + 16 * chunk < k ? from + at : kOutOfRange;
    };
    // Load q of this wave's of a block, whose offset is `off`, to a stage: b's, then those of a's with the first halves of the
    // waves' rows, which are wanted first, then the second halves'.  Past k: zeros.  Past the end of a part of the sum: the next
    // part's blocks, STAGES of them, which nobody reads.
    auto load_part = [&](int stage, int q, uint32_t off) {
        uint8_t* const to = lds + stage + wave * 1024;
        if (q < T::LB) {
            load_lds16_buf(rb[q < T::LB ? q : 0], off, to + T::BM * kScaleBlock + q * T::NW * 1024);
        } else {
            const int h = q - T::LB, j = h < T::LA / 2 ? 2 * h : 2 * (h - T::LA / 2) + 1;
            load_lds16_buf(ra[q < T::LB ? 0 : j], off, to + j * T::NW * 1024);
        }
    };
    // Scales of the blocks kGroup u ..: two lanes a row and 16 bytes a lane, through registers, since LDS wants them in
    // another order.  What lies past a row's last block is never used.
    constexpr int kMine = T::BM / T::NW;                        // rows of a wave
    const int arow = wave * kMine + (lane >> 1);
    const bool mine = lane < 2 * kMine;
    u32x4_t next_a{0u, 0u, 0u, 0u};
    uint32_t next_b = 0;
    auto fetch_scales = [&](int u) {
        const uint32_t at = static_cast<uint32_t>(begin + u * T::kGroup) * 4u;
        next_a = __builtin_amdgcn_raw_buffer_load_b128(
            rsa, mine ? static_cast<uint32_t>(arow) * static_cast<uint32_t>(p.a_scale_stride) * 4u + at + 16u * (lane & 1) : kOutOfRange, 0, 0);
        if (wave == 0)
            next_b = __builtin_amdgcn_raw_buffer_load_b32(
                rsb, lane < 2 * T::kGroup ? (lane / T::kGroup) * static_cast<uint32_t>(p.b_scale_stride) * 4u + at + 4u * (lane % T::kGroup) : kOutOfRange, 0, 0);
    };
    auto keep_scales = [&](int u) {
        float* const to = scales + (u & 1) * (T::kScales / 4);
        const int frag = arow >> 4, in_wave = frag % FM;
        const int at = ((frag / FM) * T::H + (in_wave >> 2)) * 64 + 4 * (arow & 15) + (in_wave & 3);
        if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) to[(4 * (lane & 1) + e) * T::kARow + at] = __uint_as_float(next_a[e]);
        }
        if (wave == 0 && lane < 2 * T::kGroup) to[T::kGroup * T::kARow + lane] = __uint_as_float(next_b);
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

    // A block is FM groups of FN MFMAs.  With many groups its place in LDS comes free in two steps: b's rows and the first halves
    // of the waves' rows of a with group kHalf, when all have read them, the second halves DEPTH groups before the end; the loads
    // of the block that is to lie there follow as evenly as the MFMAs, kEach a group, so that they find no queue and each has more
    // than a block's time, and the same two barriers say that the loads that are read next have landed.  With few groups a second
    // barrier costs more than it gives: all comes free DEPTH groups before the end.  In a ring of three all loads follow at once;
    // in a ring of two half of them do and half in the next block's first group, which is faster where two workgroups share a CU.
    // (us, one step | two, with inputs that no cache holds: 8192 x 22016 x 4096 gated 651 | 627, 8192 x 4096 x 11008 316 | 299;
    // 777 x 5000 x 4112, four groups, 34.3 | 38.5.  Four groups, a ring of two, half of the loads later | none: 777 x 5000 x 4112
    // 33.3 | 35.1, 640 x 8192 x 2048 18.9 | 19.4.)
    constexpr int DEPTH = 2, RING = 4;      // fragments of a are read DEPTH groups of MFMAs ahead
    constexpr bool kTwice = FM >= 8;
    constexpr int kHalf = FM / 2 - 2, kEach = kLoads / FM;
    constexpr bool kOnce = T::STAGES > 2;
    constexpr int kNow = kOnce ? kLoads : kLoads / 2;       // of the loads in one step, those that follow at once
    static_assert(!kTwice || T::STAGES == 2, "a ring of two stages frees in two steps");
    if (blocks > 0) {
        fetch_scales(0);
#pragma unroll
        for (int b = 0; b + 1 < T::STAGES; ++b)
#pragma unroll
            for (int q = 0; q < kLoads; ++q) load_part(b * T::kStage, q, load_off(b));
        keep_scales(0);
        fetch_scales(1);
        wait_vmcnt<(T::STAGES - 2) * kLoads>();
        barrier();
#pragma unroll
        for (int q = 0; q < (kTwice ? kLoads - kHalf * kEach : kNow); ++q) load_part((T::STAGES - 1) * T::kStage, q, load_off(T::STAGES - 1));
        i32x8_t w[FN], x[RING];
        f32x4_t sa[T::H];                   // scales of the rows of four fragments
        float b0, b1;                       // of the wave's columns, even and odd
        f32x4_t part[2][FN];
        const int b_at = T::kGroup * T::kARow + (GATED ? 0 : T::kGroup * (wn * FN * 16 / kScaleBlock));
        const float* sc;                    // the scales of a block
        auto scales_of = [&](int t) { sc = scales + (t / T::kGroup & 1) * (T::kScales / 4) + (t % T::kGroup) * T::kARow; };
        auto read_sa = [&](int h) { sa[h] = *reinterpret_cast<const f32x4_t*>(sc + (wm * T::H + h) * 64 + 4 * row); };
        auto read_b = [&](int t) {
            const float* const from = scales + (t / T::kGroup & 1) * (T::kScales / 4) + b_at + t % T::kGroup;
            b0 = from[0];
            b1 = GATED ? from[T::kGroup] : b0;
        };
        scales_of(0);
        read_sa(0);
        read_b(0);
#pragma unroll
        for (int j = 0; j < FN; ++j) w[j] = read(wb + j * 2048);
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) x[i] = read(xa + i * 2048);
#pragma unroll
        for (int j = 0; j < FN; ++j) part[(FM - 1) & 1][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        float s0 = 0.0f, s1 = 0.0f;         // of the group whose sums are added next
        int stage = 0;                      // of block t
        for (int t = 0; t < blocks;) {
            // The next kGroup blocks' scales into LDS, where those before the present ones have been used by all, and the ones
            // after on their way.  (Outside the loop below, whose body has to stay free of branches: the sums are moved
            // past them otherwise, and their registers spilled.)
            keep_scales(t / T::kGroup + 1);
            fetch_scales(t / T::kGroup + 2);
            const int end = t + T::kGroup < blocks ? t + T::kGroup : blocks;
#pragma unroll 1
            for (; t < end; ++t) {
                const int next = stage + T::kStage < T::kRing ? stage + T::kStage : 0, last = stage > 0 ? stage - T::kStage : T::kRing - T::kStage;
                const uint32_t off_last = load_off(t + T::STAGES - 1), off = load_off(t + T::STAGES);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    if (kTwice && i == kHalf) {
                        wait_vmcnt<(T::STAGES - 1) * kLoads>();
                        barrier();
                    }
                    if (i == FM - DEPTH) {
                        wait_vmcnt<(T::STAGES - 2) * kLoads + (kTwice ? T::LA / 2 + (FM - DEPTH - kHalf) * kEach : 0)>();
                        barrier();
                    }
                    // loads of block t + STAGES to this one's place, or the rest of the last one's
                    if (kTwice) {
#pragma unroll
                        for (int q = 0; q < kEach; ++q) {
                            if (i >= kHalf) load_part(stage, (i - kHalf) * kEach + q, off);
                            else load_part(last, (i - kHalf + FM) * kEach + q, off_last);
                        }
                    } else if (i >= FM - DEPTH) {
#pragma unroll
                        for (int q = 0; q < kNow / 2; ++q) load_part(stage, (i - FM + DEPTH) * (kNow / 2) + q, off);
                    } else if (i == 0) {
#pragma unroll
                        for (int q = kNow; q < kLoads; ++q) load_part(last, q, off_last);
                    }
                    const float t0 = s0, t1 = s1;
                    s0 = sa[i >> 2][i & 3] * b0;
                    s1 = GATED ? sa[i >> 2][i & 3] * b1 : s0;
                    if (T::H > 1 && i + 1 < T::H) read_sa(i + 1);
                    if (i + 1 == FM) {
                        scales_of(t + 1);
                        read_sa(0);
                        read_b(t + 1);
                    }
                    const int f = (i + DEPTH) % FM;
                    x[(i + DEPTH) % RING] = read(xa + (i + DEPTH < FM ? stage : next) + f * 2048);
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        part[i & 1][j] = mma_block(w[j], x[i % RING]);
                        if (i + 1 == FM) w[j] = read(wb + next + j * 2048);
                    }
                    // meanwhile the last group's into their sums
                    const int l = (i + FM - 1) % FM;
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][l][e] = fmaf(part[l & 1][j][e], e & 1 ? t1 : t0, acc[j][l][e]);
                    // an MFMA, then what the vector ALU, LDS and the loads do beside it
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        if (kTwice ? j < kEach : kOnce ? i >= FM - DEPTH : j % 2 == 0 && (i == 0 || i >= FM - DEPTH))
                            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                        if (i + 1 == FM) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
                        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                stage = next;
            }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][FM - 1][e] = fmaf(part[(FM - 1) & 1][j][e], e & 1 ? s1 : s0, acc[j][FM - 1][e]);
    }

    // a part of the sum goes to the workspace as it is
    if (p.parts > 1) {
        wait_vmcnt<0>();        // the last loads are on their way to LDS yet
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int64_t m = m0 + 16 * (wm * FM + i) + row;
                const int n = n0 + 16 * (wn * FN + j) + 4 * g;
                if (m >= p.m || n >= p.part_stride) continue;
                *reinterpret_cast<f32x4_t*>(p.part + (blockIdx.y * p.m + m) * p.part_stride + n) = acc[j][i];
            }
        return;
    }
    // ---- epilogue: lane holds row m0 + 16 (wm FM + i) + lane % 16, columns n0 + 16 (wn FN + j) + 4 (lane / 16) + e.
    // The rounded tile goes through LDS, so that every output is written by a 16-byte store of whole lines. ----
    constexpr int kRow = (GATED ? T::BN / 2 : T::BN) * 2, kChunks = kRow / 16;
    constexpr int kMix = (kChunks < 16 ? kChunks : 16) - 1;      // chunk c of row r lies at c ^ (r & kMix)
    wait_vmcnt<0>();
    __syncthreads();
    // the residual comes by loads of whole lines to where the outputs will lie
    const bool staged = !GATED && p.residual && (p.n & 7) == 0;
    if (staged) {
        constexpr int kRows = 1024 / kRow;                       // of a load
#pragma unroll
        for (int l = 0; l < T::BM / kRows / T::NW; ++l) {
            const int r0 = kRows * T::NW * l, r = kRows * wave + lane / kChunks, c = (lane % kChunks) ^ ((r0 + r) & kMix);
            int64_t left = p.m - m0 - r0;
            left = left < 0 ? 0 : left > kRows * T::NW ? kRows * T::NW : left;
            const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(p.residual + (m0 + r0) * p.n, static_cast<uint32_t>(left * p.n * 2));
            load_lds16_buf(rr, n0 + 8 * c < p.n ? 2u * (static_cast<uint32_t>(r) * static_cast<uint32_t>(p.n) + n0 + 8 * c) : kOutOfRange,
                           lds + (r0 + kRows * wave) * kRow);
        }
        wait_vmcnt<0>();
        __syncthreads();
    }
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
            const int at = GATED ? nl : 2 * nl;                  // bytes: columns nl / 2 and nl / 2 + 1, or the four
            uint8_t* const to = lds + ml * kRow + (((at >> 4) ^ (ml & kMix)) << 4) + (at & 15);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[j][i][e] + sh[e];
            if constexpr (GATED) {
                *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(gate_act<ACT>(v[0]) * v[1], gate_act<ACT>(v[2]) * v[3]);
            } else {
                if (staged) {
                    const uint2 r = *reinterpret_cast<const uint2*>(to);
                    v[0] += __uint_as_float(r.x << 16);
                    v[1] += __uint_as_float(r.x & 0xFFFF0000u);
                    v[2] += __uint_as_float(r.y << 16);
                    v[3] += __uint_as_float(r.y & 0xFFFF0000u);
                } else if (p.residual) {
                    const int64_t mc = m0 + ml < m_last ? m0 + ml : m_last;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += bf16_to_f32(p.residual[mc * p.n + (n + e < p.n ? n + e : p.n - 1)]);
                }
                *reinterpret_cast<uint2*>(to) =
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
using Tile128 = BlockTile<2, 2, 4, 4>;      // 128 x 128, a wave 64 x 64; two workgroups a CU
// The same alone on its CU, where there are no more than CUs (us, two stages | three: 1024 x 4096 x 4096 30.3 | 26.5, 512 x 5000 x
// 4112 30.1 | 26.1).
using Tile128Deep = BlockTile<2, 2, 4, 4, 3, 1>;
using Tile64 = BlockTile<1, 4, 4, 1, 3, 3>;    // 64 x 64, a wave 64 x 16

template <class T, int ACT>
hipError_t launch_tile(const GemmBlocksArgs& a, hipStream_t s) {
    const int64_t tiles_m = (a.m + T::BM - 1) / T::BM, tiles_n = (a.n + T::BN - 1) / T::BN;
    if (tiles_m * tiles_n * T::NT >= int64_t(1) << 32) return hipErrorInvalidValue;     // threads of a grid's dimension
    const dim3 grid(static_cast<unsigned>(tiles_m * tiles_n), static_cast<unsigned>(a.parts));
    gemm_blocks_kernel<T, ACT><<<grid, T::NT, 0, s>>>(a, static_cast<int>(tiles_m), static_cast<int>(tiles_n));
    return hipGetLastError();
}

template <int ACT>
hipError_t launch(const GemmBlocksArgs& a, hipStream_t s) {
    switch (a.kind) {
        case kGemmBlocksTile64: return launch_tile<Tile64, ACT>(a, s);
        case kGemmBlocksTile128: return launch_tile<Tile128, ACT>(a, s);
        case kGemmBlocksTile128Deep: return launch_tile<Tile128Deep, ACT>(a, s);
        default: return launch_tile<Tile256, ACT>(a, s);
    }
}

// What a tile takes, in us: `more`, and for each block of k slope + share w + chip f, w workgroups on its CU and a share f of all
// places of the chip taken.  Fitted to 224 sizes of 33 to 8192 rows, 300 to 22016 columns and sums of 1024 to 11008, each
// measured with every tile and number of parts; the choice by it is 0.6% slower than the best on average, 11% at worst.
struct TileCost {
    int kind, rows, cols, on_a_cu;
    double slope, share, chip, more;
};
constexpr TileCost kCosts[] = {
    {kGemmBlocksTile64, 64, 64, 3, 0.13, 0.15, 0.0, 0.8},
    {kGemmBlocksTile128, 128, 128, 2, 0.34, 0.28, 0.0, 0.8},
    {kGemmBlocksTile128Deep, 128, 128, 1, 0.48, 0.0, 0.1, 1.2},
    {kGemmBlocksTile256, 256, 256, 1, 0.66, 0.0, 0.64, 2.7},
};

}  // namespace

// Up to 32 rows: the kernel for few rows.  32 rows of b a workgroup instead of 16 from 6144 columns on (us, 16 | 32, one
// row of 4096: 4096 columns 6.1 | 6.2, 8192 9.4 | 8.4, 22016 22 | 18.5).  A sum of more than 8 turns a wave
// is cut into parts where the columns alone leave CUs idle (one row of 11008, 1024 columns: 7.2 | 6.5 in 4 parts; 2048
// columns of 4096 stay whole: 4.6 | 5.9).
// Above: the tile and the parts of the sum that the costs above say.  Parts are joined by another launch and 8 bytes an output
// and part.
void plan_gemm_blocks(GemmBlocksArgs* a) {
    constexpr int kCus = 256;
    const int all = (a->k + kScaleBlock - 1) / kScaleBlock;
    a->parts = 1;
    a->part_blocks = all;
    a->part_stride = (a->n + 3) / 4 * 4;
    a->kind = kGemmBlocks16;
    if (a->m == 0 || a->n == 0) return;
    // whole fours of blocks a part: their scales are one load
    auto cut = [&](int want, int* blocks) {
        if (want == 1 || all == 0) {
            *blocks = all;
            return 1;
        }
        *blocks = ((all + want - 1) / want + 3) / 4 * 4;
        return (all + *blocks - 1) / *blocks;
    };
    if (a->m <= 32) {
        const bool wide = a->n > 6144;
        a->kind = a->m <= 16 ? (wide ? kGemmBlocks16Wide : kGemmBlocks16) : (wide ? kGemmBlocks32Wide : kGemmBlocks32);
        const int groups = (a->n + 15) / 16;
        if (all > 32 && !wide && groups <= kCus / 2) {
            const int want = kCus / groups;
            a->parts = cut(want < 8 ? want : 8, &a->part_blocks);
        }
        return;
    }
    double best = 0;
    for (const TileCost& c : kCosts) {
        const int64_t tiles = (a->m + c.rows - 1) / c.rows * ((a->n + c.cols - 1) / c.cols);
        for (int want : {1, 2, 3, 4, 6, 8}) {
            int blocks;
            const int parts = cut(want, &blocks);
            if (parts != want || (parts > 1 && tiles >= 4 * kCus)) continue;
            const int64_t groups = tiles * parts, full = groups / (kCus * c.on_a_cu), rest = groups - full * kCus * c.on_a_cu;
            double us = static_cast<double>(full) * (blocks * (c.slope + c.share * c.on_a_cu + c.chip) + c.more);
            if (rest > 0)
                us += blocks * (c.slope + c.share * static_cast<double>((rest + kCus - 1) / kCus) + c.chip * static_cast<double>(rest) / (kCus * c.on_a_cu)) + c.more;
            if (parts > 1) us += 2.1 + parts * static_cast<double>(a->m) * a->n * 8 / 5e6;
            if (best == 0 || us < best) {
                best = us;
                a->kind = c.kind;
                a->parts = parts;
                a->part_blocks = blocks;
            }
        }
    }
}

hipError_t launch_gemm_blocks(const GemmBlocksArgs& a, int act, hipStream_t s) {
    auto go = [&]() -> hipError_t {
        switch (act) {
            case kActNone: return launch<kActNone>(a, s);
            case kActRelu: return launch<kActRelu>(a, s);
            case kActGelu: return launch<kActGelu>(a, s);
            case kActGeluErf: return launch<kActGeluErf>(a, s);
            case kActSiluMul: return launch<kActSiluMul>(a, s);
            case kActGeluMul: return launch<kActGeluMul>(a, s);
            default: return launch<kActGeluErfMul>(a, s);
        }
    };
    const hipError_t e = a.kind <= kGemmBlocks32Wide ? launch_gemm_blocks_skinny(a, act, s) : go();
    return e != hipSuccess || a.parts == 1 ? e : launch_gemm_blocks_join(a, act, s);
}

}  // namespace dlf
