// Products with block scales for few rows of a, and the join of parts of the sum over k.
#include "gemm_blocks.h"

namespace dlf {
namespace {

// Few rows of a: what bounds is the read of b, once: one row through 4096 x 4096 takes 4.7 us on the device (16.8 MB: 3.2 us at
// a copy's 5.2 TB/s, and 2.2 of an empty launch), through 22016 x 4096 18.5 as called (4.9 TB/s).  A wave has a ring of DEPTH
// stages of its own, of one block of k each, for 16 R rows of b and all 16 TM rows of a, and takes every NW-th block; no wave
// waits for another until their sums are added through LDS at the end.  With blockIdx.y the blocks are cut once more, and
// the parts go to the workspace as they are.
template <int TM, int R, int NW, int DEPTH>
struct Skinny {
    static constexpr int kLoads = 2 * R + 2 * TM + 1;           // of a wave and stage: b, a, and a's scales
    static constexpr int kStage = (R + TM) * 2048 + 256;
    static constexpr int kRing = NW * DEPTH * kStage;
    static constexpr int kRow = 16 * R + 4;                     // floats of a row of sums in LDS
    static constexpr int kSums = NW * TM * 16 * kRow * 4;
    static constexpr int kLds = kRing > kSums ? kRing : kSums;
    static_assert((DEPTH - 1) * kLoads < 64, "loads in flight are counted in 6 bits");
    static_assert(kLds <= 160 * 1024 && TM <= 4, "LDS; a's scales are one load");
};

template <int TM, int R, int NW, int DEPTH, int ACT>
__global__ __launch_bounds__(64 * NW, 2) void gemm_blocks_skinny_kernel(const GemmBlocksArgs p) {
    using S = Skinny<TM, R, NW, DEPTH>;
    constexpr bool GATED = ACT >= kActSiluMul;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = static_cast<int>(blockIdx.x) * 16 * R;
    const int k = p.k, all = (k + kScaleBlock - 1) / kScaleBlock;
    // this part's blocks, and those of them that this wave takes: first, first + NW, ..
    const int part = static_cast<int>(blockIdx.y), begin = part * p.part_blocks;
    const int first = begin + wave, end = begin + p.part_blocks < all ? begin + p.part_blocks : all;
    const int turns = first < end ? (end - first + NW - 1) / NW : 0;
    const int row = lane & 15, g = lane >> 4;

    const int64_t rows_left = p.m < 16 * TM ? p.m : 16 * TM;
    const int cols_left = p.n - n0 < 16 * R ? p.n - n0 : 16 * R;
    const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(p.a, static_cast<uint32_t>(rows_left * k));
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.b + static_cast<int64_t>(n0) * k, static_cast<uint32_t>(static_cast<int64_t>(cols_left) * k));
    const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(p.a_scale, static_cast<uint32_t>(rows_left * p.a_scale_stride * 4));
    // scales of b: uniform, so they come by scalar loads; of the even and of the odd columns
    typedef const __attribute__((address_space(4))) float* scalar_t;
    const int slab = GATED ? 2 * (n0 / (2 * kScaleBlock)) : n0 / kScaleBlock;
    const scalar_t sb0 = (scalar_t)(p.b_scale + static_cast<int64_t>(slab) * p.b_scale_stride), sb1 = GATED ? sb0 + p.b_scale_stride : sb0;
    // Loads as those of the tiles: 8 rows of whole lines each, chunk c of row r at c ^ (r / 2 % 8).  Load l holds rows
    // 8 l .., so that the order of its chunks depends on l's parity.
    const int chunk = (lane & 7) ^ (lane >> 4);
    const uint32_t from = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(k);
    uint8_t* const ring = lds + wave * (DEPTH * S::kStage);
    auto load = [&](int turn, int stage) __attribute__((always_inline)) {
        const int t = first + turn * NW;
        const uint32_t at = static_cast<uint32_t>(t) * kScaleBlock, most = turn < turns ? static_cast<uint32_t>(k) : 0u;
        uint32_t off[2];        // of an even and of an odd load, past k and past the last turn outside the buffers
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t in = at + 16u * static_cast<uint32_t>(chunk ^ (4 * h));
            off[h] = in < most ? from + in : kOutOfRange;
        }
        uint8_t* const to = ring + stage * S::kStage;
#pragma unroll
        for (int l = 0; l < 2 * R; ++l) load_lds16_stream(rb, off[l & 1] + static_cast<uint32_t>(8 * l) * static_cast<uint32_t>(k), to + l * 1024);
#pragma unroll
        for (int l = 0; l < 2 * TM; ++l)
            load_lds16_buf(ra, off[l & 1] + static_cast<uint32_t>(8 * l) * static_cast<uint32_t>(k), to + (2 * R + l) * 1024);
        load_lds4_buf(rsa, turn < turns ? 4u * (static_cast<uint32_t>(lane) * static_cast<uint32_t>(p.a_scale_stride) + static_cast<uint32_t>(t)) : kOutOfRange,
                      to + (R + TM) * 2048);
    };
    f32x4_t acc[R][TM];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (turns > 0) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(d, d);
        float b0 = sb0[first], b1 = sb1[first];
        const uint32_t lo = static_cast<uint32_t>(row * kScaleBlock + 16 * (g ^ (row >> 1))), hi = lo ^ 64u;
        auto read = [&](const uint8_t* base) __attribute__((always_inline)) {
            const u32x4_t a = *reinterpret_cast<const u32x4_t*>(base + lo), b = *reinterpret_cast<const u32x4_t*>(base + hi);
            return i32x8_t{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                           static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
        };
        int stage = 0;
#pragma unroll 1
        for (int turn = 0; turn < turns; ++turn) {
            const uint8_t* const at = ring + stage * S::kStage;
            wait_vmcnt<(DEPTH - 1) * S::kLoads>();
            __builtin_amdgcn_sched_barrier(0);
            i32x8_t w[R], x[TM];
            float sa[TM];
#pragma unroll
            for (int j = 0; j < R; ++j) w[j] = read(at + j * 2048);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                x[i] = read(at + (R + i) * 2048);
                sa[i] = reinterpret_cast<const float*>(at + (R + TM) * 2048)[16 * i + row];
            }
            __builtin_amdgcn_sched_barrier(0);
            wait_vmcnt<63>();           // the LDS reads: the stage is free
            __builtin_amdgcn_sched_barrier(0);
            load(turn + DEPTH, stage);
            const int ahead = turn + 1 < turns ? first + (turn + 1) * NW : first;
            const float c0 = sb0[ahead], c1 = sb1[ahead];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const float s0 = sa[i] * b0, s1 = GATED ? sa[i] * b1 : s0;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const f32x4_t d = mma_block(w[j], x[i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][i][e] = fmaf(d[e], e & 1 ? s1 : s0, acc[j][i][e]);
                }
            }
            b0 = c0;
            b1 = c1;
            stage = stage + 1 < DEPTH ? stage + 1 : 0;
        }
    }
    // ---- the waves' sums, in their order ----
    float* const sums = reinterpret_cast<float*>(lds);
    wait_vmcnt<0>();        // no load of zeros is on its way to LDS any more
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) *reinterpret_cast<f32x4_t*>(sums + ((wave * TM + i) * 16 + row) * S::kRow + 16 * j + 4 * g) = acc[j][i];
    __syncthreads();
    for (int q = tid; q < TM * 16 * 8 * R; q += 64 * NW) {
        const int r = q / (8 * R), c = 2 * (q - r * (8 * R)), n = n0 + c;
        const int64_t m = r;
        if (m >= p.m || n >= p.n) continue;
        f32x2_t v{0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) v += *reinterpret_cast<const f32x2_t*>(sums + (w * TM * 16 + r) * S::kRow + c);
        if (p.parts > 1) *reinterpret_cast<f32x2_t*>(p.part + (part * p.m + m) * p.part_stride + n) = v;
        else finish_pair<ACT>(p, m, n, v[0], v[1]);
    }
}

// The parts of the sum over k joined: a pair of columns a thread.
template <int ACT>
__global__ __launch_bounds__(256) void gemm_blocks_join_kernel(const GemmBlocksArgs p) {
    const int64_t pairs = p.part_stride / 2, q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t m = q / pairs;
    const int n = 2 * static_cast<int>(q - m * pairs);
    if (m >= p.m || n >= p.n) return;
    f32x2_t v{0.0f, 0.0f};
#pragma unroll 4
    for (int s = 0; s < p.parts; ++s) v += *reinterpret_cast<const f32x2_t*>(p.part + (s * p.m + m) * p.part_stride + n);
    finish_pair<ACT>(p, m, n, v[0], v[1]);
}

template <int TM, int R, int NW, int DEPTH, int ACT>
hipError_t launch_skinny(const GemmBlocksArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.n + 16 * R - 1) / (16 * R)), static_cast<unsigned>(a.parts));
    gemm_blocks_skinny_kernel<TM, R, NW, DEPTH, ACT><<<grid, 64 * NW, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    return e;
}

template <int ACT>
hipError_t launch(const GemmBlocksArgs& a, hipStream_t s) {
    switch (a.kind) {
        case kGemmBlocks16: return launch_skinny<1, 1, 4, 4, ACT>(a, s);
        case kGemmBlocks16Wide: return launch_skinny<1, 2, 4, 2, ACT>(a, s);
        case kGemmBlocks32: return launch_skinny<2, 1, 4, 2, ACT>(a, s);
        default: return launch_skinny<2, 2, 4, 2, ACT>(a, s);
    }
}

template <int ACT>
hipError_t launch_join(const GemmBlocksArgs& a, hipStream_t s) {
    gemm_blocks_join_kernel<ACT><<<static_cast<unsigned>((a.m * (a.part_stride / 2) + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_blocks_skinny(const GemmBlocksArgs& a, int act, hipStream_t s) {
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

hipError_t launch_gemm_blocks_join(const GemmBlocksArgs& a, int act, hipStream_t s) {
    switch (act) {
        case kActNone: return launch_join<kActNone>(a, s);
        case kActRelu: return launch_join<kActRelu>(a, s);
        case kActGelu: return launch_join<kActGelu>(a, s);
        case kActGeluErf: return launch_join<kActGeluErf>(a, s);
        case kActSiluMul: return launch_join<kActSiluMul>(a, s);
        case kActGeluMul: return launch_join<kActGeluMul>(a, s);
        default: return launch_join<kActGeluErfMul>(a, s);
    }
}

}  // namespace dlf
