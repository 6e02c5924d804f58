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

// A tile of 64 rows x 64 columns a workgroup of four waves, 16 columns a wave.
template <int ACT>
__global__ __launch_bounds__(256) void gemm_blocks_kernel(const GemmBlocksArgs p, const int tiles_n) {
    constexpr bool GATED = ACT >= kActSiluMul;
    constexpr int kRow = kScaleBlock + 16;
    __shared__ __attribute__((aligned(16))) uint8_t a_s[64 * kRow], b_s[64 * kRow];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int tm = static_cast<int>(blockIdx.x) / tiles_n, tn = static_cast<int>(blockIdx.x) - tm * tiles_n;
    const int64_t m0 = static_cast<int64_t>(tm) * 64;
    const int n0 = tn * 64;
    const int row = lane & 15, g = lane >> 4;
    f32x4_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int blocks = (p.k + kScaleBlock - 1) / kScaleBlock;
    for (int t = 0; t < blocks; ++t) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = (tid + 256 * j) / 8, c = (tid & 7) * 16, at = t * kScaleBlock + c;
            u32x4_t x{0u, 0u, 0u, 0u}, y{0u, 0u, 0u, 0u};
            if (at < p.k) {
                if (m0 + r < p.m) x = *reinterpret_cast<const u32x4_t*>(p.a + (m0 + r) * p.k + at);
                if (n0 + r < p.n) y = *reinterpret_cast<const u32x4_t*>(p.b + static_cast<int64_t>(n0 + r) * p.k + at);
            }
            *reinterpret_cast<u32x4_t*>(a_s + r * kRow + c) = x;
            *reinterpret_cast<u32x4_t*>(b_s + r * kRow + c) = y;
        }
        __syncthreads();
        const i32x8_t w = *reinterpret_cast<const i32x8_t*>(b_s + (16 * wave + row) * kRow + 32 * g);
        const int slab = GATED ? 2 * (n0 / (2 * kScaleBlock)) : n0 / kScaleBlock;
        const float s0 = p.b_scale[static_cast<int64_t>(slab) * p.b_scale_stride + t];
        const float s1 = GATED ? p.b_scale[static_cast<int64_t>(slab + 1) * p.b_scale_stride + t] : s0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const i32x8_t x = *reinterpret_cast<const i32x8_t*>(a_s + (16 * i + row) * kRow + 32 * g);
            const int64_t m = m0 + 16 * i + row;
            const float sa = m < p.m ? p.a_scale[m * p.a_scale_stride + t] : 0.0f;
            const f32x4_t d = mma_block(w, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(d[e], sa * (e & 1 ? s1 : s0), acc[i][e]);
        }
    }
    // lane: row m0 + 16 i + lane % 16, columns n0 + 16 wave + 4 (lane / 16) + e
    const int n = n0 + 16 * wave + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 16 * i + row;
        if (m >= p.m) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][e] + (p.shift && n + e < p.n ? p.shift[n + e] : 0.0f);
        if constexpr (GATED) {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                if (n + e < p.n) p.c[m * (p.n / 2) + (n + e) / 2] = f32_to_bf16(gate_act<ACT>(v[e]) * v[e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= p.n) continue;
                const int64_t at = m * p.n + n + e;
                if (p.residual) v[e] += bf16_to_f32(p.residual[at]);
                p.c[at] = f32_to_bf16(activate<ACT>(v[e]));
            }
        }
    }
}

template <int ACT>
hipError_t launch(const GemmBlocksArgs& a, hipStream_t s) {
    const int64_t tiles_m = (a.m + 63) / 64, tiles_n = (a.n + 63) / 64;
    if (tiles_m * tiles_n >= kMaxWorkgroups) return hipErrorInvalidValue;
    gemm_blocks_kernel<ACT><<<static_cast<unsigned>(tiles_m * tiles_n), 256, 0, s>>>(a, static_cast<int>(tiles_n));
    return hipGetLastError();
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
