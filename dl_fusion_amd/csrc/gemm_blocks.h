// Device code shared by the products with block scales: the tiles (gemm_blocks.hip) and the kernel for few rows
// (gemm_blocks_skinny.hip).
//     acc[i][j] = sum_t a_scale[i][t] b_scale[j / 128][t] sum_{k in t} a[i][k] b[j][k],   t = blocks of 128 of k
//     c = act(acc + shift [+ residual]),  or gate(acc[2j]) * acc[2j + 1]
//
// v_mfma_f32_16x16x128_f8f6f4 sums just one block: its result, from a zero start, is scaled and added to
// the fp32 sum by one FMA a value.  (Inside a block it aligns the products to the largest of a group of 8 and cuts
// what lies 2^-14 below that: measured 2e-6 rms of sum |a b| on normal values.  The 16x16x32 form does the same; exact
// sums would take the bf16 forms at half the rate, and c has 2^-9 of its own.)
#pragma once

#include "block_scale.h"
#include "kernels.h"
#include "mma_common.h"

namespace dlf {
namespace {

// the unscaled form, both operands e4m3
__device__ __forceinline__ f32x4_t mma_block(const i32x8_t& a, const i32x8_t& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// The epilogue of two neighbouring columns n and n + 1 of row m.
template <int ACT>
__device__ __forceinline__ void finish_pair(const GemmBlocksArgs& p, int64_t m, int n, float v0, float v1) {
    if (p.shift) {
        v0 += p.shift[n];
        if (n + 1 < p.n) v1 += p.shift[n + 1];
    }
    if constexpr (ACT >= kActSiluMul) {
        p.c[m * (p.n / 2) + n / 2] = f32_to_bf16(gate_act<ACT>(v0) * v1);
    } else {
        const int64_t at = m * p.n + n;
        if ((p.n & 1) == 0) {
            if (p.residual) {
                const uint32_t r = *reinterpret_cast<const uint32_t*>(p.residual + at);
                v0 += __uint_as_float(r << 16);
                v1 += __uint_as_float(r & 0xFFFF0000u);
            }
            *reinterpret_cast<uint32_t*>(p.c + at) = pack_bf16x2(activate<ACT>(v0), activate<ACT>(v1));
        } else {
            if (p.residual) {
                v0 += bf16_to_f32(p.residual[at]);
                if (n + 1 < p.n) v1 += bf16_to_f32(p.residual[at + 1]);
            }
            p.c[at] = f32_to_bf16(activate<ACT>(v0));
            if (n + 1 < p.n) p.c[at + 1] = f32_to_bf16(activate<ACT>(v1));
        }
    }
}

}  // namespace
}  // namespace dlf
