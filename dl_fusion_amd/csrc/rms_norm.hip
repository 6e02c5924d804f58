// The norm and the block quantiser of bf16 rows, and the choice between the types (rms_norm.h has the kernels,
// rms_norm_f32.hip those of fp32 rows; two files, so that they compile at the same time).
#include "rms_norm.h"

namespace dlf {

hipError_t launch_rms_norm(const RmsNormArgs& a, bool f32, int out, hipStream_t s) {
    return f32 ? launch_rms_norm_f32(a, out, s) : launch_out<uint16_t>(a, out, s);
}

hipError_t launch_quant_blocks(const QuantBlocksArgs& a, bool f32, hipStream_t s) {
    return f32 ? launch_quant_blocks_f32(a, s) : launch_quant<uint16_t>(a, s);
}

}  // namespace dlf
