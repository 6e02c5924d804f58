// The norm and the block quantiser of fp32 rows.
#include "rms_norm.h"

namespace dlf {

hipError_t launch_rms_norm_f32(const RmsNormArgs& a, int out, hipStream_t s) { return launch_out<float>(a, out, s); }

hipError_t launch_quant_blocks_f32(const QuantBlocksArgs& a, hipStream_t s) { return launch_quant<float>(a, s); }

}  // namespace dlf
