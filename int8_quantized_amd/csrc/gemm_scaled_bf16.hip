// The matrix-core GEMM of q8ta_linear_per_token and q8ta_gated_linear, bf16 out (gemm_scaled.h).
#include "gemm_scaled.h"

namespace q8ta {

hipError_t launch_tiles_bf16(const ScaledArgs& a, hipStream_t s) { return launch_mats<Bfloat>(a, s); }

}  // namespace q8ta
