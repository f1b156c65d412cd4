// The matrix-core GEMM of q8ta_linear_per_token (gemm_scaled.h).
#include "gemm_scaled.h"

namespace q8ta {

hipError_t launch_linear_tiles(const ScaledArgs& a, hipStream_t s) { return launch_type<1>(a, s); }

}  // namespace q8ta
