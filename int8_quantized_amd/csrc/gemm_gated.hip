// The matrix-core GEMM of q8ta_gated_linear (gemm_scaled.h).
#include "gemm_scaled.h"

namespace q8ta {

hipError_t launch_gated_tiles(const ScaledArgs& a, hipStream_t s) { return launch_type<2>(a, s); }

}  // namespace q8ta
