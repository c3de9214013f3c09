// gemm_f32.hip -- the tiled product for fp32 operands.
#include "gemm_kernel.h"

namespace vpa {

hipError_t launch_gemm_tiles_f32(const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    return launch_tiles<4>(t, p, stream);
}

}  // namespace vpa
