// gemm_bf16.hip -- the tiled product for bf16 operands.
#include "gemm_kernel.h"

namespace vpa {

hipError_t launch_gemm_tiles_bf16(const GemmTask& t, const GemmPlan& p, hipStream_t stream) {
    return launch_tiles<2>(t, p, stream);
}

}  // namespace vpa
