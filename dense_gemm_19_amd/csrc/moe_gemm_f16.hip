// moe_gemm_f16.hip -- the experts' products for f16 inputs (see moe_gemm.hpp).
#include "moe_gemm.hpp"

namespace dg {

hipError_t launch_moe_gemm_f16(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units,
                                hipStream_t stream) {
    return moe::launch<IN_F16>(load, tile, b_mode, wgrad, a, units, stream);
}

}  // namespace dg
