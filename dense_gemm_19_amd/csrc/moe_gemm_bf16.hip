// moe_gemm_bf16.hip -- the experts' products for bf16 inputs (see moe_gemm.hpp).
#include "moe_gemm.hpp"

namespace dg {

hipError_t launch_moe_gemm_bf16(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units,
                                hipStream_t stream) {
    return moe::launch<IN_BF16>(load, tile, b_mode, wgrad, a, units, stream);
}

}  // namespace dg
