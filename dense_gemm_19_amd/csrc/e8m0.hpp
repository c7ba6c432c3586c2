// e8m0.hpp -- scale bytes of microscaled weights that are converted to 16 bits.
#pragma once
#include "device_common.hpp"

namespace dg {

// 2^(b - 127) (0: subnormal, 255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __builtin_bit_cast(float, max(b << 23, 0x00400000u) | (b == 255u ? 0x00400000u : 0u));
}

// A block's weights are converted times `in`, exactly, and their products' sum enters the
// FP32 accumulator times `out`.
// BF16: 6 * 2^126 and 2 * 2^127 are past its range (and FP32's), though their products
// with small activations are not: a quarter of the two largest scales, and 4 times the sum.
// (in: the conversion reads the exponent's bits alone, 0 is 2^-127, all ones NaN.)
// FP16 holds few of the scales, and sums of its products without them pass no range.
struct BlockScale { float in, out; };
template <int IN>
__device__ __forceinline__ BlockScale block_scale(uint32_t b) {
    if constexpr (IN == IN_BF16) {
        const bool past = b - 253u < 2u;
        return {__builtin_bit_cast(float, (past ? b - 2u : b) << 23), past ? 4.0f : 1.0f};
    }
    return {1.0f, e8m0_value(b)};
}

// Not zero where a byte of v is 192 or more, 253 and 254, which BF16 does not hold every
// code times, among them.
__device__ __forceinline__ uint32_t top_scales(uint32_t v) { return v & (v << 1) & 0x80808080u; }

}  // namespace dg
