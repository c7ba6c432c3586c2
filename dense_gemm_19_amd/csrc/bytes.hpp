// bytes.hpp -- loads of 16 bytes at any alignment, and of the end of a row.
#pragma once
#include "device_common.hpp"

namespace dg {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));

// 16 bytes from p on: elements of BYTES bytes `stride` apart, of which only the
// first `left` may be read; zeros after them.  Single elements are loaded all at
// once: one after another they cost a memory latency each.
template <int BYTES>
__device__ __forceinline__ u32x4 load_part(const char *p, int64_t stride, int left) {
    constexpr int N = 16 / BYTES;
    if (stride == BYTES && left >= N) return *reinterpret_cast<const u32x4_any *>(p);
    uint32_t v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        v[j] = 0;
        if (j < left) v[j] = BYTES == 1   ? *reinterpret_cast<const uint8_t *>(p + j * stride)
                             : BYTES == 2 ? *reinterpret_cast<const uint16_t *>(p + j * stride)
                                          : *reinterpret_cast<const uint32_t *>(p + j * stride);
    }
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        out[w] = 0;
#pragma unroll
        for (int j = 0; j < N / 4; ++j) out[w] |= v[w * (N / 4) + j] << (8 * BYTES * j % 32);
    }
    return out;
}

// The 128 bits of v moved down by `by` bytes (0 to 16), zeros above.
__device__ __forceinline__ u32x4 down_bytes(u32x4 v, int by) {
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    if (by >= 8) {
        lo = by >= 16 ? 0 : hi >> (8 * (by - 8));
        hi = 0;
    } else if (by > 0) {
        lo = lo >> (8 * by) | hi << (64 - 8 * by);
        hi >>= 8 * by;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The first n (1 to 15) bytes of v, zeros above.
__device__ __forceinline__ u32x4 first_bytes(u32x4 v, int n) {
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    if (n < 8) lo &= ((uint64_t)1 << (8 * n)) - 1;
    hi = n > 8 ? hi & (((uint64_t)1 << (8 * (n - 8))) - 1) : 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// 16 bytes from `at` on of a row of `bytes`, zeros past its end.
__device__ __forceinline__ u32x4 row_piece(const char *row, int at, int bytes) {
    const int n = bytes - at;
    if (n >= 16) return *reinterpret_cast<const u32x4_any *>(row + at);
    if (n <= 0) return u32x4{0u, 0u, 0u, 0u};
    if (bytes >= 16) return down_bytes(*reinterpret_cast<const u32x4_any *>(row + bytes - 16), 16 - n);
    return load_part<1>(row + at, 1, n);
}

}  // namespace dg
