// mx4_quant.hip -- quantiser of the microscaled 4-bit format (MXFP4, OCP Microscaling
// Formats v1.0) and its inverse.
//
// A block is 32 elements along K.  With a the largest size of an element,
//   e = floor(log2 a) - 2         (FLOOR: sizes above 6 * 2^e become 6 * 2^e), or
//   e = the least with a <= 6 * 2^e   (CEIL: nothing saturates),
//   b = max(e + 127, 0)           the scale's byte, 2^(b - 127)
//   q = E2M1(x / 2^(b - 127))     0, .5, 1, 1.5, 2, 3, 4 or 6 with sign, ties to even.
// Both are read off the FP32 bits of a: its exponent field less 2, one more for CEIL
// where the fraction is above 1.5.  The division by a power of two and the rounding
// are one instruction for two elements.  A block that holds a NaN or an infinity gets
// b = 255 (NaN) and codes of zero.
//
// Bound by memory: 2.53 bytes an element for 16-bit X, the same on the way back.  BF16
// rows, 4096 x 8192: 18.9 us (4.5 TB/s), columns 21.7 (3.9), read back 14336 x 4096 30.3
// (4.9; a copy reaches 5.2).
#include "bytes.hpp"
#include "device_common.hpp"
#include "mx4.hpp"

namespace dg {
namespace {

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int esize(int kind) { return kind == OUT_F32 ? 4 : 2; }

// The scale's byte for a block whose largest size has these FP32 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, int ceil) {
    if (top >= 0x7f800000u) return 255u;
    const int b = (int)(top >> 23) - 2 + (ceil && (top & 0x7fffffu) > 0x400000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}

// 2^(b - 127) for b < 255.
__device__ __forceinline__ float power(uint32_t b) { return __builtin_bit_cast(float, max(b << 23, 0x00400000u)); }

// 8 elements as 32-bit words: 8 FP32 values, or 4 pairs of 16-bit ones.
template <int KIND> struct Chunk { static constexpr int W = KIND == OUT_F32 ? 8 : 4; uint32_t w[W]; };

// FP32 bits of the largest size among them.
template <int KIND>
__device__ __forceinline__ uint32_t largest(const Chunk<KIND> &c) {
    if constexpr (KIND == OUT_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, c.w[j] & 0x7fffffffu);
        return m;
    } else {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo = max(lo, c.w[j] & 0x7fffu);
            hi = max(hi, c.w[j] & 0x7fff0000u);
        }
        const uint32_t m = max(lo, hi >> 16);
        return KIND == OUT_BF16 ? m << 16 : __builtin_bit_cast(uint32_t, f16_bits_to_f32((uint16_t)m));
    }
}

// The codes of 8 elements, element j in nibble j.
template <int KIND>
__device__ __forceinline__ uint32_t codes(const Chunk<KIND> &c, float scale) {
    uint32_t q = 0;
    if constexpr (KIND == OUT_F32) {
#define DG_PAIR(j) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __builtin_bit_cast(float, c.w[2 * j]), __builtin_bit_cast(float, c.w[2 * j + 1]), scale, j)
        DG_PAIR(0); DG_PAIR(1); DG_PAIR(2); DG_PAIR(3);
#undef DG_PAIR
    } else if constexpr (KIND == OUT_F16) {
#define DG_PAIR(j) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, c.w[j]), scale, j)
        DG_PAIR(0); DG_PAIR(1); DG_PAIR(2); DG_PAIR(3);
#undef DG_PAIR
    } else {
#define DG_PAIR(j) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, c.w[j]), scale, j)
        DG_PAIR(0); DG_PAIR(1); DG_PAIR(2); DG_PAIR(3);
#undef DG_PAIR
    }
    return q;
}

template <int KIND>
__device__ __forceinline__ void set(Chunk<KIND> &c, int j, const char *p) {
    if constexpr (KIND == OUT_F32) c.w[j] = *reinterpret_cast<const uint32_t *>(p);
    else c.w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p) << (16 * (j & 1));
}

// Elements [0, left) of the chunk at p, zeros after them.
template <int KIND>
__device__ __forceinline__ Chunk<KIND> load(const char *p, int left) {
    Chunk<KIND> c;
    if (left >= 8) {
#pragma unroll
        for (int h = 0; h < Chunk<KIND>::W / 4; ++h) {
            const u32x4 v = *reinterpret_cast<const u32x4_any *>(p + 16 * h);
#pragma unroll
            for (int j = 0; j < 4; ++j) c.w[4 * h + j] = v[j];
        }
        return c;
    }
#pragma unroll
    for (int j = 0; j < Chunk<KIND>::W; ++j) c.w[j] = 0u;
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < left) set<KIND>(c, j, p + j * esize(KIND));
    return c;
}

// Chunk `rest` of a row at most a run of MX4_RUN * 256 behind chunk 0 of a row: the rows
// to go on, and the chunk of that row.  Quotients by a reciprocal where a row has fewer
// than 4096 chunks (rest < 8192: exact), else they are 0 or 1.
__device__ __forceinline__ int rows_in(int rest, int chunks, uint32_t mul) {
    if (chunks >= 4096) return rest >= chunks ? 1 : 0;
    return (int)__umulhi((uint32_t)rest, mul);
}
__device__ __forceinline__ void next_matrix(int &row, int &e, int M) {
    if (row < M) return;
    const int d = row / M;
    row -= d * M;
    e += d;
}

// The first chunk of this workgroup: matrix, row and chunk of the row.
__device__ __forceinline__ void first_chunk(int64_t at, int M, int chunks, int &e, int &row, int &c) {
    const int64_t r = at / chunks;
    c = (int)(at - r * chunks);
    e = (int)(r / M);
    row = (int)(r - (int64_t)e * M);
}

// Rows of X contiguous: a thread holds RUN chunks of 8 elements, 4 adjacent lanes a
// block.
template <int KIND, int RUN>
__global__ void __launch_bounds__(256) mx4_quant_rows(Mx4QuantArgs a) {
    int e0, row0, c0;
    first_chunk((int64_t)blockIdx.x * (256 * RUN), a.M, a.chunks, e0, row0, c0);
    Chunk<KIND> x[RUN];
    int e[RUN], row[RUN], c[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        const int rest = c0 + u * 256 + (int)threadIdx.x, down = rows_in(rest, a.chunks, a.chunk_mul);
        c[u] = rest - down * a.chunks;
        row[u] = row0 + down;
        e[u] = e0;
        next_matrix(row[u], e[u], a.M);
        const int left = e[u] < a.E ? a.K - 8 * c[u] : 0;
        x[u] = load<KIND>(a.X + (int64_t)e[u] * a.x_es + (int64_t)row[u] * a.x_rs + (int64_t)c[u] * (8 * esize(KIND)), left);
    }
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        uint32_t top = largest<KIND>(x[u]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const uint32_t b = scale_byte(top, a.ceil);
        const int left = e[u] < a.E ? a.K - 8 * c[u] : 0;
        const uint32_t q = b == 255u ? 0u : codes<KIND>(x[u], power(b));
        if (left <= 0) continue;
        char *to = a.Q + (int64_t)e[u] * a.q_es + (int64_t)row[u] * a.q_rs + 4 * (int64_t)c[u];
        if (left >= 7) {
            *reinterpret_cast<u32_any *>(to) = q;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (2 * j < left) to[j] = (char)(q >> (8 * j));
        }
        if ((c[u] & 3) == 0)
            a.S[(int64_t)e[u] * a.s_es + (int64_t)row[u] * a.s_rs + (int64_t)(c[u] >> 2) * a.s_cs] = (char)b;
    }
}

// Any other X: a workgroup takes 256 rows x MX4_TILE_K elements of K, a lane 4 adjacent rows,
// wave w block w.  Where X's columns are contiguous (a transpose) a lane's 4
// elements are one load, a wave's 512 or 1024 bytes.  Codes and scales leave through LDS,
// 128 contiguous bytes of codes a row.
template <int KIND, bool VEC>
__global__ void __launch_bounds__(2 * MX4_TILE_K) mx4_quant_columns(Mx4QuantArgs a) {
    constexpr int NT = 2 * MX4_TILE_K, BLOCKS = MX4_TILE_K / 32;   // a wave for every block of a row
    constexpr int PITCH = MX4_TILE_K / 2 + 16;     // (a lane's rows are 4 apart, 16 words on the banks: the codes' way in conflicts)
    __shared__ __attribute__((aligned(16))) char lq[MX4_TILE_M * PITCH];
    __shared__ uint8_t ls[MX4_TILE_M * BLOCKS];    // [row][block]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = blockIdx.x / (a.tiles_m * a.tiles_k), t = blockIdx.x - e * (a.tiles_m * a.tiles_k);
    const int tk = t / a.tiles_m, m0 = (t - tk * a.tiles_m) * MX4_TILE_M, k0 = tk * MX4_TILE_K;
    const int m = m0 + 4 * lane, kb = k0 + 32 * wave;
    const int rows = min(a.M - m, 4), left = min(a.K - kb, 32);   // of this lane, of this wave
    const char *src = a.X + (int64_t)e * a.x_es + (int64_t)m * a.x_rs + (int64_t)kb * a.x_cs;
    if (left > 0) {
        // w[j]: elements kb + 2 j, 2 j + 1 of a row for 16 bits, kb + j for 32
        constexpr int W = KIND == OUT_F32 ? 32 : 16;
        uint32_t w[4][W];
        if (VEC && rows == 4) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const char *p = src + (int64_t)min(k, left - 1) * a.x_cs;   // (past K: cleared below)
                if constexpr (KIND == OUT_F32) {
                    const u32x4 v = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[r][k] = v[r];
                } else {
                    const u32x2 v = *reinterpret_cast<const u32x2_any *>(p);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t h = r & 1 ? v[r >> 1] >> 16 : v[r >> 1] & 0xffffu;
                        if (k & 1) w[r][k >> 1] |= h << 16;
                        else w[r][k >> 1] = h;
                    }
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const char *p = src + (int64_t)max(min(r, rows - 1), 0) * a.x_rs + (int64_t)min(k, left - 1) * a.x_cs;
                    uint32_t h = 0;
                    if (rows > 0) h = KIND == OUT_F32 ? *reinterpret_cast<const uint32_t *>(p) : *reinterpret_cast<const uint16_t *>(p);
                    if (KIND == OUT_F32) w[r][k] = h;
                    else if (k & 1) w[r][k >> 1] |= h << 16;
                    else w[r][k >> 1] = h;
                }
        }
        if (left < 32) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (k >= left) {
                        if (KIND == OUT_F32) w[r][k] = 0u;
                        else w[r][k >> 1] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
                    }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            uint32_t top = 0;
            Chunk<KIND> c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < W / 4; ++j) c[i].w[j] = w[r][i * (W / 4) + j];
                top = max(top, largest<KIND>(c[i]));
            }
            const uint32_t b = scale_byte(top, a.ceil);
            u32x4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = b == 255u ? 0u : codes<KIND>(c[i], power(b));
            *reinterpret_cast<u32x4 *>(lq + (4 * lane + r) * PITCH + 16 * wave) = q;
            ls[(4 * lane + r) * BLOCKS + wave] = (uint8_t)b;
        }
    }
    __syncthreads();
    const int bytes = (a.K + 1) / 2 - k0 / 2;      // of a row, from this tile on
    char *q = a.Q + (int64_t)e * a.q_es + (int64_t)m0 * a.q_rs + k0 / 2;
#pragma unroll
    for (int i = tid; i < MX4_TILE_M * BLOCKS; i += NT) {
        const int r = i / BLOCKS, at = 16 * (i % BLOCKS), n = min(bytes - at, 16);
        if (m0 + r >= a.M || n <= 0) continue;
        const char *from = lq + r * PITCH + at;
        char *to = q + (int64_t)r * a.q_rs + at;
        if (n == 16) {
            *reinterpret_cast<u32x4_any *>(to) = *reinterpret_cast<const u32x4 *>(from);
        } else {
            for (int j = 0; j < n; ++j) to[j] = from[j];
        }
    }
    const int blocks = min((a.K + 31) / 32 - k0 / 32, BLOCKS);
    char *s = a.S + (int64_t)e * a.s_es + (int64_t)m0 * a.s_rs + (int64_t)(k0 / 32) * a.s_cs;
    for (int i = tid; i < MX4_TILE_M * BLOCKS; i += NT) {
        const int r = i / BLOCKS, j = i % BLOCKS;
        if (m0 + r < a.M && j < blocks) s[(int64_t)r * a.s_rs + (int64_t)j * a.s_cs] = (char)ls[i];
    }
}

// A thread holds RUN words of 8 codes.
template <int KIND, int RUN>
__global__ void __launch_bounds__(256) mx4_dequant(Mx4DequantArgs a) {
    int e0, row0, c0;
    first_chunk((int64_t)blockIdx.x * (256 * RUN), a.M, a.chunks, e0, row0, c0);
    uint32_t q[RUN], b[RUN];
    int e[RUN], row[RUN], c[RUN], left[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        const int rest = c0 + u * 256 + (int)threadIdx.x, down = rows_in(rest, a.chunks, a.chunk_mul);
        c[u] = rest - down * a.chunks;
        row[u] = row0 + down;
        e[u] = e0;
        next_matrix(row[u], e[u], a.M);
        left[u] = e[u] < a.E ? a.K - 8 * c[u] : 0;
        const char *p = a.Q + (int64_t)e[u] * a.q_es + (int64_t)row[u] * a.q_rs + 4 * (int64_t)c[u];
        q[u] = b[u] = 0u;
        if (left[u] >= 7) {
            q[u] = *reinterpret_cast<const u32_any *>(p);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (2 * j < left[u]) q[u] |= (uint32_t)(uint8_t)p[j] << (8 * j);
        }
        if (left[u] > 0)
            b[u] = (uint8_t)a.S[(int64_t)e[u] * a.s_es + (int64_t)row[u] * a.s_rs + (int64_t)(c[u] >> 2) * a.s_cs];
    }
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        if (left[u] <= 0) continue;
        // NaN where b is 255; codes and powers of two have at most 3 significant bits:
        // exact in FP32, and in BF16 and FP16 within their range
        const float s = b[u] == 255u ? __builtin_bit_cast(float, 0x7fc00000u) : power(b[u]);
        float v[8];
#define DG_PAIR(j)                                                                     \
    do {                                                                               \
        const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, j);          \
        v[2 * j] = p[0];                                                               \
        v[2 * j + 1] = p[1];                                                           \
    } while (0)
        DG_PAIR(0); DG_PAIR(1); DG_PAIR(2); DG_PAIR(3);
#undef DG_PAIR
        char *to = a.Y + (int64_t)e[u] * a.y_es + (int64_t)row[u] * a.y_rs + 8 * (int64_t)c[u] * a.y_cs;
        if (a.vec && left[u] >= 8) {
            if constexpr (KIND == OUT_F32) {
                *reinterpret_cast<f32x4_any *>(to) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4_any *>(to + 16) = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = KIND == OUT_BF16 ? f32_to_bf16_bits(v[2 * j]) | (uint32_t)f32_to_bf16_bits(v[2 * j + 1]) << 16
                                            : f32_to_f16_bits(v[2 * j]) | (uint32_t)f32_to_f16_bits(v[2 * j + 1]) << 16;
                *reinterpret_cast<u32x4_any *>(to) = w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left[u]) store_out(to + j * a.y_cs, KIND, v[j]);
        }
    }
}

}  // namespace

hipError_t launch_mx4_quant(bool by_columns, const Mx4QuantArgs &a, int64_t units, hipStream_t s) {
    const dim3 grid((unsigned)units);
#define DG_KIND(kind)                                                                                        \
    do {                                                                                                     \
        if (!by_columns && a.run == 1) hipLaunchKernelGGL((mx4_quant_rows<kind, 1>), grid, dim3(256), 0, s, a); \
        else if (!by_columns) hipLaunchKernelGGL((mx4_quant_rows<kind, MX4_RUN>), grid, dim3(256), 0, s, a); \
        else if (a.vec) hipLaunchKernelGGL((mx4_quant_columns<kind, true>), grid, dim3(2 * MX4_TILE_K), 0, s, a);       \
        else hipLaunchKernelGGL((mx4_quant_columns<kind, false>), grid, dim3(2 * MX4_TILE_K), 0, s, a);                 \
    } while (0)
    if (a.x_kind == OUT_F32) DG_KIND(OUT_F32);
    else if (a.x_kind == OUT_F16) DG_KIND(OUT_F16);
    else DG_KIND(OUT_BF16);
#undef DG_KIND
    return hipGetLastError();
}

hipError_t launch_mx4_dequant(const Mx4DequantArgs &a, int64_t units, hipStream_t s) {
    const dim3 grid((unsigned)units);
#define DG_KIND(kind)                                                                                        \
    do {                                                                                                     \
        if (a.run == 1) hipLaunchKernelGGL((mx4_dequant<kind, 1>), grid, dim3(256), 0, s, a);                \
        else hipLaunchKernelGGL((mx4_dequant<kind, MX4_RUN>), grid, dim3(256), 0, s, a);                     \
    } while (0)
    if (a.y_kind == OUT_F32) DG_KIND(OUT_F32);
    else if (a.y_kind == OUT_F16) DG_KIND(OUT_F16);
    else DG_KIND(OUT_BF16);
#undef DG_KIND
    return hipGetLastError();
}

}  // namespace dg
