// mx4_tile.hpp -- what the kernels of the MXFP4 products share: the matrix instruction, a
// workgroup's part of the product, and the store of its tile.
#pragma once
#include <type_traits>

#include "device_common.hpp"
#include "gemm_dtl.hpp"
#include "moe_slot.hpp"
#include "mx4.hpp"

namespace dg {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_half __attribute__((ext_vector_type(4), aligned(2)));

// One block column of the matrix cores: 64 elements of K (two blocks, of the lanes below
// 32 and of the others), scale byte STEP of each lane's word.
template <int STEP>
__device__ __forceinline__ f32x16 mx4_mfma(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 c) {
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}, y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, STEP, (int)sa, STEP, (int)sb);
}

// This workgroup's expert, its rows, and the tile.  live: false for the rows of no expert,
// which are zero.
struct Mx4Part { int e, begin, M, m0, n0, t, z, live; };

// False: nothing to do.
template <int BM, int BN, bool SPLIT = false>
__device__ __forceinline__ bool mx4_part(const Mx4GemmArgs &a, Mx4Part &p) {
    p.e = 0; p.begin = 0; p.M = a.M; p.z = 0; p.live = 1;
    if (a.offsets) {
        moe::Slot s;
        if (!moe::find_slot<BM>(a.offsets, a.o_s, a.E, a.M, a.tiles_n, a.units, blockIdx.x, s)) return false;
        p.e = s.e; p.begin = s.begin; p.M = s.rows; p.t = s.unit;
        if (p.e == a.E) p.e = p.live = 0;
    } else {
        p.t = moe::xcd_run(blockIdx.x, a.units);
        if (SPLIT && a.splits > 1) {
            const int u = p.t / a.splits;
            p.z = p.t - u * a.splits;
            p.t = u;
        }
    }
    int tm, tn;
    dtl::raster(p.t, (p.M + BM - 1) / BM, a.tiles_n, a.group_m, tm, tn);
    p.m0 = tm * BM;
    p.n0 = tn * BN;
    return true;
}

// Bytes of LDS that a wave's store takes: 32 rows, 4 words apart on the banks.
template <int TN> constexpr int MX4_STORE_LDS = 32 * (32 * TN + 4) * 4;

// A wave's 32 TM x 32 TN sums at (r0, c0) of the tile: a lane holds row l and 4 adjacent
// columns, four times, of each 32 x 32 block (ROWS: column l and 4 adjacent rows).  32 rows at a time go through the wave's own
// part of LDS, so that 8 adjacent columns leave in one access, whole lines of a row from
// adjacent lanes, and the code for types and edges is there once (stored from where they
// are, the 256 x 256 tile's sums took 10000 instructions).  The caller's waves have all
// left the ring.
template <int TM, int TN, bool ROWS = false>
__device__ __forceinline__ void mx4_store(const Mx4GemmArgs &a, const Mx4Part &p, const f32x16 (&acc)[TM][TN], int r0, int c0, int lane, char *lds) {
    constexpr int PITCH = 32 * TN + 4, CPR = 4 * TN;   // floats of a row, chunks of 8 columns in it
    const int l = lane & 31, h = lane >> 5;
    float *buf = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (ROWS) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) buf[(8 * q + 4 * h + e) * PITCH + 32 * j + l] = acc[i][j][4 * q + e];
                } else {
                    *reinterpret_cast<f32x4 *>(buf + l * PITCH + 32 * j + 8 * q + 4 * h) =
                        f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                }
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int c = lane; c < 32 * CPR; c += 64) {
            const int r = c / CPR, k = c % CPR, m = p.m0 + r0 + 32 * i + r, n = p.n0 + c0 + 8 * k;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = buf[r * PITCH + 8 * k + e];
            if (m >= p.M || n >= a.N) continue;
            if (a.act != ACT_NONE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = activate(a.act, v[e]);
            }
            char *to = a.C + (int64_t)(p.begin + m) * a.c_rs + (int64_t)n * a.c_cs;
            if (a.vec4 && n + 8 <= a.N) {
                if (a.out_kind == OUT_F32) {
                    *reinterpret_cast<f32x4_any *>(to) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4_any *>(to + 16) = f32x4{v[4], v[5], v[6], v[7]};
                } else {
                    u32x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = a.out_kind == OUT_BF16 ? f32_to_bf16_bits(v[2 * e]) | (uint32_t)f32_to_bf16_bits(v[2 * e + 1]) << 16
                                                      : f32_to_f16_bits(v[2 * e]) | (uint32_t)f32_to_f16_bits(v[2 * e + 1]) << 16;
                    *reinterpret_cast<u32x4_half *>(to) = w;
                }
            } else {
#pragma unroll 1
                for (int e = 0; e < 8 && n + e < a.N; ++e) store_out(to + e * a.c_cs, a.out_kind, activate(a.act, buf[r * PITCH + 8 * k + e]));
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the rows have been read
    }
}

}  // namespace dg
