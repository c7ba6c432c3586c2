// moe_gemm.hpp -- the experts' products for gfx950 (templates; instantiated per
// input type by moe_gemm_{f16,bf16}.hip).
//
//   forward: C[r] = act(A[r] . W[e])         for offsets[e] <= r < offsets[e + 1]
//   wgrad  : dW[e] = sum of A[r]^T D[r]      over the same rows
//
// The row counts live in device memory (the router's choices of this step), so
// the host cannot cut the work into tiles.  Forward: every wave scans the
// offsets itself, gives each expert ceil(rows / BM) rows of tiles, and finds
// the expert and tile of its workgroup; the grid is an upper bound of the tile
// count and the workgroups past the real count leave at once.  Weight gradient:
// the tiles are known (E matrices of K x N), only the summed rows vary.
//
// Two kernels share this mapping.  The direct-to-LDS kernel is the library's
// dense one (gemm_dtl.hpp) on the expert's part of the operands.  The
// register-staged kernel below serves rows at any alignment (16-byte loads) and
// any strides (element loads).
//
// Many rows are bound by the dense kernel's rate (8 experts, 16384 rows, 4096 ->
// 14336 BF16: 1.73 ms, 1.1 PFLOP/s; its weight gradient over 4096 x 4096 FP32: 312
// us, 0.88 PFLOP/s, the tiles' ends included), few rows by the weights' bytes (32
// rows of them: 160 to 178 us, 5.3 to 5.9 TB/s).
#pragma once
#include "gemm_dtl.hpp"
#include "moe.hpp"
#include "moe_slot.hpp"

namespace dg {
namespace moe {

// The product of this workgroup's expert: p's pointers and extents, and the
// tile.  False: nothing to do.
// Split K (a.p.splits pieces a tile): a tile's pieces are units of their own,
// one after another; p's sums and counters become the expert's.
template <int BM, int BN, bool WGRAD, bool SPLIT>
__device__ __forceinline__ bool expert_product(const MoeArgs &a, MfmaArgs &p, int &t) {
    constexpr int KEL = dtl::KB / 2;
    p = a.p;
    const int S = SPLIT ? a.p.splits : 1;
    int before;                              // tiles of the experts before
    if constexpr (WGRAD) {
        // The experts in turn, each one's tiles dealt over all XCDs: experts
        // differ in rows, and a run of whole experts per XCD would leave the
        // XCD with the longest ones working alone (8 experts of 500 to 1900
        // rows, 4096 x 4096 FP32: 492 us that way, 310 us this way).
        const int tiles = a.p.tiles_m * a.p.tiles_n, e = blockIdx.x / (tiles * S);
        int begin, rows;
        group_rows(a.offsets, a.o_s, a.E, a.n, e, begin, rows);
        begin = __builtin_amdgcn_readfirstlane(begin);
        rows = __builtin_amdgcn_readfirstlane(rows);
        t = xcd_run(blockIdx.x - e * tiles * S, tiles * S);
        before = e * tiles;
        p.a.ptr += (int64_t)begin * p.a.k_stride;
        p.b.ptr += (int64_t)begin * p.b.k_stride;
        p.epi.C += (int64_t)e * a.e_cs;
        p.K = rows;
        p.ktiles = (rows + KEL - 1) / KEL;
    } else {
        Slot s;
        if (!find_slot<BM>(a.offsets, a.o_s, a.E, a.n, a.p.tiles_n * S, a.units, blockIdx.x, s)) return false;
        before = s.above * a.p.tiles_n;
        p.a.ptr += (int64_t)s.begin * p.a.r_stride;
        p.epi.C += (int64_t)s.begin * p.epi.c_rs;
        p.M = s.rows;
        p.tiles_m = (s.rows + BM - 1) / BM;
        t = s.unit;
        if (s.e < a.E) p.b.ptr += (int64_t)s.e * a.e_bs;
        else p.K = p.ktiles = 0;             // rows of no expert: zero (every activation keeps 0)
    }
    if constexpr (SPLIT) {
        p.kt_per_split = (p.ktiles + S - 1) / S;
        p.ws += (int64_t)before * S * (BM * BN);
        p.counters += before;
    }
    return true;
}

template <int IN, int BM, int BN, int WGM, int WGN, int NS, int AMODE, int BMODE, int NL, bool WGRAD, bool SPLIT>
__global__ void __launch_bounds__(64 * WGM * WGN) moe_dtl(MoeArgs a) {
    MfmaArgs p;
    int t;
    if (!expert_product<BM, BN, WGRAD, SPLIT>(a, p, t)) return;
    dtl::mfma_dtl_body<IN, BM, BN, WGM, WGN, NS, AMODE, BMODE, SPLIT, NL, false, true>(p, t);
}

// ------------------------------------------------------------------ register-staged kernel

typedef uint32_t u32x4_h __attribute__((ext_vector_type(4), aligned(2)));

// The 128 bits of v moved down by `by` 16-bit elements (0 to 8), zeros above.
__device__ __forceinline__ u32x4 down_elements(u32x4 v, int by) {
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    if (by >= 4) {
        lo = by >= 8 ? 0 : hi >> (16 * (by - 4));
        hi = 0;
    } else if (by > 0) {
        lo = lo >> (16 * by) | hi << (64 - 16 * by);
        hi >>= 16 * by;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// One operand's K tile (R rows x 64 elements) through registers: chunks of 8
// elements, contiguous along K (KMAJ) or along the rows (MNMAJ).
template <int MODE, int R, int LOAD, int NT>
struct RegIO {
    static constexpr int NCH = R * 8 / NT, CPR = R / 8;
    static_assert(R * 8 % NT == 0, "whole chunks per thread");

    __device__ static void load(u32x4 (&reg)[NCH], const Operand &op, int r0, int k0, int Rlim, int Klim, int tid) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * NT;
            const int r = r0 + (MODE == KMAJ ? c >> 3 : (c % CPR) * 8), k = k0 + (MODE == KMAJ ? (c & 7) * 8 : c / CPR);
            if constexpr (LOAD == MOE_VEC) {
                // A chunk that crosses the end of its row is read whole, ending
                // there, and moved down; rows of C it adds are never stored, K
                // elements past the end are zero.
                const int cr = min(r, MODE == KMAJ ? Rlim - 1 : Rlim - 8), ck = min(k, MODE == KMAJ ? Klim - 8 : Klim - 1);
                const u32x4 v = *reinterpret_cast<const u32x4_h *>(op.ptr + (int64_t)cr * op.r_stride + (int64_t)ck * op.k_stride);
                reg[i] = v;
            } else {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int rr = MODE == KMAJ ? r : r + e, kk = MODE == KMAJ ? k + e : k;
                    if (rr < Rlim && kk < Klim)
                        w[e >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(
                                         op.ptr + (int64_t)rr * op.r_stride + (int64_t)kk * op.k_stride) << (16 * (e & 1));
                }
                reg[i] = u32x4{w[0], w[1], w[2], w[3]};
            }
        }
    }

    // The loaded chunks of a tile that reaches past an end (VEC): see load.
    __device__ static void trim(u32x4 (&reg)[NCH], int r0, int k0, int Rlim, int Klim, int tid) {
        if (LOAD != MOE_VEC || (k0 + 64 <= Klim && (MODE == KMAJ || r0 + R <= Rlim))) return;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * NT;
            const int r = r0 + (MODE == KMAJ ? c >> 3 : (c % CPR) * 8), k = k0 + (MODE == KMAJ ? (c & 7) * 8 : c / CPR);
            if (MODE == KMAJ) reg[i] = down_elements(reg[i], min(k - min(k, Klim - 8), 8));
            else reg[i] = k < Klim ? down_elements(reg[i], min(r - min(r, Rlim - 8), 8)) : u32x4{0u, 0u, 0u, 0u};
        }
    }

    __device__ static void store(char *lds, const u32x4 (&reg)[NCH], int tid) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * NT;
            const int off = MODE == KMAJ ? dtl::kmaj_off(c >> 3, c & 7) : dtl::mnmaj_off<2, R>(c / CPR, c % CPR);
            *reinterpret_cast<u32x4 *>(lds + off) = reg[i];
        }
    }
};

// B x B tiles, 4 waves (2 x 2), a two-stage LDS ring: the next tile's loads are
// in flight while the current one is multiplied.  SPLIT: a piece of K, whose sums
// the tile's last piece adds in the order of K, as in the dense kernels.
template <int IN, int B, int AMODE, int BMODE, int LOAD, bool WGRAD, bool SPLIT>
__global__ void __launch_bounds__(256) moe_reg(MoeArgs a) {
    constexpr int NT = 256, T = B / 32, STAGE = 2 * B * dtl::KB, KEL = 64;
    using AIO = RegIO<AMODE, B, LOAD, NT>;
    using BIO = RegIO<BMODE, B, LOAD, NT>;
    __shared__ __attribute__((aligned(16))) char ring[2 * STAGE];
    MfmaArgs p;
    int t;
    if (!expert_product<B, B, WGRAD, SPLIT>(a, p, t)) return;
    const int S = SPLIT ? p.splits : 1, piece = t, z = SPLIT ? t % S : 0;
    t /= S;
    const int kt0 = SPLIT ? z * p.kt_per_split : 0, kt1 = SPLIT ? min(kt0 + p.kt_per_split, p.ktiles) : p.ktiles;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    dtl::raster(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int m0 = tm * B, n0 = tn * B;
    f32x4 acc[T][T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 ra[AIO::NCH], rb[BIO::NCH];
    auto fetch = [&](int kt) __attribute__((always_inline)) {
        AIO::load(ra, p.a, m0, kt * KEL, p.M, p.K, tid);
        BIO::load(rb, p.b, n0, kt * KEL, p.N, p.K, tid);
    };
    auto put = [&](char *st, int kt) __attribute__((always_inline)) {
        AIO::trim(ra, m0, kt * KEL, p.M, p.K, tid);
        BIO::trim(rb, n0, kt * KEL, p.N, p.K, tid);
        AIO::store(st, ra, tid);
        BIO::store(st + B * dtl::KB, rb, tid);
    };
    if (kt0 < kt1) {
        fetch(kt0);
        put(ring + (kt0 & 1) * STAGE, kt0);
    }
    __syncthreads();
    for (int kt = kt0; kt < kt1; ++kt) {
        const bool more = kt + 1 < kt1;
        if (more) fetch(kt + 1);
        const char *la = ring + (kt & 1) * STAGE, *lb = la + B * dtl::KB;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u32x4 fa[T], fb[T];
#pragma unroll
            for (int i = 0; i < T; ++i) fa[i] = dtl::frag16<AMODE, B>(la, wm * (B / 2) + 16 * i, ks, lane);
#pragma unroll
            for (int j = 0; j < T; ++j) fb[j] = dtl::frag16<BMODE, B>(lb, wn * (B / 2) + 16 * j, ks, lane);
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j) acc[i][j] = dtl::mfma16<IN>(fb[j], fa[i], acc[i][j]);
        }
        if (more) put(ring + ((kt & 1) ^ 1) * STAGE, kt + 1);
        __syncthreads();
    }
    if constexpr (SPLIT) {
        // [tile][piece][element][thread]: every thread adds its own elements
        __shared__ int is_last;
        float *tile = p.ws + (int64_t)(piece - z) * (B * B) + tid;
        auto at = [&](int q, int i, int j, int e) __attribute__((always_inline)) {
            return tile + (int64_t)q * (B * B) + ((i * T + j) * 4 + e) * NT;
        };
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int j = 0; j < T; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    __hip_atomic_store(at(z, i, j, e), acc[i][j][e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) is_last = take_last_ticket(p.counters + t, S);
        __syncthreads();
        if (!is_last) return;
#pragma unroll 1
        for (int q = 0; q < S; ++q) {
            f32x4 v[T][T];
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][j][e] = __hip_atomic_load(at(q, i, j, e), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j) acc[i][j] = q == 0 ? v[i][j] : acc[i][j] + v[i][j];
        }
        if (tid == 0) __hip_atomic_store(p.counters + t, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // a lane holds row lane % 16 and 4 adjacent columns of each 16 x 16 block
    const Epilogue &ep = p.epi;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int m = m0 + wm * (B / 2) + 16 * i + (lane & 15);
        if (m >= p.M) continue;
        char *row = ep.C + (int64_t)m * ep.c_rs;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int n = n0 + wn * (B / 2) + 16 * j + 4 * (lane >> 4);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activate(ep.act, acc[i][j][e]);
            if (ep.vec4 && n + 3 < p.N) {
                store_out4(row + (int64_t)n * ep.c_cs, ep.out_kind, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) store_out(row + (int64_t)(n + e) * ep.c_cs, ep.out_kind, v[e]);
            }
        }
    }
}

// ------------------------------------------------------------------ dispatch

#define DG_MOE_LAUNCH(kernel, threads) \
    hipLaunchKernelGGL(kernel, dim3((unsigned)units), dim3(threads), 0, s, a)

// Direct loads: A's rows are K-contiguous and B either way (forward), or both
// operands M/N-contiguous (wgrad).  The tiles are the dense kernel's, plus 32 x
// 128 for a few rows per expert.
// The host counts the tiles by the same tile: one that a direction does not
// have (or not split) is an error, never another kernel.
template <int IN, int BMODE, bool WGRAD, bool SPLIT>
hipError_t launch_dtl(int tile, const MoeArgs &a, int64_t units, hipStream_t s) {
    constexpr int AMODE = WGRAD ? MNMAJ : KMAJ;
    if (tile == T128x128) {
        DG_MOE_LAUNCH((moe_dtl<IN, 128, 128, 2, 2, 2, AMODE, BMODE, 0, WGRAD, SPLIT>), 256);
        return hipGetLastError();
    }
    if constexpr (!WGRAD) {
        if (tile == T64x128) {
            DG_MOE_LAUNCH((moe_dtl<IN, 32, 128, 1, 4, 7, AMODE, BMODE, 0, WGRAD, SPLIT>), 256);
            return hipGetLastError();
        }
    }
    if constexpr (!SPLIT) {
        if (tile == T256x256) {
            DG_MOE_LAUNCH((moe_dtl<IN, 256, 256, 2, 4, 2, AMODE, BMODE, 4, WGRAD, SPLIT>), 512);
            return hipGetLastError();
        }
    }
    if constexpr (!SPLIT && !WGRAD) {
        if (tile == MOE_T192) {
            DG_MOE_LAUNCH((moe_dtl<IN, 192, 256, 2, 4, 2, AMODE, BMODE, 4, WGRAD, SPLIT>), 512);
            return hipGetLastError();
        }
    }
    return hipErrorInvalidValue;
}

// any strides (MOE_ELEM): the element loads make every operand K-contiguous in LDS
template <int IN, int LOAD, int B, bool SPLIT>
hipError_t launch_reg(int b_mode, bool wgrad, const MoeArgs &a, int64_t units, hipStream_t s) {
    constexpr int MN = LOAD == MOE_ELEM ? KMAJ : MNMAJ;
    if (wgrad) DG_MOE_LAUNCH((moe_reg<IN, B, MN, MN, LOAD, true, SPLIT>), 256);
    else if (LOAD == MOE_ELEM || b_mode == KMAJ) DG_MOE_LAUNCH((moe_reg<IN, B, KMAJ, KMAJ, LOAD, false, SPLIT>), 256);
    else DG_MOE_LAUNCH((moe_reg<IN, B, KMAJ, MN, LOAD, false, SPLIT>), 256);
    return hipGetLastError();
}

template <int IN, bool SPLIT>
hipError_t launch_s(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units, hipStream_t s) {
    if (load == MOE_DTL && wgrad) return launch_dtl<IN, MNMAJ, true, SPLIT>(tile, a, units, s);
    if (load == MOE_DTL && b_mode == KMAJ) return launch_dtl<IN, KMAJ, false, SPLIT>(tile, a, units, s);
    if (load == MOE_DTL) return launch_dtl<IN, MNMAJ, false, SPLIT>(tile, a, units, s);
    if constexpr (!SPLIT) {
        if (load == MOE_VEC && tile == T128x128) return launch_reg<IN, MOE_VEC, 128, SPLIT>(b_mode, wgrad, a, units, s);
    }
    if (load == MOE_VEC && tile == T64x64) return launch_reg<IN, MOE_VEC, 64, SPLIT>(b_mode, wgrad, a, units, s);
    if (load == MOE_ELEM && tile == T64x64) return launch_reg<IN, MOE_ELEM, 64, SPLIT>(b_mode, wgrad, a, units, s);
    return hipErrorInvalidValue;
}

template <int IN>
hipError_t launch(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units, hipStream_t s) {
    return a.p.splits > 1 ? launch_s<IN, true>(load, tile, b_mode, wgrad, a, units, s)
                          : launch_s<IN, false>(load, tile, b_mode, wgrad, a, units, s);
}
#undef DG_MOE_LAUNCH

}  // namespace moe
}  // namespace dg
