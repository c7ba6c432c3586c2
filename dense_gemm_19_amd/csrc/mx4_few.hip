// mx4_few.hip -- products with MXFP4 weights where few rows meet them, bound by the bytes of
// the codes: every wave streams its part of the weights' rows from memory straight to
// registers, no two waves the same, and all of a wave's loads are in flight before the
// first is used.
//
// A workgroup's 8 waves share 16 NF columns and split K: a unit is 512 elements, 256 bytes
// of a row of codes and 16 of its scales.  Lane (g, n), n = lane % 16, loads of row n the 16
// bytes 64 j + 16 g at each of four steps j, a whole block, and all 16 scale bytes.
// Bytes of codes bound it; what it reaches (BF16 / codes): 1 x 14336 x 4096, 31 MB, 10.1 /
// 8.6 us, 3.6 TB/s with a launch of 1.5 in it; 16 x 4096 x 14336 14.8 / 11.3 us.
//   A in codes: those are the operands of v_mfma_scale_f32_16x16x128_f8f6f4 as they lie.
//   A in 16 bits: the lanes of a row first exchange words (a 4 x 4 transpose in four
//   instructions), so that an instruction of 32 elements meets one block of every row.
//   BF16 weights are converted times their scale, exactly; FP16 does not hold every
//   scale, so its codes are converted as they are and a block's sum, in FP32, is added
//   times its scale.
#include <algorithm>

#include "bytes.hpp"
#include "device_common.hpp"
#include "gemm_dtl.hpp"
#include "moe_slot.hpp"
#include "mx4_tile.hpp"

namespace dg {
namespace {

constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int UNIT = 256;        // bytes of a row of codes
constexpr int CODES = MX4_CODES;   // beside IN_F16, IN_BF16

template <int N> using Int = std::integral_constant<int, N>;

// 16 bytes from `at` on of a row of `bytes`, zeros past its end.
__device__ __forceinline__ u32x4 row_piece(const char *row, int at, int bytes) {
    const int n = bytes - at;
    if (n >= 16) return *reinterpret_cast<const u32x4_any *>(row + at);
    if (n <= 0) return u32x4{0u, 0u, 0u, 0u};
    if (bytes >= 16) return down_bytes(*reinterpret_cast<const u32x4_any *>(row + bytes - 16), 16 - n);
    return load_part<1>(row + at, 1, n);
}

// words[i] of lane row g <- words[g] of lane row i (lane rows of 16 lanes)
__device__ __forceinline__ u32x4 exchange(u32x4 v) {
    auto s0 = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto s1 = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto t0 = __builtin_amdgcn_permlane16_swap(s0[0], s1[0], false, false);
    auto t1 = __builtin_amdgcn_permlane16_swap(s0[1], s1[1], false, false);
    return u32x4{t0[0], t0[1], t1[0], t1[1]};
}

__device__ __forceinline__ float power(uint32_t b) {   // 2^(b - 127); 0: subnormal, 255: NaN
    return __builtin_bit_cast(float, max(b << 23, 0x00400000u) | (b == 255u ? 0x00400000u : 0u));
}

// 8 codes as 16-bit numbers, times the power of two in the exponent bits of s (the
// conversion reads no others: 0 is 2^-127, all ones NaN).
template <int IN>
__device__ __forceinline__ u32x4 decode(uint32_t q, float s) {
    u32x4 v;
#define DG_PAIR(j)                                                                                                          \
    if constexpr (IN == IN_BF16) v[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, j));   \
    else v[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, j));
    DG_PAIR(0) DG_PAIR(1) DG_PAIR(2) DG_PAIR(3)
#undef DG_PAIR
    return v;
}

// STAGED (16-bit A at aligned words): a wave brings its units of A to LDS by loads of whole
// rows, 1 KB each, and reads fragments there: straight to registers a fragment takes as
// much of the way from the cache whether its 16 rows differ or not (1 x 14336 x 4096: 11.6
// us, staged 10.1).
template <int KIND, int TM, int NF, bool STAGED>
__global__ void __launch_bounds__(NT) mx4_few(Mx4GemmArgs a) {
    constexpr int MR = 16 * TM, NC = 16 * NF, REGS = TM * NF * 256, PER = (REGS + NT - 1) / NT;
    constexpr int AP = KIND == CODES ? 4 : 16;     // 16-byte pieces of A in a unit, of a lane
    extern __shared__ __attribute__((aligned(16))) char lds[];   // the waves' sums; STAGED before: [wave][row] 1 KB of A
    float *red = reinterpret_cast<float *>(lds);
    __shared__ int is_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;

    int e = 0, begin = 0, M = a.M, unit, z = 0, units = (a.row_bytes + UNIT - 1) / UNIT;
    if (a.offsets) {
        moe::Slot s;
        if (!moe::find_slot<MR>(a.offsets, a.o_s, a.E, a.M, a.tiles_n, a.units, blockIdx.x, s)) return;
        e = s.e; begin = s.begin; M = s.rows; unit = s.unit;
        if (e == a.E) e = units = 0;               // rows of no expert: zero
    } else {
        unit = moe::xcd_run(blockIdx.x, a.units);
        if (a.splits > 1) {
            const int u = unit / a.splits;
            z = unit - u * a.splits;
            unit = u;
        }
    }
    const int tiles_m = (M + MR - 1) / MR, tn = unit / tiles_m, m0 = (unit - tn * tiles_m) * MR, n0 = tn * NC;
    const int u0 = z * a.kt_per_split, u1 = min(u0 + a.kt_per_split, units);   // (whole: kt_per_split is all)

    const char *wrow[NF], *srow[NF], *arow[TM], *sarow[TM];
#pragma unroll
    for (int f = 0; f < NF; ++f) {                 // rows past the end: the last one (not stored)
        const int64_t r = min(n0 + 16 * f + n, a.N - 1);
        wrow[f] = a.Q + (int64_t)e * a.q_es + r * a.q_rs;
        srow[f] = a.S + (int64_t)e * a.s_es + r * a.s_rs;
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int64_t r = begin + min(m0 + 16 * t + n, M - 1);
        arow[t] = a.A + r * a.a_rs;
        if (KIND == CODES) sarow[t] = a.SA + r * a.sa_rs;
    }

    f32x4 acc[TM][NF];
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[t][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto one = [&](auto wholec, int u) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(wholec)::value;
        constexpr bool LDS_A = STAGED && WHOLE;
        u32x4 w[NF][4], s[NF], x[TM][LDS_A ? 1 : AP], sx[TM];
        char *own = lds + wave * (a.a_rows * 1024);
        if constexpr (LDS_A) {
            // chunk c of row r at c ^ r, so that 16 rows' reads fall on distinct banks
            const uint32_t to = dtl::lds_addr(own);
            const char *base = a.A + (int64_t)(begin + m0) * a.a_rs + u * (4 * UNIT);
#pragma unroll 1
            for (int r = 0; r < min(M - m0, MR); ++r) dtl::lds_load16(base + r * a.a_rs, 16 * (lane ^ r), to + r * 1024);
        }
        auto piece = [&](const char *row, int at, int bytes) __attribute__((always_inline)) {
            return WHOLE ? *reinterpret_cast<const u32x4_any *>(row + at) : row_piece(row, at, bytes);
        };
        auto scales = [&](const char *row, int64_t cs) __attribute__((always_inline)) {
            return WHOLE ? *reinterpret_cast<const u32x4_any *>(row + 16 * u) : load_part<1>(row + 16 * u * cs, cs, min(a.blocks - 16 * u, 16));
        };
        // all loads at once, in the order of use
#pragma unroll
        for (int f = 0; f < NF; ++f) s[f] = scales(srow[f], a.s_cs);
        if constexpr (KIND == CODES) {
#pragma unroll
            for (int t = 0; t < TM; ++t) sx[t] = scales(sarow[t], a.sa_cs);
        }
        const int at = u * UNIT + 16 * g, x_at = KIND == CODES ? at : u * (4 * UNIT) + 16 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int f = 0; f < NF; ++f) w[f][j] = piece(wrow[f], at + 64 * j, a.row_bytes);
            if constexpr (!LDS_A) {
#pragma unroll
                for (int t = 0; t < TM; ++t)
#pragma unroll
                    for (int i = j * (AP / 4); i < (j + 1) * (AP / 4); ++i) x[t][i] = piece(arow[t], x_at + 64 * i, KIND == CODES ? a.row_bytes : 2 * a.K);
            }
        }
        if constexpr (LDS_A) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(5 * NF) : "memory");   // A, but not the codes
        else __builtin_amdgcn_sched_barrier(0);
        const int row = min(n, M - m0 - 1);
        auto fragment = [&](int t, int i) __attribute__((always_inline)) {
            if constexpr (LDS_A) return *reinterpret_cast<const u32x4 *>(own + row * 1024 + 16 * ((4 * i + g) ^ row));
            else return x[t][i];
        };
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                if constexpr (KIND == CODES) {
                    const i32x8 y = {(int)w[f][j][0], (int)w[f][j][1], (int)w[f][j][2], (int)w[f][j][3], 0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < TM; ++t) {
                        const i32x8 v = {(int)x[t][j][0], (int)x[t][j][1], (int)x[t][j][2], (int)x[t][j][3], 0, 0, 0, 0};
                        acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, y, acc[t][f], 4, 4, 0, (int)(sx[t][j] >> (8 * g)), 0, (int)(s[f][j] >> (8 * g)));
                    }
                } else {
                    const u32x4 q = exchange(w[f][j]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // byte i of the word as a power of two, or where only its exponent counts
                        const float sc = KIND == IN_F16 ? power((s[f][j] >> (8 * i)) & 255u)
                                                        : __builtin_bit_cast(float, i < 3 ? s[f][j] << (23 - 8 * i) : s[f][j] >> 1);
                        const u32x4 y = decode<KIND>(q[i], KIND == IN_BF16 ? sc : 1.0f);
#pragma unroll
                        for (int t = 0; t < TM; ++t) {
                            if constexpr (KIND == IN_BF16) acc[t][f] = dtl::mfma16<KIND>(fragment(t, 4 * j + i), y, acc[t][f]);
                            else {
                                const f32x4 b = dtl::mfma16<KIND>(fragment(t, 4 * j + i), y, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[t][f][r] = fmaf(sc, b[r], acc[t][f][r]);
                            }
                        }
                    }
                }
            }
    };
    // units without an end in them, whose scales lie side by side
    const int whole = a.s_cs == 1 && (KIND != CODES || a.sa_cs == 1) ? min(u1, a.K / (2 * UNIT)) : u0;
    int u = u0 + wave;
#pragma unroll 1
    for (; u < whole; u += WAVES) one(Int<1>(), u);
#pragma unroll 1
    for (; u < u1; u += WAVES) one(Int<0>(), u);

    if (STAGED) __syncthreads();                   // every wave has read its rows of A
    // the waves' sums: register r of lane (g, n) is C[16 t + 4 g + r][16 f + n]
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave * REGS + (t * NF + f) * 256 + r * 64 + lane] = acc[t][f][r];
    __syncthreads();
    float v[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = k * NT + tid;
        v[k] = 0.f;
        if (i >= REGS) continue;
        v[k] = red[i];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v[k] += red[w * REGS + i];
    }
    if (a.splits > 1) {                            // the pieces' sums, in the order of K
        float *part = a.ws + (int64_t)unit * a.splits * REGS;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k * NT + tid < REGS) __hip_atomic_store(part + z * REGS + k * NT + tid, v[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) is_last = take_last_ticket(a.counters + unit, a.splits);
        __syncthreads();
        if (!is_last) return;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k * NT + tid < REGS)
                v[k] = sum_partials(a.splits, [&](int q) { return __hip_atomic_load(part + q * REGS + k * NT + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); });
        if (tid == 0) __hip_atomic_store(a.counters + unit, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = k * NT + tid, b = i >> 8, t = b / NF, f = b - t * NF;
        const int m = m0 + 16 * t + 4 * ((i >> 4) & 3) + ((i >> 6) & 3), col = n0 + 16 * f + (i & 15);
        if (i < REGS && m < M && col < a.N)
            store_out(a.C + (int64_t)(begin + m) * a.c_rs + (int64_t)col * a.c_cs, a.out_kind, activate(a.act, v[k]));
    }
}

template <int KIND, int TM, int NF, bool STAGED>
hipError_t launch(const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    const auto k = mx4_few<KIND, TM, NF, STAGED>;
    const int bytes = std::max(WAVES * TM * NF * 1024, STAGED ? WAVES * a.a_rows * 1024 : 0);
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)units), dim3(NT), bytes, s, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_rows(int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    if (a.a_rows) return nf == 1 ? launch<KIND, 1, 1, true>(a, units, s) : launch<KIND, 1, 2, true>(a, units, s);
    return nf == 1 ? launch<KIND, 1, 1, false>(a, units, s) : launch<KIND, 1, 2, false>(a, units, s);
}

}  // namespace

hipError_t launch_mx4_few(int kind, int tm, int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    if (nf != 1 && nf != 2) return hipErrorInvalidValue;
    if (kind == MX4_CODES && tm == 1) return nf == 1 ? launch<CODES, 1, 1, false>(a, units, s) : launch<CODES, 1, 2, false>(a, units, s);
    if (kind == MX4_CODES && tm == 2) return nf == 1 ? launch<CODES, 2, 1, false>(a, units, s) : launch<CODES, 2, 2, false>(a, units, s);
    if (kind == IN_BF16 && tm == 1) return launch_rows<IN_BF16>(nf, a, units, s);
    if (kind == IN_F16 && tm == 1) return launch_rows<IN_F16>(nf, a, units, s);
    return hipErrorInvalidValue;
}

}  // namespace dg
