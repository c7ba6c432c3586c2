// mx4_few.hip -- products with MXFP4 weights where few rows meet them, bound by the bytes of
// the codes: every wave streams its part of the weights' rows from memory straight to
// registers, no two waves the same, and all of a wave's loads are in flight before the
// first is used.
//
// A workgroup's 8 waves share 16 NF columns and split K: a unit is 512 elements, 256 bytes
// of a row of codes and 16 of its scales.  Lane (g, n), n = lane % 16, loads of row n the 16
// bytes 64 j + 16 g at each of four steps j, a whole block, and all 16 scale bytes.
// Bytes of codes bound it for a few rows, the way of A from the caches beyond (all columns'
// workgroups read it): 1 x 14336 x 4096, 31 MB, 8.7 us BF16 and 8.1 codes, 3.6 TB/s with a
// launch of 1.5 us in it; 16 rows 11.3 / 9.2; 33 x 4096 x 14336 17.5 us BF16.
//   A in codes: those are the operands of v_mfma_scale_f32_16x16x128_f8f6f4 as they lie.
//   A in 16 bits: the lanes of a row first exchange words (a 4 x 4 transpose in four
//   instructions), so that an instruction of 32 elements meets one block of every row.
//   The weights are converted times their scale, exactly, in BF16 and for STEPS (see below)
//   in FP16, too, where the type holds them; elsewhere as block_scale says, and a block's
//   sum, in FP32, is added times its factor.
#include <algorithm>

#include "bytes.hpp"
#include "device_common.hpp"
#include "e8m0.hpp"
#include "gemm_dtl.hpp"
#include "moe_slot.hpp"
#include "mx4_tile.hpp"

namespace dg {
namespace {

constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int UNIT = 256;        // bytes of a row of codes
constexpr int CODES = MX4_CODES;   // beside IN_F16, IN_BF16

template <int N> using Int = std::integral_constant<int, N>;

// words[i] of lane row g <- words[g] of lane row i (lane rows of 16 lanes)
__device__ __forceinline__ u32x4 exchange(u32x4 v) {
    auto s0 = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto s1 = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto t0 = __builtin_amdgcn_permlane16_swap(s0[0], s1[0], false, false);
    auto t1 = __builtin_amdgcn_permlane16_swap(s0[1], s1[1], false, false);
    return u32x4{t0[0], t0[1], t1[0], t1[1]};
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

// Waits until at most n loads of this wave are on the way (n: 1 to MAX, the same in all lanes).
template <int MAX>
__device__ __forceinline__ void all_but(int n) {
    if constexpr (MAX > 1) {
        if (n < MAX) return all_but<MAX - 1>(n);
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MAX) : "memory");
}

// How a 16-bit A gets to the lanes.  Straight to registers a fragment takes as much of the
// way from the cache whether its 16 rows differ or not (1 x 14336 x 4096: 11.6 us), so
// where A's rows begin at whole words they go through a wave's own part of LDS:
//  ROWS : the rows of whole units, 1 KB to a load, of 8 rows at most (8.8 us);
//  STEPS: 128 elements of 4 rows to a load, a step ahead of their use.
enum { STRAIGHT = 0, ROWS = 1, STEPS = 2 };

// MR rows (16 TM, or as many of them as LDS has room for) x 16 NF columns.  (Codes of four
// units on the way at once, or A's lines touched ahead, gave nothing.)
template <int KIND, int TM, int NF, int HOW>
__global__ void __launch_bounds__(NT) mx4_few(Mx4GemmArgs a) {
    constexpr int MR = mx4_few_rows(TM), NC = 16 * NF, REGS = mx4_few_sums(TM, NF), PER = (REGS + NT - 1) / NT;
    constexpr bool CHECK = KIND == IN_F16 && HOW == STEPS;   // FP16: are the scales in its range?
    extern __shared__ __attribute__((aligned(16))) char lds[];   // A, see above; then the waves' sums
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
    // the products of a step (128 elements) of row blocks t0 on and columns f: codes w, scales
    // s.  one: the codes are taken times their scale
    auto step16 = [&](auto one, const u32x4 w, uint32_t s, int f, int t0, const auto &x) __attribute__((always_inline)) {
        constexpr int T = sizeof(x) / sizeof(x[0]);
        const u32x4 q = exchange(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (decltype(one)::value) {
                // byte i of the word at the exponent's bits, the only ones that count
                const u32x4 y = decode<KIND>(q[i], __builtin_bit_cast(float, i < 3 ? s << (23 - 8 * i) : s >> 1));
#pragma unroll
                for (int t = 0; t < T; ++t) acc[t0 + t][f] = dtl::mfma16<KIND>(x[t][i], y, acc[t0 + t][f]);
            } else {
                const BlockScale sc = block_scale<KIND>((s >> (8 * i)) & 255u);
                const u32x4 y = decode<KIND>(q[i], sc.in);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const f32x4 b = dtl::mfma16<KIND>(x[t][i], y, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t0 + t][f][r] = fmaf(sc.out, b[r], acc[t0 + t][f][r]);
                }
                __builtin_amdgcn_sched_barrier(0);   // (registers)
            }
        }
    };
    auto step4 = [&](const u32x4 w, uint32_t s, int f, const u32x4 (&x)[TM], const uint32_t (&sx)[TM]) __attribute__((always_inline)) {
        const i32x8 y = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const i32x8 v = {(int)x[t][0], (int)x[t][1], (int)x[t][2], (int)x[t][3], 0, 0, 0, 0};
            acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, y, acc[t][f], 4, 4, 0, (int)(sx[t] >> (8 * g)), 0, (int)(s >> (8 * g)));
        }
    };

    // Step st of 128 elements as it comes: an end in it, scales apart, or scales that the
    // type does not hold.
    auto any_step = [&](int st) __attribute__((always_inline)) {
        const int u = st >> 2, j = st & 3, at = u * UNIT + 16 * g + 64 * j, b = 16 * u + 4 * j;
        auto scales = [&](const char *row, int64_t cs) __attribute__((always_inline)) {
            uint32_t v = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (b + i < a.blocks) v |= (uint32_t)*reinterpret_cast<const uint8_t *>(row + (b + i) * cs) << (8 * i);
            return v;
        };
        if constexpr (KIND == CODES) {
            u32x4 x[TM];
            uint32_t sx[TM];
#pragma unroll
            for (int t = 0; t < TM; ++t) { x[t] = row_piece(arow[t], at, a.row_bytes); sx[t] = scales(sarow[t], a.sa_cs); }
#pragma unroll
            for (int f = 0; f < NF; ++f) step4(row_piece(wrow[f], at, a.row_bytes), scales(srow[f], a.s_cs), f, x, sx);
        } else {
            u32x4 w[NF];
            uint32_t sw[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f) { w[f] = row_piece(wrow[f], at, a.row_bytes); sw[f] = scales(srow[f], a.s_cs); }
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                u32x4 x[1][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[0][i] = row_piece(arow[t], u * (4 * UNIT) + 16 * g + 256 * j + 64 * i, 2 * a.K);
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    if (KIND == IN_BF16 && !__builtin_amdgcn_ballot_w64(top_scales(sw[f]) != 0)) step16(Int<1>(), w[f], sw[f], f, t, x);
                    else step16(Int<0>(), w[f], sw[f], f, t, x);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };

    // Units without an end in them, whose scales lie side by side.
    const int whole = a.s_cs == 1 && (KIND != CODES || a.sa_cs == 1) ? min(u1, a.K / (2 * UNIT)) : u0;
    const int rows = min(M - m0, MR);
    const char *base = a.A + (int64_t)(begin + m0) * a.a_rs;
    char *own = lds + wave * (HOW == STEPS ? 2 * ((a.a_rows + 3) / 4) * 1024 : a.a_rows * 1024);
    const uint32_t to = dtl::lds_addr(own);
    // STEPS: load i brings rows 4 i to 4 i + 3, chunk c of row r at c ^ r % 16 (16 rows' reads
    // fall on distinct banks; ROWS: c ^ r)
    constexpr int LOADS = (MR + 3) / 4;
    const int loads = (rows + 3) / 4, flip = 1024 * ((a.a_rows + 3) / 4);
    uint32_t a_off[LOADS];
    if constexpr (HOW == STEPS) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            a_off[i] = (uint32_t)min(4 * i + g, rows - 1) * (uint32_t)a.a_rs + 16 * (n ^ ((4 * i + g) & 15));
    }
    auto load_step = [&](int u, int j) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what was there has been read
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (i < loads) dtl::lds_load16(base + u * (4 * UNIT) + j * UNIT, a_off[i], to + (j & 1) * flip + i * 1024);
    };
    int u = u0 + wave;
    auto whole_units = [&]() __attribute__((always_inline)) {
        if constexpr (HOW == STEPS) {
            if (u < whole) load_step(u, 0);
        }
#pragma unroll 1
        for (; u < whole; u += WAVES) {
            u32x4 w[NF][4], s[NF], x4[TM][4], sx[TM];
            if constexpr (HOW == ROWS) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the last unit's have been read
#pragma unroll 1
                for (int r = 0; r < rows; ++r) dtl::lds_load16(base + (int64_t)r * a.a_rs + u * (4 * UNIT), 16 * (lane ^ r), to + r * 1024);
            }
            // all loads at once, in the order of use
#pragma unroll
            for (int f = 0; f < NF; ++f) s[f] = *reinterpret_cast<const u32x4_any *>(srow[f] + 16 * u);
            if constexpr (KIND == CODES) {
#pragma unroll
                for (int t = 0; t < TM; ++t) sx[t] = *reinterpret_cast<const u32x4_any *>(sarow[t] + 16 * u);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int f = 0; f < NF; ++f) w[f][j] = *reinterpret_cast<const u32x4_any *>(wrow[f] + u * UNIT + 16 * g + 64 * j);
                if constexpr (KIND == CODES) {
#pragma unroll
                    for (int t = 0; t < TM; ++t) x4[t][j] = *reinterpret_cast<const u32x4_any *>(arow[t] + u * UNIT + 16 * g + 64 * j);
                }
            }
            if constexpr (HOW == ROWS) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(5 * NF) : "memory");   // A, but not the codes
            else __builtin_amdgcn_sched_barrier(0);
            if constexpr (CHECK) {
                // FP16 holds codes times 2^-23 .. 2^13; zeros whatever their scale, if it is a number
                uint32_t far = 0;
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4 c = w[f][j];
                        const uint32_t b = (s[f][j] >> (8 * g)) & 255u, some = (c[0] | c[1] | c[2] | c[3]) & 0x77777777u;
                        far |= b - 104u > 36u && (some != 0 || b == 255u);
                    }
                if (__builtin_amdgcn_ballot_w64(far != 0)) break;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (KIND == CODES) {
                    u32x4 x[TM];
                    uint32_t sj[TM];
#pragma unroll
                    for (int t = 0; t < TM; ++t) { x[t] = x4[t][j]; sj[t] = sx[t][j]; }
#pragma unroll
                    for (int f = 0; f < NF; ++f) step4(w[f][j], s[f][j], f, x, sj);
                } else {
                    u32x4 x[TM][4];
                    if constexpr (HOW == STEPS) {
                        load_step(j < 3 || u + WAVES >= whole ? u : u + WAVES, (j + 1) & 3);   // (at the end: one that is not used)
                        all_but<LOADS>(loads);
                    }
#pragma unroll
                    for (int t = 0; t < TM; ++t) {
                        const int r = min(16 * t + n, rows - 1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = 16 * j + 4 * i + g;   // chunk of the unit
                            if constexpr (HOW == STEPS) x[t][i] = *reinterpret_cast<const u32x4 *>(own + (j & 1) * flip + r * 256 + 16 * ((c & 15) ^ (r & 15)));
                            else if constexpr (HOW == ROWS) x[t][i] = *reinterpret_cast<const u32x4 *>(own + r * 1024 + 16 * (c ^ r));
                            else x[t][i] = *reinterpret_cast<const u32x4_any *>(arow[t] + u * (4 * UNIT) + 16 * c);
                        }
                    }
#pragma unroll
                    for (int f = 0; f < NF; ++f) step16(Int<KIND == IN_BF16 || CHECK>(), w[f][j], s[f][j], f, 0, x);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    // The steps that are not of whole units, shared by the waves (a wave's four one after
    // another: 40 x 333 x 1000 codes 11.5 us beside 5.7).
    const int rest = 4 * max(whole, u0) + wave;
    if constexpr (CHECK) {                         // (each there once: registers)
#pragma unroll 1
        while (true) {
            whole_units();
            const bool far = u < whole;            // this unit's scales, else the rest
#pragma unroll 1
            for (int st = far ? 4 * u : rest; st < (far ? 4 * u + 4 : 4 * u1); st += far ? 1 : WAVES) any_step(st);
            if (!far) break;
            u += WAVES;
        }
    } else {
        whole_units();
        // BF16: a weight past its range makes a sum infinite or NaN, whatever A holds.  Units with
        // such a sum are summed once more, by steps (a look at every scale takes 3 to 7 % of a
        // call of one row).
        bool again = false;
        if constexpr (KIND == IN_BF16) {
            float odd = 0.f;                       // NaN then
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r) odd = fmaf(acc[t][f][r], 0.f, odd);
            again = __builtin_expect(__builtin_amdgcn_ballot_w64(odd != 0.f) != 0, 0);
        }
        if (again) {
#pragma unroll
            for (int t = 0; t < TM; ++t)
#pragma unroll
                for (int f = 0; f < NF; ++f) acc[t][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        int st = again ? 4 * (u0 + wave) : rest;
        if (__builtin_expect(st < 4 * u1, 0)) {    // (code that a K of whole units does not fetch)
#pragma unroll 1
            do {
                any_step(st);
                if (st >= 4 * whole) {
                    st += WAVES;
                } else if ((++st & 3) == 0) {      // the wave's next unit, or the rest
                    st += 4 * (WAVES - 1);
                    if (st >= 4 * whole) st = rest;
                }
            } while (st < 4 * u1);
        }
    }

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (HOW != STRAIGHT) __syncthreads();          // every wave has read its rows of A, none is on the way
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
        if (i < REGS && m < m0 + rows && col < a.N)
            store_out(a.C + (int64_t)(begin + m) * a.c_rs + (int64_t)col * a.c_cs, a.out_kind, activate(a.act, v[k]));
    }
}

template <int KIND, int TM, int NF, int HOW>
hipError_t launch(const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    const auto k = mx4_few<KIND, TM, NF, HOW>;
    const int lines = HOW == ROWS ? a.a_rows : HOW == STEPS ? 2 * ((a.a_rows + 3) / 4) : 0, bytes = WAVES * std::max(4 * mx4_few_sums(TM, NF), 1024 * lines);
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)units), dim3(NT), bytes, s, a);
    return hipGetLastError();
}
template <int KIND, int TM, int HOW>
hipError_t launch_columns(int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    return nf == 1 ? launch<KIND, TM, 1, HOW>(a, units, s) : nf == 2 ? launch<KIND, TM, 2, HOW>(a, units, s) : hipErrorInvalidValue;
}
template <int KIND>
hipError_t launch_half(int tm, int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    if (tm == 1 && nf == 1 && a.a_rows == 0) return launch<KIND, 1, 1, STRAIGHT>(a, units, s);
    if (a.a_rows <= 0 || a.a_rows > mx4_few_rows(tm)) return hipErrorInvalidValue;
    if (tm == 1 && nf == 1 && a.a_rows <= 8 && !a.offsets) return launch<KIND, 1, 1, ROWS>(a, units, s);
    if (tm == 1) return launch_columns<KIND, 1, STEPS>(nf, a, units, s);
    if (tm == 2) return launch_columns<KIND, 2, STEPS>(nf, a, units, s);
    return tm == 3 ? launch_columns<KIND, 3, STEPS>(nf, a, units, s) : hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_mx4_few(int kind, int tm, int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    if (kind == MX4_CODES && tm == 1) return launch_columns<CODES, 1, STRAIGHT>(nf, a, units, s);
    if (kind == MX4_CODES && tm == 2) return launch_columns<CODES, 2, STRAIGHT>(nf, a, units, s);
    if (kind == MX4_CODES && tm == 4) return launch_columns<CODES, 4, STRAIGHT>(nf, a, units, s);
    if (kind == IN_BF16) return launch_half<IN_BF16>(tm, nf, a, units, s);
    if (kind == IN_F16) return launch_half<IN_F16>(tm, nf, a, units, s);
    return hipErrorInvalidValue;
}

}  // namespace dg
