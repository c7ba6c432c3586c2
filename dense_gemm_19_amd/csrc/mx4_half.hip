// mx4_half.hip -- products of 16-bit activations with microscaled 4-bit weights where many
// rows meet every weight (few: mx4_few.hip; between: w4.hpp):
//
//   C[m][n] = act(sum over blocks b of 32 k's of 2^(s[n][b] - 127) * sum over k in b of A[m][k] w[n][k])
//
// BF16: the weights of a block times their scale are BF16 numbers, exactly (E2M1 has two
// significant bits; the two largest scales apart), which one instruction converts two at a
// time; the matrix cores do the rest.  FP16 does not hold every scale: a workgroup whose
// scales all lie in its range goes the same way, in another the codes are converted as they
// are, a block's sum is formed in FP32 on the matrix cores and enters the FP32 accumulator
// times its scale (2048 x 4096 x 4096: 64 us, 85 that way; BF16 62).  A BF16 workgroup that
// met one of the largest scales sums its tile once more that way, as block_scale says.
// What bounds it: the matrix instructions, 27 us of those 62 at the full clock, with 4.5
// vector instructions to each, and one round of tiles whose first loads and stores
// nothing overlaps (8192^3: 875 us, 1.26 PFLOP/s).
#include "bytes.hpp"
#include "device_common.hpp"
#include "e8m0.hpp"
#include "gemm_dtl.hpp"
#include "moe_slot.hpp"
#include "mx4_tile.hpp"

namespace dg {
namespace {

constexpr int KB = 128;          // bytes of a row in LDS: 64 elements of A, 256 codes of W

__device__ __forceinline__ void load_lds16(const char *base, uint32_t off, uint32_t a) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(a), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void load_lds4(const char *base, uint32_t off, uint32_t a) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(a), "v"(off), "s"(base) : "m0");
}
// one byte a lane, a word each in LDS
__device__ __forceinline__ void load_lds1(const char *base, uint32_t off, uint32_t a) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2" ::"s"(a), "v"(off), "s"(base) : "m0");
}
template <int N>
__device__ __forceinline__ void arrive() {   // all but the last N loads of this wave are there, in every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int N> using Int = std::integral_constant<int, N>;

// 2^(b - 127) for the conversion, which reads its exponent alone.
template <int IN>
__device__ __forceinline__ float power(uint32_t b) {
    if constexpr (IN == IN_BF16) return __builtin_bit_cast(float, b << 23);
    return e8m0_value(b);
}

// 8 codes as 16-bit numbers, times the scale.
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

template <int IN>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// BM x BN tiles, waves WGM x WGN.  LDS: a ring of four 64-element parts of A, two tiles of
// 256 codes of W, the scale bytes of two such tiles, a word each ([block][row]).
// A part is four steps of 16 elements.  BF16: lanes 0-31 take the part's first block and
// lanes 32-63 its second, 8 elements at each step, so that a lane's codes are one read and
// its scale is one.  FP16: a step lies within a block, 8 elements of either half.
//  - Fragments are read a step ahead.  The barrier before a part's last step says that the
//    part has been read by every wave and the next one has arrived; the loads of four
//    parts later go into its slot (W's of two tiles later where the part is a tile's last).
//  - Loads return in order and every wave issues the same number, so the waits count them.
//  - A ragged K: parts past the end are not computed; what the last one holds past it is
//    cleared, scales and codes too, since a large scale makes infinities of what is there.
// WORDS: the scales come four to a word (side by side, aligned, K in whole groups of 128): a
// load of 64 rows takes as long for a byte of each as for a word, 28 ns (BF16 2048 x 4096 x
// 4096: 62 us, byte by byte 71).
// VIA: A and W at any alignment, any K: through registers, each load a part (W: a tile) on
// the way before it is written where a load to LDS would have put it; the end of K apart
// (BF16 2048 x 4096 x 4100: 93 us).
template <int IN, int BM, int BN, int WGM, int WGN, bool WORDS, bool VIA>
__global__ void __launch_bounds__(64 * WGM * WGN) mx4_half(Mx4GemmArgs a) {
    constexpr int NW = WGM * WGN, NT = 64 * NW, WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 32, TN = WTN / 32;
    constexpr bool SPLIT = BM == 64;               // K in pieces
    constexpr int PART = BM * KB, W_OFF = 4 * PART, WTILE = BN * KB, S_OFF = W_OFF + 2 * WTILE, SB = WORDS ? 4 : 1, STILE = 8 / SB * BN * 4, LDS = S_OFF + 2 * STILE;
    constexpr int AI = BM * 8 / 64 / NW, WI = BN * 8 / 64 / NW, SI = 8 / SB * BN / 64 / NW, S1 = (SI + 1) / 2, SR = BN / 64;
    static_assert(AI * 64 * NW == BM * 8 && WI * 64 * NW == BN * 8 && SI * SB * 64 * NW == 8 * BN && NW % SR == 0, "whole loads");
    static_assert(LDS + 64 <= 160 * 1024 && NW * MX4_STORE_LDS<TN> <= LDS, "LDS");
    __shared__ __attribute__((aligned(16))) char lds[LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN, l = lane & 31, h = lane >> 5;
    Mx4Part p;
    if (!mx4_part<BM, BN, SPLIT>(a, p)) return;
    // this piece of K: whole tiles, the last one what is left of K too
    const int k0 = p.z * a.kt_per_split * 256, K = !p.live ? 0 : !SPLIT || p.z == a.splits - 1 ? a.K - k0 : a.kt_per_split * 256, parts = (K + 63) / 64;
    const int row_bytes = (K + 1) / 2, blocks = (K + 31) / 32;

    const char *pa = a.A + (int64_t)(p.begin + p.m0) * a.a_rs + (int64_t)k0 * 2;
    const char *pw = a.Q + (int64_t)p.e * a.q_es + (int64_t)p.n0 * a.q_rs + k0 / 2, *ps = a.S + (int64_t)p.e * a.s_es + (int64_t)p.n0 * a.s_rs + (int64_t)(k0 / 32) * a.s_cs;
    const uint32_t lds0 = dtl::lds_addr(lds);
    const int last_m = p.M - 1 - p.m0, last_n = a.N - 1 - p.n0;   // rows past them read these (not stored)
    uint32_t a_off[AI], w_off[WI], s_off;
    int w_most[WI];
    // chunk (16 bytes) of this lane's loads: position ^ row / 2 of A and W alike
    const int chunk = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) << 4;
    static_assert(NW * 4 % 8 == 0, "one chunk for every load of a lane");
#pragma unroll
    for (int j = 0; j < AI; ++j) a_off[j] = (uint32_t)min((wave + NW * j) * 8 + (lane >> 3), last_m) * (uint32_t)a.a_rs;
#pragma unroll
    for (int j = 0; j < WI; ++j) {
        const int row = min((wave + NW * j) * 8 + (lane >> 3), last_n);
        w_off[j] = (uint32_t)row * (uint32_t)a.q_rs;
        // the last row's last chunk ends with it; any other one may reach into the next row
        w_most[j] = row == last_n ? row_bytes - 16 : (row_bytes - 1) & ~15;
    }
    s_off = (uint32_t)min((wave % SR) * 64 + lane, last_n) * (uint32_t)a.s_rs;
    u32x4 va[VIA ? AI : 1], vw[VIA ? WI : 1];      // VIA: on the way
    auto put_a = [&](int j, int t) __attribute__((always_inline)) { *reinterpret_cast<u32x4 *>(lds + (t & 3) * PART + (wave + NW * j) * 1024 + 16 * lane) = va[j]; };
    auto put_w = [&](int j, int T) __attribute__((always_inline)) { *reinterpret_cast<u32x4 *>(lds + W_OFF + (T & 1) * WTILE + (wave + NW * j) * 1024 + 16 * lane) = vw[j]; };
    auto load_a = [&](int j, int t) __attribute__((always_inline)) {   // chunks past K: the last one
        if constexpr (VIA) va[j] = *reinterpret_cast<const u32x4_any *>(pa + (a_off[j] + (uint32_t)min(t * KB + chunk, 2 * K - 16)));
        else load_lds16(pa, a_off[j] + (uint32_t)min(t * KB + chunk, 2 * K - 16), lds0 + (uint32_t)((t & 3) * PART + (wave + NW * j) * 1024));
    };
    auto load_w = [&](int j, int T) __attribute__((always_inline)) {
        if constexpr (VIA) vw[j] = *reinterpret_cast<const u32x4_any *>(pw + (w_off[j] + (uint32_t)min(T * KB + chunk, row_bytes - 16)));
        else load_lds16(pw, w_off[j] + (uint32_t)min(T * KB + chunk, w_most[j]), lds0 + (uint32_t)(W_OFF + (T & 1) * WTILE + (wave + NW * j) * 1024));
    };
    auto load_s = [&](int j, int T) __attribute__((always_inline)) {   // one block, or word, of 64 rows
        const int b = wave / SR + (NW / SR) * j;
        if constexpr (WORDS) load_lds4(ps, s_off + (uint32_t)min(8 * T + 4 * b, blocks - 4), lds0 + (uint32_t)(S_OFF + (T & 1) * STILE + b * (BN * 4) + (wave % SR) * 256));
        else load_lds1(ps, s_off + (uint32_t)min(8 * T + b, blocks - 1) * (uint32_t)a.s_cs, lds0 + (uint32_t)(S_OFF + (T & 1) * STILE + b * (BN * 4) + (wave % SR) * 256));
    };

    f32x16 acc[TM][TN];
    auto zero_sums = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    };
    zero_sums();
    uint32_t top = 0;                              // BF16: the largest scale byte that this lane met
    __shared__ int past;                           // and whether BF16 does not hold one of them
    // ONE: a lane's elements of a part are of one block, and W's are taken times its scale.
    auto run = [&](auto one) __attribute__((always_inline)) {
        constexpr bool ONE = decltype(one)::value;
        constexpr int CH = ONE ? 1 : 2;            // W: chunks and scales of a part that a lane reads
        u32x4 fa[2][TM], wq[2][TN][CH];                // of even and odd steps; of even and odd parts
        uint32_t sw[2][TN][CH];                        // scale bytes
        BlockScale sc[TN][CH];                         // what they stand for (ONE: all in the conversion): the part at hand
        const int ra = (wm * WTM + l) * KB, rw = W_OFF + (wn * WTN + l) * KB, rs = S_OFF + (wn * WTN + l) * 4, swz = (l >> 1) & 7;
        auto read_a = [&](int step, int i, int slot) __attribute__((always_inline)) {
            fa[step & 1][i] = *reinterpret_cast<const u32x4 *>(lds + ra + slot * PART + 32 * i * KB + (((ONE ? 4 * h + step : 2 * step + h) ^ swz) << 4));
        };
        auto read_w = [&](int j, int q, int T) __attribute__((always_inline)) {   // the codes and scales of part q of tile T
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int b = 2 * q + (ONE ? h : c);
                const char *at = lds + rs + (T & 1) * STILE + 128 * j;
                wq[q & 1][j][c] = *reinterpret_cast<const u32x4 *>(lds + rw + (T & 1) * WTILE + 32 * j * KB + ((b ^ swz) << 4));
                if constexpr (WORDS) sw[q & 1][j][c] = *reinterpret_cast<const uint8_t *>(at + (q >> 1) * (BN * 4) + (b & 3));
                else sw[q & 1][j][c] = *reinterpret_cast<const uint32_t *>(at + b * (BN * 4));
            }
        };
        f32x16 blk[ONE ? 1 : TM][ONE ? 1 : TN];          // a block's sums
        auto multiply = [&](auto s, int q) __attribute__((always_inline)) {
            constexpr int STEP = decltype(s)::value;
            u32x4 fb[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (ONE) fb[j] = decode<IN>(wq[q & 1][j][0][STEP], sc[j][0].in);
                else {
                    const u32x4 c = wq[q & 1][j][STEP >> 1];
                    fb[j] = decode<IN>(h ? c[2 * (STEP & 1) + 1] : c[2 * (STEP & 1)], sc[j][STEP >> 1].in);
                }
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if constexpr (ONE) acc[i][j] = mfma<IN>(fa[STEP & 1][i], fb[j], acc[i][j]);
                    else {
                        f32x16 zero;
#pragma unroll
                        for (int r = 0; r < 16; ++r) zero[r] = 0.f;
                        blk[i][j] = mfma<IN>(fa[STEP & 1][i], fb[j], STEP & 1 ? blk[i][j] : zero);
                    }
                }
            if constexpr (!ONE && (STEP & 1)) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(sc[j][STEP >> 1].out, blk[i][j][r], acc[i][j][r]);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // Part q of tile T (part t = 4 T + q of K).  REFILL: its slots are filled again; MORE:
        // another whole part follows, whose first fragments are read; LEFT: loads that may be
        // in flight then.
        auto part = [&](auto qc, auto refill, auto more, auto left, int T) __attribute__((always_inline)) {
            constexpr int Q = decltype(qc)::value;
            const int t = 4 * T + Q;
            auto next = [&](int step) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < TM; ++i) read_a(step, i, Q);
                __builtin_amdgcn_sched_barrier(0);
            };
            next(1);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint32_t b = sw[Q & 1][j][c];
                    if constexpr (ONE) sc[j][c] = {power<IN>(b), 1.0f};
                    else sc[j][c] = block_scale<IN>(b);
                    if (ONE && IN == IN_BF16) top = max(top, b);
                }
            multiply(Int<0>(), Q);
            next(2);
            multiply(Int<1>(), Q);
            next(3);
            multiply(Int<2>(), Q);
            if constexpr (decltype(more)::value) {
                arrive<VIA ? 0 : decltype(left)::value>();
#pragma unroll
                for (int i = 0; i < TM; ++i) read_a(0, i, (Q + 1) & 3);
#pragma unroll
                for (int j = 0; j < TN; ++j) read_w(j, (Q + 1) & 3, T + (Q == 3));
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (decltype(refill)::value && Q < 2) {
#pragma unroll
                    for (int j = Q * S1; j < (Q ? SI : S1); ++j) load_s(j, T + 1);
                }
                if constexpr (decltype(refill)::value) {
#pragma unroll
                    for (int j = 0; j < AI; ++j) {
                        if constexpr (VIA) put_a(j, t + 3);
                        load_a(j, t + 4);
                    }
                }
                if constexpr (VIA && decltype(refill)::value && Q == 0) {
#pragma unroll
                    for (int j = 0; j < WI; ++j) put_w(j, T + 1);
                }
                if constexpr (decltype(refill)::value && Q == 3) {
#pragma unroll
                    for (int j = 0; j < WI; ++j) load_w(j, T + 2);
                }
            }
            multiply(Int<3>(), Q);
        };
        using Yes = Int<1>;
        using No = Int<0>;


        const int whole = K / 64;                  // parts without an end in them
        if (whole > 0) {
            arrive<VIA ? 0 : 3 * AI + WI>();
#pragma unroll
            for (int i = 0; i < TM; ++i) read_a(0, i, 0);
#pragma unroll
            for (int j = 0; j < TN; ++j) read_w(j, 0, 0);
        }
        // Loads in flight that a part does not wait for: those that the two parts before it
        // issued, but the scales that the part after a tile's last one reads.
        int T = 0;
#pragma unroll 1
        for (; 4 * T + 4 < whole; ++T) {
            part(Int<0>(), Yes(), Yes(), Int<2 * AI + WI>(), T);
            part(Int<1>(), Yes(), Yes(), Int<2 * AI + WI + S1>(), T);
            part(Int<2>(), Yes(), Yes(), Int<2 * AI + SI>(), T);
            part(Int<3>(), Yes(), Yes(), Int<2 * AI>(), T);
        }
        if constexpr (VIA) {
#pragma unroll
            for (int j = 0; j < AI; ++j) put_a(j, 4 * T + 3);
        }
        // the last one to four whole parts
        const int rest = whole - 4 * T;
        if (rest == 1) part(Int<0>(), No(), No(), Int<0>(), T);
        if (rest > 1) {
            part(Int<0>(), No(), Yes(), Int<0>(), T);
            if (rest == 2) part(Int<1>(), No(), No(), Int<0>(), T);
        }
        if (rest > 2) {
            part(Int<1>(), No(), Yes(), Int<0>(), T);
            if (rest == 3) part(Int<2>(), No(), No(), Int<0>(), T);
        }
        if (rest > 3) {
            part(Int<2>(), No(), Yes(), Int<0>(), T);
            part(Int<3>(), No(), No(), Int<0>(), T);
        }
        if (!WORDS && parts > whole) {
            const int t = whole, TT = t >> 2, q = t & 3, left = row_bytes - TT * KB, n = left & 15, there = blocks - 8 * TT;
            if (q == 0 && t > 0) {                 // the first of its tile: no part before loaded these
#pragma unroll
                for (int j = 0; j < SI; ++j) load_s(j, TT);
                if constexpr (!VIA) {
#pragma unroll
                    for (int j = 0; j < AI; ++j) load_a(j, t);
                }
            }
            arrive<0>();
            if constexpr (VIA) {
#pragma unroll 1
                for (int i = tid; i < BM * 8; i += NT)
                    *reinterpret_cast<u32x4 *>(lds + (t & 3) * PART + 16 * i) = row_piece(pa + (uint32_t)min(i >> 3, last_m) * (uint32_t)a.a_rs, t * KB + 16 * ((i & 7) ^ ((i >> 4) & 7)), 2 * K);
#pragma unroll 1
                for (int i = tid; i < BN * 8; i += NT)
                    *reinterpret_cast<u32x4 *>(lds + W_OFF + (TT & 1) * WTILE + 16 * i) = row_piece(pw + (uint32_t)min(i >> 3, last_n) * (uint32_t)a.q_rs, TT * KB + 16 * ((i & 7) ^ ((i >> 4) & 7)), row_bytes);
            } else {
#pragma unroll 1
                for (int i = tid; i < BM * 8; i += NT)   // A: chunks from K on (K is a multiple of 8)
                    if (64 * t + 8 * ((i & 7) ^ ((i >> 4) & 7)) >= K) *reinterpret_cast<u32x4 *>(lds + (t & 3) * PART + 16 * i) = u32x4{0u, 0u, 0u, 0u};
                if (n != 0) {                          // W: the last chunk of the rows
#pragma unroll 1
                    for (int r = tid; r < BN; r += NT) {
                        u32x4 *c = reinterpret_cast<u32x4 *>(lds + W_OFF + (TT & 1) * WTILE + r * KB + (((left >> 4) ^ ((r >> 1) & 7)) << 4));
                        *c = r >= last_n ? down_bytes(*c, 16 - n) : first_bytes(*c, n);
                    }
            }
            }
#pragma unroll 1
            for (int i = tid; i < 8 * BN; i += NT)   // scales of blocks past the end
                if (i / BN >= there) *reinterpret_cast<uint32_t *>(lds + S_OFF + (TT & 1) * STILE + 4 * i) = 0u;
            arrive<0>();
            auto ragged = [&](auto qc) __attribute__((always_inline)) {
                constexpr int Q = decltype(qc)::value;
#pragma unroll
                for (int i = 0; i < TM; ++i) read_a(0, i, Q);
#pragma unroll
                for (int j = 0; j < TN; ++j) read_w(j, Q, TT);
                part(qc, No(), No(), Int<0>(), TT);
            };
            if (q == 0) ragged(Int<0>());
            else if (q == 1) ragged(Int<1>());
            else if (q == 2) ragged(Int<2>());
            else ragged(Int<3>());
        }
    };
    // as the four parts before the first would have issued them
    auto first_loads = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < WI; ++j) {
            load_w(j, 0);
            if constexpr (VIA) put_w(j, 0);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t < 2) {
#pragma unroll
                for (int j = t * S1; j < (t ? SI : S1); ++j) load_s(j, 0);
            }
#pragma unroll
            for (int j = 0; j < AI; ++j) {
                load_a(j, t);
                if (VIA && t < 3) put_a(j, t);
            }
        }
#pragma unroll
        for (int j = 0; j < WI; ++j) load_w(j, 1);   // (past the end: the rows' ends)
    };
    if (parts > 0) {
        first_loads();
        if constexpr (IN == IN_BF16) {
            if (tid == 0) past = 0;                // (barriers lie between)
            run(Int<1>());
            if (top >= 253u) past = 1;
            arrive<0>();                           // every wave has read its last fragments
            if (__builtin_expect(__builtin_amdgcn_readfirstlane(past), 0)) {
                zero_sums();
                first_loads();
                run(Int<0>());
            }
        } else if constexpr (!WORDS) run(Int<0>());
        else {
            // does FP16 hold every code times its scale: 2^-24 .. 2^15, scales 2^-23 .. 2^13?
            uint32_t far = 0;
            const int words = blocks / 4, rows = min(BN, last_n + 1);
#pragma unroll 1
            for (int c = lane & 15; c < words; c += 16)
#pragma unroll 8
                for (int r = tid >> 4; r < BN; r += NT / 16) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(ps + (int64_t)min(r, rows - 1) * a.s_rs + 4 * c);
#pragma unroll
                    for (int b = 0; b < 4; ++b) far |= ((v >> (8 * b)) & 255u) - 104u > 36u;
                }
            if (__syncthreads_or((int)far)) run(Int<0>());
            else run(Int<1>());
        }
    }
    arrive<0>();                                   // every wave has read its last fragments
    if (SPLIT && a.splits > 1) {
        // [tile][piece][element][thread]: every thread adds its own elements, in the order of
        // K, four pieces on the way at once
        constexpr int REGS = TM * TN * 16;
        __shared__ int is_last;
        float *sums = a.ws + (int64_t)p.t * a.splits * (BM * BN) + tid;
#pragma unroll
        for (int k = 0; k < REGS; ++k)
            __hip_atomic_store(sums + (int64_t)p.z * (BM * BN) + k * NT, acc[k / 16 / TN][k / 16 % TN][k % 16], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) is_last = take_last_ticket(a.counters + p.t, a.splits);
        __syncthreads();
        if (!is_last) return;
#pragma unroll
        for (int k = 0; k < REGS; ++k) acc[k / 16 / TN][k / 16 % TN][k % 16] = 0.f;
#pragma unroll 1
        for (int q = 0; q < a.splits; q += 4) {
            float v[4][REGS];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (q + u < a.splits)
#pragma unroll
                    for (int k = 0; k < REGS; ++k) v[u][k] = __hip_atomic_load(sums + (int64_t)(q + u) * (BM * BN) + k * NT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (q + u < a.splits)
#pragma unroll
                    for (int k = 0; k < REGS; ++k) acc[k / 16 / TN][k / 16 % TN][k % 16] += v[u][k];
        }
        if (tid == 0) __hip_atomic_store(a.counters + p.t, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    mx4_store<TM, TN, true>(a, p, acc, wm * WTM, wn * WTN, lane, lds + wave * MX4_STORE_LDS<TN>);
}

}  // namespace

hipError_t launch_mx4_half(int in_kind, int tile, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
#define DG_HALF(IN, BM, BN, GM, GN)                                                                                                                     \
    do {                                                                                                                                                \
        if (a.via) hipLaunchKernelGGL((mx4_half<IN, BM, BN, GM, GN, false, true>), dim3((unsigned)units), dim3(64 * GM * GN), 0, s, a);                 \
        else if (a.s_words) hipLaunchKernelGGL((mx4_half<IN, BM, BN, GM, GN, true, false>), dim3((unsigned)units), dim3(64 * GM * GN), 0, s, a);        \
        else hipLaunchKernelGGL((mx4_half<IN, BM, BN, GM, GN, false, false>), dim3((unsigned)units), dim3(64 * GM * GN), 0, s, a);                      \
    } while (0)
    if (tile == MX4_T128x256 && in_kind == IN_BF16) DG_HALF(IN_BF16, 128, 256, 2, 4);
    else if (tile == MX4_T128x256) DG_HALF(IN_F16, 128, 256, 2, 4);
    else if (tile == MX4_T64x128 && in_kind == IN_BF16) DG_HALF(IN_BF16, 64, 128, 2, 2);
    else if (tile == MX4_T64x128) DG_HALF(IN_F16, 64, 128, 2, 2);
    else return hipErrorInvalidValue;
#undef DG_HALF
    return hipGetLastError();
}

}  // namespace dg
