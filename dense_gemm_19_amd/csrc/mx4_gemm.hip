// mx4_gemm.hip -- products of two microscaled 4-bit (MXFP4) operands, for one matrix or
// for the experts of a mixture:
//
//   C[m][n] = act(sum over blocks b of 32 k's of 2^(sa[m][b] + s[n][b] - 254) * sum over k in b of a[m][k] w[n][k])
//
// gfx950 multiplies the format as it is: one v_mfma_scale_f32_32x32x64_f8f6f4 takes 32
// rows of each operand x 64 elements of K and a scale byte for each row and block, and
// adds into FP32.  (Register-only loops on this part: 9.6 PFLOP/s on zeros, 6.5 on random
// codes; the 16x16x128 form 4.2.)
//
// This kernel takes any K, layout and number of rows; large tiles of a regular K go to
// mx4_ring.hip, few rows to mx4_few.hip.  Two stages of 256 elements.  What bounds it: with
// 256 x 256 tiles the wait for the next stage beside the matrix instructions (4096 x 4096 x
// 5000: 58 us, 2.9 PFLOP/s), with 64 x 64 tiles the bytes in flight of one stage (64 x 14336
// x 4096: 16.7 us, 2.0 TB/s).
#include "bytes.hpp"
#include "mx4_tile.hpp"

namespace dg {
namespace {

constexpr int KB = 128;          // bytes of K in a tile: 256 elements, 8 blocks

// The scale bytes of 8 blocks from `at` on of a row of `blocks`, zeros past its end: the
// codes read there, whatever they are, then count 2^-254 times at most 36, nothing.
// RUN: bytes adjacent, 8 of them at least: loaded from 8 before the row's end at the
// latest, and moved down when they are used.
template <bool RUN>
__device__ __forceinline__ u32x2 load_scales(const char *row, int64_t stride, int at, int blocks) {
    if constexpr (RUN) {
        return *reinterpret_cast<const u32x2_byte *>(row + min(at, blocks - 8));
    } else {
        row += at * stride;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0;
            if (at + j < blocks) v[j] = *reinterpret_cast<const uint8_t *>(row + j * stride);
        }
        return u32x2{v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24, v[4] | v[5] << 8 | v[6] << 16 | v[7] << 24};
    }
}
template <bool RUN>
__device__ __forceinline__ u32x2 place_scales(u32x2 v, int at, int blocks) {
    if constexpr (RUN) {
        const uint64_t w = (v[0] | (uint64_t)v[1] << 32) >> (8 * max(at + 8 - blocks, 0));
        return u32x2{(uint32_t)w, (uint32_t)(w >> 32)};
    }
    return v;
}

// One operand's K tile: R rows x 128 bytes, 16-byte chunks XOR-swizzled by row / 2, so that
// the rows whose reads share a cycle fall on distinct banks.
__device__ __forceinline__ int chunk_off(int r, int c) { return r * KB + ((c ^ ((r >> 1) & 7)) << 4); }

template <int R, int NW>
struct TileIO {
    static constexpr int INSTS = R * 8 / 64 / NW;   // load-to-LDS instructions of a wave
    static constexpr int CHUNKS = R * 8 / (64 * NW);   // chunks of a thread
    struct Src { uint32_t off[INSTS]; };
    // rows past `lim` read the last one (their results are not stored)
    __device__ static Src sources(int64_t rs, int r0, int lim, int wave, int lane) {
        Src s;
#pragma unroll
        for (int j = 0; j < INSTS; ++j) {
            const int pos = (wave + NW * j) * 64 + lane, row = pos >> 3;
            s.off[j] = (uint32_t)min(row, lim - 1 - r0) * (uint32_t)rs + (((pos & 7) ^ ((row >> 1) & 7)) << 4);
        }
        return s;
    }
    __device__ static void issue(uint32_t lds, const Src &s, const char *base, int wave_u) {
#pragma unroll
        for (int j = 0; j < INSTS; ++j) dtl::lds_load16(base, s.off[j], lds + (uint32_t)((wave_u + NW * j) * 1024));
    }
    // through registers, at any alignment
    __device__ static void load(u32x4 (&reg)[CHUNKS], const char *base, int64_t rs, int r0, int lim, int at, int bytes, int tid) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int pos = tid + i * 64 * NW, row = pos >> 3;
            reg[i] = row_piece(base + (int64_t)min(row, lim - 1 - r0) * rs, at + (((pos & 7) ^ ((row >> 1) & 7)) << 4), bytes);
        }
    }
    __device__ static void store(char *lds, const u32x4 (&reg)[CHUNKS], int tid) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) *reinterpret_cast<u32x4 *>(lds + (tid + i * 64 * NW) * 16) = reg[i];
    }
};

// How codes get to LDS: through registers; by load-to-LDS instructions, from addresses of
// whole words; or so but for the ends of the last rows, where a row is no whole words long.
enum { REGS = 0, WORDS = 1, WORDS_ENDS = 2 };

// BM x BN tiles, waves WGM x WGN, a two-stage LDS ring.  DIRECT: rows begin at multiples
// of 4 bytes and codes go from memory to LDS by load-to-LDS instructions; else through
// registers.  RUN: see load_scales.
// K order within a tile: lanes 0-31 take blocks 0-3 and lanes 32-63 blocks 4-7, one at
// each of the four steps, so that a row's four scale bytes of a lane are one word and
// the step picks the byte.
// A ragged K, DIRECT: chunks past the end of a row read the next row, or for the last row its
// end again.  Whole blocks past the end have scale bytes of zero; of the last block the
// codes past the end are cleared in W's tile, and the last rows' are moved to where they
// belong in both (WORDS_ENDS: their last 16 bytes, which begin at any address, on their
// way in registers beside the tile).
template <int BM, int BN, int WGM, int WGN, int LOADS, bool RUN, bool SPLIT>
__global__ void __launch_bounds__(64 * WGM * WGN) mx4_tile(Mx4GemmArgs a) {
    constexpr bool DIRECT = LOADS != REGS, ENDS = LOADS == WORDS_ENDS;
    constexpr int NW = WGM * WGN, NT = 64 * NW, WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 32, TN = WTN / 32;
    constexpr int A_BYTES = BM * KB, B_BYTES = BN * KB, SA_OFF = A_BYTES + B_BYTES, SB_OFF = SA_OFF + BM * 8, STAGE = SB_OFF + BN * 8;
    constexpr int SROWS = (BM + BN + NT - 1) / NT;  // scale rows of a thread
    using AIO = TileIO<BM, NW>;
    using BIO = TileIO<BN, NW>;
    static_assert((BM + BN) % NT == 0 || BM + BN < NT, "whole scale rows");
    static_assert(!ENDS || BM + BN <= NT, "a row's end for a thread");
    static_assert(2 * STAGE <= 160 * 1024 - 64 && NW * MX4_STORE_LDS<TN> <= 2 * STAGE, "LDS");
    __shared__ __attribute__((aligned(16))) char ring[2 * STAGE];
    __shared__ int is_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wave_u = __builtin_amdgcn_readfirstlane(wave);
    const int wm = wave / WGN, wn = wave % WGN, l = lane & 31, h = lane >> 5;

    Mx4Part p;
    if (!mx4_part<BM, BN, SPLIT>(a, p)) return;
    const int e = p.e, begin = p.begin, M = p.M, m0 = p.m0, n0 = p.n0, N = a.N, ktiles = p.live ? a.ktiles : 0;
    const int kt0 = SPLIT ? p.z * a.kt_per_split : 0, kt1 = SPLIT ? min(kt0 + a.kt_per_split, ktiles) : ktiles;

    const char *pa = a.A + (int64_t)(begin + m0) * a.a_rs, *pb = a.Q + (int64_t)e * a.q_es + (int64_t)n0 * a.q_rs;
    const char *psa = a.SA + (int64_t)(begin + m0) * a.sa_rs, *psb = a.S + (int64_t)e * a.s_es + (int64_t)n0 * a.s_rs;
    const uint32_t ring_lds = dtl::lds_addr(ring);
    typename AIO::Src a_src;
    typename BIO::Src b_src;
    if (DIRECT) {
        a_src = AIO::sources(a.a_rs, m0, M, wave, lane);
        b_src = BIO::sources(a.q_rs, n0, N, wave, lane);
    }
    u32x4 ra[DIRECT ? 1 : AIO::CHUNKS], rb[DIRECT ? 1 : BIO::CHUNKS];
    // this thread's rows of scales: A's, then W's
    const char *srow[SROWS];
    int64_t scol[SROWS];
    u32x2 rs[SROWS];
#pragma unroll
    for (int i = 0; i < SROWS; ++i) {
        const int r = min(tid + i * NT, BM + BN - 1);
        const bool is_a = r < BM;
        srow[i] = is_a ? psa + (int64_t)min(r, M - 1 - m0) * a.sa_rs : psb + (int64_t)min(r - BM, N - 1 - n0) * a.s_rs;
        scol[i] = is_a ? a.sa_cs : a.s_cs;
    }
    auto fetch_scales = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < SROWS; ++i) rs[i] = load_scales<RUN>(srow[i], scol[i], kt * 8, a.blocks);
    };
    auto fetch = [&](int stage, int kt) __attribute__((always_inline)) {
        fetch_scales(kt);
        if constexpr (DIRECT) {
            const uint32_t st = ring_lds + (uint32_t)(stage * STAGE);
            AIO::issue(st, a_src, pa + kt * KB, wave_u);
            BIO::issue(st + A_BYTES, b_src, pb + kt * KB, wave_u);
        } else {
            AIO::load(ra, pa, a.a_rs, m0, M, kt * KB, a.row_bytes, tid);
            BIO::load(rb, pb, a.q_rs, n0, N, kt * KB, a.row_bytes, tid);
        }
    };
    // The ragged last tile, DIRECT: chunks begin at row_bytes - 16 (the last word before it) at
    // the latest in the last rows, and anywhere up to the row's end in the others, whose next
    // row is there.
    u32x4 end;                                     // ENDS: of the last row of the operand whose row is this thread's in mend
    auto fetch_ragged = [&](int stage, int kt) __attribute__((always_inline)) {
        fetch_scales(kt);
        if constexpr (ENDS)
            end = *reinterpret_cast<const u32x4_any *>((tid < BM ? pa + (int64_t)(M - 1 - m0) * a.a_rs : pb + (int64_t)(N - 1 - n0) * a.q_rs) + a.row_bytes - 16);
        const uint32_t st = ring_lds + (uint32_t)(stage * STAGE);
        auto issue = [&](auto io, uint32_t lds, const char *base, int64_t stride, int r0, int lim) __attribute__((always_inline)) {
#pragma unroll 1
            for (int j = 0; j < decltype(io)::INSTS; ++j) {
                const int pos = (wave + NW * j) * 64 + lane, row = min(pos >> 3, lim - 1 - r0);
                const int at = kt * KB + (((pos & 7) ^ ((pos >> 4) & 7)) << 4);
                const int most = row == lim - 1 - r0 ? (ENDS ? (a.row_bytes - 16) & ~3 : a.row_bytes - 16) : (a.row_bytes - 1) & ~15;
                dtl::lds_load16(base, (uint32_t)row * (uint32_t)stride + (uint32_t)min(at, most), lds + (uint32_t)((wave_u + NW * j) * 1024));
            }
        };
        issue(AIO(), st, pa, a.a_rs, m0, M);
        issue(BIO(), st + A_BYTES, pb, a.q_rs, n0, N);
    };
    auto put = [&](int stage, int kt) __attribute__((always_inline)) {
        char *st = ring + stage * STAGE;
#pragma unroll
        for (int i = 0; i < SROWS; ++i)
            if (NT * SROWS == BM + BN || tid + i * NT < BM + BN)
                *reinterpret_cast<u32x2 *>(st + SA_OFF + (tid + i * NT) * 8) = place_scales<RUN>(rs[i], kt * 8, a.blocks);
        if constexpr (!DIRECT) {
            AIO::store(st, ra, tid);
            BIO::store(st + A_BYTES, rb, tid);
        }
    };
    // The last chunks of a ragged last tile, DIRECT: see above.
    auto mend = [&](int stage, int kt) __attribute__((always_inline)) {
        const int left = a.row_bytes - kt * KB, n = left & 15;
        if (n == 0) return;
#pragma unroll 1
        for (int r = tid; r < BM + BN; r += NT) {
            const bool is_a = r < BM, last = is_a ? m0 + r >= M - 1 : n0 + r - BM >= N - 1;
            if (is_a && !last) continue;
            u32x4 *p = reinterpret_cast<u32x4 *>(ring + stage * STAGE + (is_a ? 0 : A_BYTES) + chunk_off(is_a ? r : r - BM, left >> 4));
            const u32x4 v = *p;
            *p = last ? down_bytes(ENDS ? end : v, 16 - n) : first_bytes(v, n);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    auto compute = [&](int stage) __attribute__((always_inline)) {
        const char *st = ring + stage * STAGE, *la = st + (wm * WTM + l) * KB, *lb = st + A_BYTES + (wn * WTN + l) * KB;
        uint32_t sa[TM], sb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const uint32_t *>(st + SA_OFF + (wm * WTM + 32 * i + l) * 8 + 4 * h);
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = *reinterpret_cast<const uint32_t *>(st + SB_OFF + (wn * WTN + 32 * j + l) * 8 + 4 * h);
        // fragments are read a step ahead of their use
        u32x4 fa[2][TM], fb[2][TN];
        auto read = [&](int s) __attribute__((always_inline)) {
            const int at = ((4 * h + s) ^ ((l >> 1) & 7)) << 4;
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[s & 1][i] = *reinterpret_cast<const u32x4 *>(la + 32 * i * KB + at);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[s & 1][j] = *reinterpret_cast<const u32x4 *>(lb + 32 * j * KB + at);
        };
        auto step = [&](auto s) __attribute__((always_inline)) {
            constexpr int STEP = decltype(s)::value;
            if (STEP < 3) read(STEP + 1);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma<STEP>(fb[STEP & 1][j], sb[j], fa[STEP & 1][i], sa[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        };
        read(0);
        step(std::integral_constant<int, 0>());
        step(std::integral_constant<int, 1>());
        step(std::integral_constant<int, 2>());
        step(std::integral_constant<int, 3>());
    };

    // tile kt is in LDS, tile kt - 1 has been read
    auto arrive = [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    if (kt0 < kt1) {
        const bool ragged = DIRECT && kt1 * KB > a.row_bytes;   // the last tile
        const int full = kt1 - (ragged ? 1 : 0);
        if (kt0 < full) fetch(kt0 & 1, kt0);
        else fetch_ragged(kt0 & 1, kt0);
        put(kt0 & 1, kt0);
        int kt = kt0;
        for (; kt + 1 < full; ++kt) {
            arrive();
            fetch((kt & 1) ^ 1, kt + 1);
            compute(kt & 1);
            put((kt & 1) ^ 1, kt + 1);
        }
        if (ragged) {
            if (kt < full) {
                arrive();
                fetch_ragged((kt & 1) ^ 1, kt + 1);
                compute(kt & 1);
                put((kt & 1) ^ 1, kt + 1);
                ++kt;
            }
            arrive();
            mend(kt & 1, kt);
        }
        arrive();
        compute(kt & 1);
    }

    if constexpr (SPLIT) {
        // [tile][piece][element][thread]: every thread adds its own elements, in the order of K
        const int S = a.splits;
        float *part = a.ws + (int64_t)p.t * S * (BM * BN) + tid;
        auto at = [&](int q, int i, int j, int r) __attribute__((always_inline)) { return part + (int64_t)q * (BM * BN) + ((i * TN + j) * 16 + r) * NT; };
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) __hip_atomic_store(at(p.z, i, j, r), acc[i][j][r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) is_last = take_last_ticket(a.counters + p.t, S);
        __syncthreads();
        if (!is_last) return;
#pragma unroll 1
        for (int q = 0; q < S; ++q) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    float v[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) v[r] = __hip_atomic_load(at(q, i, j, r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] = q == 0 ? v[r] : acc[i][j][r] + v[r];
                }
        }
        if (tid == 0) __hip_atomic_store(a.counters + p.t, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();                               // every wave has read its last tile
    mx4_store<TM, TN>(a, p, acc, wm * WTM, wn * WTN, lane, ring + wave * MX4_STORE_LDS<TN>);
}

}  // namespace

hipError_t launch_mx4_gemm(int tile, int load, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    const bool ends = a.row_bytes % 4 != 0;
#define DG_TILE(B, GM, GN, L, R, S) hipLaunchKernelGGL((mx4_tile<B, B, GM, GN, L, R, S>), dim3((unsigned)units), dim3(64 * GM * GN), 0, s, a)
#define DG_64(L, R)                                      \
    do {                                                 \
        if (a.splits > 1) DG_TILE(64, 2, 2, L, R, true); \
        else DG_TILE(64, 2, 2, L, R, false);             \
    } while (0)
    if (tile != MX4_T64 && a.splits > 1) return hipErrorInvalidValue;
    if (tile == MX4_T256 && load == MX4_DIRECT) {
        if (ends) DG_TILE(256, 2, 4, WORDS_ENDS, true, false);
        else DG_TILE(256, 2, 4, WORDS, true, false);
    } else if (tile == MX4_T128 && load == MX4_DIRECT) {
        if (ends) DG_TILE(128, 2, 2, WORDS_ENDS, true, false);
        else DG_TILE(128, 2, 2, WORDS, true, false);
    } else if (tile == MX4_T128 && load == MX4_BYTES) DG_TILE(128, 2, 2, REGS, true, false);
    else if (tile == MX4_T64 && load == MX4_DIRECT) {
        if (ends) DG_64(WORDS_ENDS, true);
        else DG_64(WORDS, true);
    } else if (tile == MX4_T64 && load == MX4_BYTES) DG_64(REGS, true);
    else if (tile == MX4_T64 && load == MX4_ANY) DG_64(REGS, false);
    else return hipErrorInvalidValue;
#undef DG_64
#undef DG_TILE
    return hipGetLastError();
}

}  // namespace dg
