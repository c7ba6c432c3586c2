// mx4_ring.hip -- products of two MXFP4 operands (see mx4_gemm.hip) whose K is a multiple
// of 512 and whose rows and scale rows begin at multiples of 16 bytes: large tiles whose
// loads, fragment reads and matrix instructions overlap.
//
// What bounds it (4096 x 4096 x 4096: 43 us, 3.2 PFLOP/s; 8192^3: 274 us, 4.0): the matrix
// cores on operands like these run at 1.65 to 1.75 GHz for power (register-only loops of
// 32x32x64 instructions: 9.6 PFLOP/s on zeros, 6.5 on random codes), where the loop
// without its loads takes 2330 cycles for a tile of K and its matrix instructions alone
// 2050; the loads raise that to 3100 to 3400.  The sums leave in 6 us more, all CUs at
// once, at 5 TB/s.  Tried and left: four stages of 128 elements, whose rows of 64 bytes
// cost twice the line requests (8192^3 307 us), 4 waves of 128 x 128 (304), slots freed a
// step earlier (299), the loads on 4 of the waves or 2 (289, 302).
#include "device_common.hpp"
#include "gemm_dtl.hpp"
#include "mx4_tile.hpp"

namespace dg {
namespace {

constexpr int KB = 128;          // bytes of K in a tile: 256 elements, 8 blocks

// A load to LDS as dtl::lds_load16, which other memory accesses may cross: the barriers
// order them.
__device__ __forceinline__ void load_lds(const char *base, uint32_t off, uint32_t a) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(a), "v"(off), "s"(base) : "m0");
}

template <int N> using Int = std::integral_constant<int, N>;

// BM x BN tiles, waves WGM x WGN.
// LDS holds two tiles of K and the scales of two groups of 512 elements (16 bytes a row,
// one load: a load of a few bytes of each row costs as many line requests as one of all
// its codes).  K order within a tile as in mx4_gemm.hip: four steps, lanes 0-31 blocks 0
// to 3, lanes 32-63 blocks 4 to 7.
//  - Fragments are read a step ahead of their use, the next tile's first ones in a tile's
//    last step.  The barrier before that step says that every wave has read the tile and
//    that the next one has arrived; the loads of the tile after that go into the freed
//    slot, between the matrix instructions.
//  - 16-byte chunks of a row are XOR-swizzled by row / 2, so that the 16 rows whose reads
//    of 16 bytes share a cycle cover all 64 banks (by row: twice the cycles).
template <int BM, int BN, int WGM, int WGN>
__global__ void __launch_bounds__(64 * WGM * WGN) mx4_ring(Mx4GemmArgs a) {
    constexpr int NW = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 32, TN = WTN / 32;
    constexpr int B_OFF = BM * KB, SLOT = B_OFF + BN * KB, S_OFF = 2 * SLOT, SBUF = (BM + BN) * 16;
    constexpr int AI = BM * 8 / 64 / NW, CI = AI + BN * 8 / 64 / NW, SI = (BM + BN) / 64 / NW, F = TM + TN;
    static_assert(BM * 8 % (64 * NW) == 0 && BN * 8 % (64 * NW) == 0 && (BM + BN) % (64 * NW) == 0 && BM % 64 == 0, "whole loads");
    static_assert(2 * SLOT + 2 * SBUF <= 160 * 1024 && NW * MX4_STORE_LDS<TN> <= 2 * SLOT, "LDS");
    __shared__ __attribute__((aligned(16))) char lds[2 * SLOT + 2 * SBUF];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN, l = lane & 31, h = lane >> 5;
    Mx4Part p;
    if (!mx4_part<BM, BN>(a, p)) return;
    const int tiles = p.live ? a.ktiles : 0;       // even

    const char *pa = a.A + (int64_t)(p.begin + p.m0) * a.a_rs, *pb = a.Q + (int64_t)p.e * a.q_es + (int64_t)p.n0 * a.q_rs;
    const char *psa = a.SA + (int64_t)(p.begin + p.m0) * a.sa_rs, *psb = a.S + (int64_t)p.e * a.s_es + (int64_t)p.n0 * a.s_rs;
    const uint32_t lds0 = dtl::lds_addr(lds);
    const int last_a = p.M - 1 - p.m0, last_b = a.N - 1 - p.n0;   // rows past them read these (not stored)
    uint32_t off[CI], s_off[SI];
#pragma unroll
    for (int j = 0; j < CI; ++j) {
        const int pos = (wave + NW * (j < AI ? j : j - AI)) * 64 + lane, row = pos >> 3;
        off[j] = (uint32_t)min(row, j < AI ? last_a : last_b) * (uint32_t)(j < AI ? a.a_rs : a.q_rs) + (((pos & 7) ^ ((row >> 1) & 7)) << 4);
    }
#pragma unroll
    for (int j = 0; j < SI; ++j) {
        const int r = (wave + NW * j) * 64 + lane;
        s_off[j] = r < BM ? (uint32_t)min(r, last_a) * (uint32_t)a.sa_rs : (uint32_t)min(r - BM, last_b) * (uint32_t)a.s_rs;
    }
    auto load = [&](int j, int slot, int kt) __attribute__((always_inline)) {   // load j of the wave's for tile kt
        const uint32_t to = lds0 + (uint32_t)(slot * SLOT);
        if (j < AI) load_lds(pa + (int64_t)kt * KB, off[j], to + (uint32_t)((wave + NW * j) * 1024));
        else load_lds(pb + (int64_t)kt * KB, off[j], to + B_OFF + (uint32_t)((wave + NW * (j - AI)) * 1024));
    };
    auto load_scales = [&](int g) __attribute__((always_inline)) {              // of tiles 2 g and 2 g + 1
#pragma unroll
        for (int j = 0; j < SI; ++j)
            load_lds(((wave + NW * j) * 64 < BM ? psa : psb) + (int64_t)g * 16, s_off[j], lds0 + S_OFF + (uint32_t)((g & 1) * SBUF + (wave + NW * j) * 1024));
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    u32x4 fa[2][TM], fb[2][TN];                    // of even and odd steps
    uint32_t sa[2][TM], sb[2][TN];                 // of even and odd tiles
    const int ra = (wm * WTM + l) * KB, rb = B_OFF + (wn * WTN + l) * KB;
    const int rsa = S_OFF + (wm * WTM + l) * 16 + 4 * h, rsb = S_OFF + (BM + wn * WTN + l) * 16 + 4 * h;
    auto read = [&](int step, int k, int slot) __attribute__((always_inline)) {   // fragment k of a step: W's, then A's
        const int at = slot * SLOT + (((4 * h + step) ^ ((l >> 1) & 7)) << 4);
        if (k < TN) fb[step & 1][k] = *reinterpret_cast<const u32x4 *>(lds + rb + 32 * k * KB + at);
        else fa[step & 1][k - TN] = *reinterpret_cast<const u32x4 *>(lds + ra + 32 * (k - TN) * KB + at);
    };
    auto read_scale = [&](int k, int kt) __attribute__((always_inline)) {
        const int at = ((kt >> 1) & 1) * SBUF + (kt & 1) * 8;
        if (k < TN) sb[kt & 1][k] = *reinterpret_cast<const uint32_t *>(lds + rsb + 512 * k + at);
        else sa[kt & 1][k - TN] = *reinterpret_cast<const uint32_t *>(lds + rsa + 512 * (k - TN) + at);
    };
    // A step of tile kt (in slot PAR = kt % 2): in each of TM parts some of the next step's
    // fragments, REFILL some loads of tile kt + 2, and TN matrix instructions.  The order
    // is fixed: left to itself the compiler collects the reads and the instructions.
    auto step = [&](auto s, auto par, auto refill, int kt) __attribute__((always_inline)) {
        constexpr int STEP = decltype(s)::value, PAR = decltype(par)::value;
        constexpr int READS = (F + TM - 1) / TM, LOADS = decltype(refill)::value ? (CI + TM - 1) / TM : 0;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int k = i * READS; k < (i + 1) * READS && k < F; ++k) {
                if (STEP == 3) {
                    read_scale(k, ((kt + 1) & ~1) + (PAR ^ 1));
                    read(0, k, PAR ^ 1);
                } else {
                    read(STEP + 1, k, PAR);
                }
            }
#pragma unroll
            for (int j = i * LOADS; j < (i + 1) * LOADS && j < CI; ++j) load(j, PAR, kt + 2);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma<STEP>(fb[STEP & 1][j], sb[PAR][j], fa[STEP & 1][i], sa[PAR][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto arrive = [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    auto tile = [&](auto par, auto refill, auto more, int kt) __attribute__((always_inline)) {
        step(Int<0>(), par, Int<0>(), kt);
        step(Int<1>(), par, Int<0>(), kt);
        step(Int<2>(), par, Int<0>(), kt);
        if constexpr (decltype(more)::value) arrive();
        step(Int<3>(), par, refill, kt);           // (the last tile's reads find what is there)
    };

    if (tiles > 0) {
        load_scales(0);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < CI; ++j) load(j, t, t);
        arrive();
#pragma unroll
        for (int k = 0; k < F; ++k) {
            read_scale(k, 0);
            read(0, k, 0);
        }
        int kt = 0;
#pragma unroll 1
        for (; kt + 2 < tiles; kt += 2) {
            load_scales((kt >> 1) + 1);
            tile(Int<0>(), Int<1>(), Int<1>(), kt);
            tile(Int<1>(), Int<1>(), Int<1>(), kt + 1);
        }
        tile(Int<0>(), Int<0>(), Int<1>(), kt);
        tile(Int<1>(), Int<0>(), Int<0>(), kt + 1);
    }
    arrive();                                      // every wave has read its last fragments
    mx4_store<TM, TN>(a, p, acc, wm * WTM, wn * WTN, lane, lds + wave * MX4_STORE_LDS<TN>);
}

}  // namespace

hipError_t launch_mx4_ring(int tile, const Mx4GemmArgs &a, int64_t units, hipStream_t s) {
    if (tile == MX4_T256) hipLaunchKernelGGL((mx4_ring<256, 256, 2, 4>), dim3((unsigned)units), dim3(512), 0, s, a);
    else if (tile == MX4_T128) hipLaunchKernelGGL((mx4_ring<128, 128, 2, 2>), dim3((unsigned)units), dim3(256), 0, s, a);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace dg
