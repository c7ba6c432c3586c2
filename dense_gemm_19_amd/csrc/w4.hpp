// w4.hpp -- products with 4-bit weights and group scales, for one weight matrix
// or for the experts of a mixture (templates; instantiated by w4.hip, and by
// w4_mx.hip for microscaled weights):
//
//   C[m][n] = act(sum over k of A[m][k] * s[n][k/G] * (q[n][k] - z[n][k/G]))
//
// Codes and zero points are whole numbers of at most 255, exact in FP16 and
// BF16, and so are their differences, which go to the matrix cores; each scale
// group's sum is formed in FP32 there and then enters the FP32 accumulator times its
// scale, once.  No weight is rounded.
//
// Microscaled weights (SB = 1, a byte per scale) differ in two places only: a code is
// an E2M1 number, exact in both types, which gfx950 converts two at a time, and a
// group's scale is the power of two that its byte names.  BF16 codes are converted times
// their scale (block_scale): a group's sum without it may pass FP32.
//
// Bound by the bytes of the codes where few rows meet many weights (half a byte
// per weight), by the latency of the loads and the instructions fetched for small
// calls, by LDS reads and the vector ALUs that decode for more rows.
#pragma once
#include "bytes.hpp"
#include "device_common.hpp"
#include "e8m0.hpp"
#include "gemm_dtl.hpp"
#include "moe.hpp"
#include "moe_slot.hpp"

namespace dg {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int UNIT = 256;        // K elements of a unit: 128 bytes of a weight row, a whole cache line
constexpr int UNIT_LDS = 2048;   // its 16 rows

template <int IN>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) { return dtl::mfma16<IN>(a, b, c); }

// 8 codes (k in nibble k), a byte each, in the order of k.
__device__ __forceinline__ u32x2 code_bytes(uint32_t x) {
    const uint32_t lo = x & 0x0f0f0f0fu, hi = (x >> 4) & 0x0f0f0f0fu;
    return u32x2{__builtin_amdgcn_perm(hi, lo, 0x05010400u), __builtin_amdgcn_perm(hi, lo, 0x07030602u)};
}

// 8 codes minus z as FP16 or BF16, exactly (a difference has at most 8 significant
// bits).  A byte q under 0x64 is the FP16 number 1024 + q, so one packed add gives
// two differences.  BF16 has no packed arithmetic here: a code under a zero byte is
// the FP16 number q * 2^-24, a mixed FP16 -> FP32 multiply-add makes it q - z, and
// the upper halves of two are the pair (19 instructions for 8 codes).
template <int IN>
__device__ __forceinline__ u32x4 decode(uint32_t x, float z) {
    u32x4 out;
    if (IN == IN_F16) {
        const u32x2 e = code_bytes(x);
        const _Float16 c = (_Float16)(-1024.0f - z);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = __builtin_amdgcn_perm(0x64646464u, e[j / 2], j & 1 ? 0x04030402u : 0x04010400u);
            out[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v) + f16x2{c, c});
        }
    } else {
        const uint32_t lo = x & 0x0f0f0f0fu, hi = (x >> 4) & 0x0f0f0f0fu;
        float unit = 0x1p24f;
        asm("" : "+s"(unit));   // keeps the multiply, so that conversion and add are one instruction
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(hi, lo, 0x0c040c00u + 0x00010001u * j));
            const float p = fmaf((float)v[0], unit, -z), q = fmaf((float)v[1], unit, -z);
            out[j] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, q), __builtin_bit_cast(uint32_t, p), 0x07060302u);
        }
    }
    return out;
}

// 8 E2M1 codes times a scale as FP16 or BF16 (4 instructions).
template <int IN>
__device__ __forceinline__ u32x4 decode_e2m1(uint32_t x, float scale) {
    u32x4 out;
    auto pair = [&](auto j) { if constexpr (IN == IN_F16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, scale, decltype(j)::value));
                              else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, decltype(j)::value)); };
    out[0] = pair(std::integral_constant<int, 0>());
    out[1] = pair(std::integral_constant<int, 1>());
    out[2] = pair(std::integral_constant<int, 2>());
    out[3] = pair(std::integral_constant<int, 3>());
    return out;
}

// An offset that every lane shares, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// The kernel's arguments read again: what only the end needs does not hold
// scalar registers over the main loop.
__device__ __forceinline__ const W4Args &arguments() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const W4Args *)p;
}

__device__ __forceinline__ void wait_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// At most n vector loads of this wave in flight.
#define DG_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | (0x7 << 4) | (0xF << 8))
// The same for a wave-uniform n (the instruction holds a constant): one of the
// values there are, at most n (all sixteen up to 15 took as long).
__device__ __forceinline__ void wait_loads(int n) {
    if (n >= 8) {
        if (n >= 16) {
            if (n >= 24) DG_VM(24);
            else DG_VM(16);
        } else {
            if (n >= 12) DG_VM(12);
            else DG_VM(8);
        }
    } else {
        if (n >= 4) {
            if (n >= 6) DG_VM(6);
            else DG_VM(4);
        } else {
            if (n >= 3) DG_VM(3);
            else DG_VM(0);
        }
    }
}

// This workgroup's rows, columns, expert and piece of K.
struct Part { int e, begin, rows, nk, m0, n0, here, cols, c0, c1, unit, z; };

template <int TM>
__device__ __forceinline__ bool find_part(const W4Args &a, Part &p) {
    constexpr int MR = 16 * TM, CHUNK = w4_chunk(TM);
    p.e = 0; p.begin = 0; p.rows = a.M; p.nk = a.K; p.z = 0;
    if (a.offsets) {
        moe::Slot s;
        if (!moe::find_slot<MR>(a.offsets, a.o_s, a.E, a.M, a.slabs, a.units, blockIdx.x, s)) return false;
        p.e = s.e; p.begin = s.begin; p.rows = s.rows; p.unit = s.unit;
        if (p.e == a.E) { p.e = 0; p.nk = 0; }   // rows of no expert: zero
    } else {
        p.unit = moe::xcd_run(blockIdx.x, a.units);
        if (a.splits > 1) {
            const int u = p.unit / a.splits;
            p.z = p.unit - u * a.splits;
            p.unit = u;
        }
    }
    const int tiles_m = (p.rows + MR - 1) / MR;
    int tm = 0, tn = p.unit;
    if (tiles_m > 1) {
        tn = p.unit / tiles_m;
        tm = p.unit - tn * tiles_m;
    }
    p.m0 = tm * MR;
    p.n0 = tn * w4_cols(TM);
    p.here = min(p.rows - p.m0, MR);               // rows of this tile
    p.cols = min(w4_cols(TM), a.N - p.n0);
    p.c0 = p.z * a.chunks;
    p.c1 = min(p.c0 + a.chunks, (p.nk + CHUNK - 1) / CHUNK);
    return true;
}

// The waves' sums added, the pieces' too, activated and stored.
// Register (t, r) of lane (l, g) of wave (wk, wn) is C[16 t + 4 g + r][16 wn + l].
template <int TM>
__device__ __forceinline__ void finish(const Part &p, const f32x4 (&acc)[TM], char *lds, int *is_last, int tid, int wk, int wn) {
    constexpr int WN = w4_cols(TM) / 16, WK = WAVES / WN, REGS = TM * WN * 256, PER = REGS / NT;
    const int lane = tid & 63;
    float *red = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wk * REGS + (wn * TM + t) * 256 + r * 64 + lane] = acc[t][r];
    __syncthreads();
    float v[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        v[u] = red[u * NT + tid];
#pragma unroll
        for (int w = 1; w < WK; ++w) v[u] += red[w * REGS + u * NT + tid];
    }
    const W4Args &o = arguments();
    if (o.splits > 1) {
        float *part = o.ws + (int64_t)p.unit * o.splits * REGS + tid;
#pragma unroll
        for (int u = 0; u < PER; ++u)
            __hip_atomic_store(part + p.z * REGS + u * NT, v[u], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) *is_last = take_last_ticket(o.counters + p.unit, o.splits);
        __syncthreads();
        if (!*is_last) return;
        // in the order of K, QB pieces' loads at a time (past the last: it again)
        constexpr int QB = PER == 1 ? 8 : 4;
#pragma unroll 1
        for (int q0 = 0; q0 < o.splits; q0 += QB) {
            float x[QB][PER];
#pragma unroll
            for (int q = 0; q < QB; ++q)
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    x[q][u] = __hip_atomic_load(part + min(q0 + q, o.splits - 1) * REGS + u * NT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int q = 0; q < QB; ++q)
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (q0 + q < o.splits) v[u] = q0 + q == 0 ? x[q][u] : v[u] + x[q][u];
        }
        if (tid == 0) __hip_atomic_store(o.counters + p.unit, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if constexpr (PER == 1) {
        const int t = (tid >> 8) % TM, m = p.m0 + 16 * t + 4 * ((lane >> 4) & 3) + ((tid >> 6) & 3), n = p.n0 + 16 * ((tid >> 8) / TM) + (lane & 15);
        if (m >= p.rows || n >= o.N) return;
        store_out(o.C + (int64_t)(p.begin + m) * o.c_rs + (int64_t)n * o.c_cs, o.out_kind, activate(o.act, v[0]));
        return;
    }
    // through LDS once more: a thread stores 4 columns of a row
#pragma unroll
    for (int u = 0; u < PER; ++u) red[u * NT + tid] = v[u];
    __syncthreads();
    const int esize = o.out_kind == OUT_F32 ? 4 : 2;
#pragma unroll 1
    for (int i = tid; i < REGS / 4; i += NT) {
        const int t = (i >> 6) % TM, r = (i >> 4) & 3, m = p.m0 + 16 * t + 4 * ((i >> 2) & 3) + r;
        const int n = p.n0 + 16 * ((i >> 6) / TM) + 4 * (i & 3);
        if (m >= p.rows || n >= o.N) continue;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = activate(o.act, red[4 * i + e]);
        char *c = o.C + (int64_t)(p.begin + m) * o.c_rs + (int64_t)n * o.c_cs;
        if (o.c_cs == esize && n + 3 < o.N) {
            store_out4(c, o.out_kind, y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < o.N) store_out(c + e * o.c_cs, o.out_kind, y[e]);
        }
    }
}

// The usual layout (W4Args::whole): rows of A and of the codes in whole, aligned
// 16-byte pieces, scales and zero points one run of whole aligned words that LDS holds
// at once.
// A workgroup computes 16 * TM rows x 16 * WN columns over its chunks of K.  Its
// 8 waves are WK x WN: wave (wk, wn) takes 16 columns and unit wk of every chunk.
//  - Everything goes to LDS by load-to-LDS instructions, which cost no registers
//    and fetch codes in whole cache lines (8 rows of 128 bytes each): scales and
//    zero points first, then chunk after chunk the rows of A (all waves together)
//    and the wave's own unit of codes, `ahead` chunks deep.
//  - Loads return in order and every wave issues the same number per chunk, so it
//    waits for exactly the chunk at hand.
//  - Address arithmetic is what the vector and scalar units have left to do beside
//    the decoding, and it bounds few rows: lane offsets are kept, a fetch only adds
//    scalars to them.
// Pieces of 16 bytes are XOR-swizzled by their row in LDS (fetched so from memory)
// and rows of scales are an odd number of words apart, so that the 16 rows of a
// read fall on distinct banks.
// Measured: 1 x 14336 x 4096 BF16 12.0 us (zero points as a second product of the
// same rows, which needs 9 instructions for 8 codes, takes 10.6 but rounds at the size
// of |A|(q + z): sums of zero weights were not zero), 33 x 4096 x 14336 FP16 19.1 us,
// 16 rows over 16 experts of 7168 x 4096 50 to 60 us, the codes at 4.6 to 5.6 TB/s.
template <int IN, int TM, int GV, int SB, bool ZP>
__global__ void __launch_bounds__(NT, TM == 1 ? 4 : 2) w4_whole(W4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // codes, A, scales, zero points; then the waves' sums
    __shared__ int is_last;
    constexpr int WN = w4_cols(TM) / 16, WK = WAVES / WN, CHUNK = w4_chunk(TM), ROW = CHUNK * 2, PR = ROW / 16;
    static_assert(WK * UNIT == CHUNK, "a unit per wave");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK;
    const int l = lane & 15, g = lane >> 4;
    Part p;
    if (!find_part<TM>(a, p)) return;
    const int nk = p.nk, c0 = p.c0, c1 = p.c1, here = p.here;

    const char *qb = a.Q + uniform((int64_t)p.e * a.q_es + (int64_t)p.n0 * a.q_rs);
    const char *ab = a.A + uniform((int64_t)(p.begin + p.m0) * a.a_rs);
    const int a_bytes = here * ROW;                // a chunk of the rows there are
    // Chunks in LDS at a time: a.depth units, as far as A's part holds the rows; all
    // of them are issued before the first is computed where that is all there are,
    // else one less, since a slot is refilled while the next one is computed.
    const int bufs = a.a_lds >= 4 * a_bytes ? 4 : a.a_lds >= 3 * a_bytes ? 3 : a.a_lds >= 2 * a_bytes ? 2 : 1;
    const int slots = min(bufs, a.depth), lead = c1 - c0 <= slots ? slots : slots - 1;
    const uint32_t lds0 = dtl::lds_addr(lds);
    const int q_ring = wave * (a.depth * UNIT_LDS), a_ring = WAVES * a.depth * UNIT_LDS;
    const int s_at = a_ring + a.a_lds, z_at = s_at + ((w4_cols(TM) * a.s_pitch + 255) & ~255);

    // Scales (and zero points) of this piece's groups from g0 on: the aligned words
    // that hold column r's, word d at r * pitch + 4 d, the pitch an odd number of
    // words.  The first byte is the (r * rs + from)'th of them, modulo 4.
    // group of 32-element step `step` of K: see w4_stream
    auto group_of = [&](int step) { return min((int)(a.g_mul ? __umulhi((uint32_t)step, a.g_mul) : (uint32_t)step), a.groups - 1); };
    const int g0 = __builtin_amdgcn_readfirstlane(group_of(c0 * (CHUNK / 32)) & ~3);
    auto words = [&](const char *base, int64_t rs, int pitch, uint32_t mul, int at, int bytes) __attribute__((always_inline)) {
        const int per = pitch / 4, total = w4_cols(TM) * per;
        const uint32_t from = (uint32_t)(uintptr_t)base & 3u;
        base -= from;
#pragma unroll 1
        for (int j = wave; j * 64 < total; j += WAVES) {
            const int i = j * 64 + lane, r = (int)__umulhi((uint32_t)i, mul), d = i - r * per;
            const uint32_t row = (uint32_t)min(r, p.cols - 1) * (uint32_t)rs + from;
            dtl::lds_load4(base, (row & ~3u) + min(4u * (uint32_t)d, ((row & 3u) + (uint32_t)bytes - 1u) & ~3u),
                           __builtin_amdgcn_readfirstlane(lds0 + at + j * 256));
        }
    };
    const char *s_base = a.S + uniform((int64_t)p.e * a.s_es + (int64_t)p.n0 * a.s_rs + (int64_t)g0 * SB);
    const char *z_base = ZP ? a.Z + uniform((int64_t)p.e * a.z_es + (int64_t)p.n0 * a.z_rs + g0) : nullptr;
    if (c0 < c1) {
        const int n = min(a.groups - g0, a.seg_groups);
        words(s_base, a.s_rs, a.s_pitch, a.s_mul, s_at, n * SB);
        if (ZP) words(z_base, a.z_rs, a.z_pitch, a.z_mul, z_at, n);
    }

    // Chunk c into slot `slot` of both rings.  Codes: piece i of row r of a unit at
    // r * 128 + 16 * (i ^ (r & 7)); load h fills rows 8 h .. 8 h + 7.  A: piece i of
    // row r at r * ROW + 16 * (i ^ (r & 15)).
    const int q_row = lane >> 3, q_piece = 16 * ((lane & 7) ^ q_row);
    const uint32_t q_off[2] = {(uint32_t)min(16 * wn + q_row, p.cols - 1) * (uint32_t)a.q_rs,
                               (uint32_t)min(16 * wn + q_row + 8, p.cols - 1) * (uint32_t)a.q_rs};
    const int q_bytes = nk / 2;
    constexpr int LPR = PR / 64;                   // loads of a wave in a row of A
    static_assert(PR % 64 == 0, "no load crosses a row");
    const int a_loads = (a_bytes / 1024 - wave + WAVES - 1) / WAVES;   // of a chunk, by this wave
    auto issue = [&](int c, int slot) __attribute__((always_inline)) {
        const int last = nk * 2 - c * ROW - 16;    // A's pieces past K read the last one (cleared below)
        const char *ac = ab + (int64_t)c * ROW;
        uint32_t dst = lds0 + a_ring + slot * a_bytes + wave * 1024;
#pragma unroll 1
        for (int j = wave; j * 1024 < a_bytes; j += WAVES) {
            const int r = j / LPR;
            const uint32_t piece = (uint32_t)min(16 * (lane ^ (r & 15)) + j % LPR * 1024, last);
            dtl::lds_load16(ac + (int64_t)r * a.a_rs, piece, __builtin_amdgcn_readfirstlane(dst));
            dst += WAVES * 1024;
        }
        const int at = c * (CHUNK / 2) + wk * (UNIT / 2);
        const bool in = at < q_bytes;              // a unit past K: its first line again, to keep the count of loads
        const char *base = qb + (in ? at : 0);
        const uint32_t piece = (uint32_t)min(q_piece, in ? q_bytes - at - 16 : 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) dtl::lds_load16(base, q_off[h] + piece, lds0 + q_ring + slot * UNIT_LDS + h * 1024);
    };
    // The K elements past the end of a unit that the loads of A left there
    auto clear = [&](int slot) __attribute__((always_inline)) {
        const int p0 = (nk % CHUNK) / 8, n = UNIT / 8 - p0 % (UNIT / 8);
#pragma unroll 1
        for (int j = tid; j < here * n; j += NT) {
            const int r = j / n, q = p0 + j % n;
            *reinterpret_cast<u32x4 *>(lds + a_ring + slot * a_bytes + r * ROW + 16 * (q ^ (r & 15))) = u32x4{0u, 0u, 0u, 0u};
        }
    };

    f32x4 acc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // this lane's addresses: words of codes, fragments of A (rows past the tile: one of it again)
    const int q_lane = q_ring + l * 128 + 4 * g, q_swz = 16 * (l & 7);
    int fa_at[4][TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int row = min(16 * t + l, here - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) fa_at[i][t] = a_ring + wk * 512 + row * ROW + 16 * ((4 * i + g) ^ (row & 15));
    }
    const uint32_t col = (uint32_t)min(16 * wn + l, p.cols - 1);
    const char *ls = lds + s_at + (16 * wn + l) * a.s_pitch + ((col * (uint32_t)a.s_rs + (uint32_t)(uintptr_t)s_base) & 3u);
    const char *lz = lds + z_at + (16 * wn + l) * a.z_pitch + ((col * (uint32_t)a.z_rs + (uint32_t)(uintptr_t)z_base) & 3u);
    auto compute = [&](int c, int slot) __attribute__((always_inline)) {
        const int k0 = c * CHUNK + wk * UNIT, qs = q_lane + slot * UNIT_LDS, as = slot * a_bytes;
        uint32_t qw[8];                            // lane row g: bytes 4 g .. + 3 of the 16 of a 32-element step
#pragma unroll
        for (int i = 0; i < 8; ++i) qw[i] = *reinterpret_cast<const uint32_t *>(lds + qs + (q_swz ^ (16 * i)));
#pragma unroll
        for (int w = 0; w < 2; ++w) {              // 128 elements each
            if (k0 + 128 * w >= nk) break;
            const uint32_t *q = qw + 4 * w;
            u32x4 fa[4][TM];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < TM; ++t) fa[i][t] = *reinterpret_cast<const u32x4 *>(lds + as + fa_at[i][t] + 256 * w);
            float s[GV], zp[GV], in[GV];           // (in: microscaled, the codes' part of the scale)
#pragma unroll
            for (int v = 0; v < GV; ++v) {
                const int gi = group_of(k0 / 32 + 4 * w + v * (4 / GV)) - g0;
                if constexpr (SB == 1) {
                    const BlockScale b = block_scale<IN>(*reinterpret_cast<const uint8_t *>(ls + gi));
                    s[v] = b.out;
                    in[v] = b.in;
                } else if constexpr (SB == 4) s[v] = *reinterpret_cast<const float *>(ls + 4 * gi);
                else {
                    const uint16_t h = *reinterpret_cast<const uint16_t *>(ls + 2 * gi);
                    s[v] = a.s_kind == OUT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
                }
                zp[v] = ZP ? (float)*reinterpret_cast<const uint8_t *>(lz + gi) : 8.0f;
            }
            // groups past K (these elements hold its end): their sums are zero, but
            // zero times an infinite last scale would be NaN
            if (GV > 1 && k0 + 128 * (w + 1) > nk) {
#pragma unroll
                for (int v = 1; v < GV; ++v)
                    if (k0 + 128 * w + v * (128 / GV) >= nk) s[v] = 0.0f;
            }
            f32x4 blk[TM];                         // a group's sums
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int PER = 4 / GV;        // 32-wide steps of a group
                const bool first = i % PER == 0;
                const u32x4 fb = SB == 1 ? decode_e2m1<IN>(q[i], in[i / PER]) : decode<IN>(q[i], zp[i / PER]);
#pragma unroll
                for (int t = 0; t < TM; ++t) blk[t] = mfma<IN>(fa[i][t], fb, first ? f32x4{0.f, 0.f, 0.f, 0.f} : blk[t]);
                if (i % PER == PER - 1) {
#pragma unroll
                    for (int t = 0; t < TM; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[t][r] = fmaf(s[i / PER], blk[t][r], acc[t][r]);
                }
            }
        }
    };

    // Chunk c + lead is issued while chunk c is computed (lead 0: chunk c just
    // before it is), into a slot that every wave has left by then.  The first trips
    // only issue: one place for it keeps the code, which a short call fetches anew,
    // small.
    int next = 0, slot = 0;
    for (int c = c0 - lead; c < c1; ++c) {
        if (c >= c0) {
            wait_loads(min(lead - 1, c1 - 1 - c) * (a_loads + 2));   // chunk c has landed
            wait_barrier();                        // in every wave, and every wave is done with chunk c - 1
        }
        if (c + lead < c1) {
            issue(c + lead, next);
            next = next + 1 == slots ? 0 : next + 1;
        }
        if (c < c0) continue;
        if (lead == 0) {
            DG_VM(0);
            wait_barrier();
        }
        if ((c + 1) * CHUNK > nk && nk % UNIT != 0) {
            clear(slot);
            wait_barrier();
        }
        compute(c, slot);
        slot = slot + 1 == slots ? 0 : slot + 1;
    }
    wait_barrier();                                // every wave has read its last chunk
    finish<TM>(p, acc, lds, &is_last, tid, wk, wn);
}

// Any other layout: the same split of the work, everything through registers, at
// any alignment.  Each wave loads its next unit of codes before it computes the
// one at hand, and A's rows are in LDS whole where they fit, else a chunk at a time
// with the next one's pieces on their way in registers.
// GV: scale groups that 128 K elements can touch (1, 2 or 4); SB: bytes of a scale.
template <int IN, int TM, int GV, int SB, bool ZP>
__global__ void __launch_bounds__(NT, TM == 1 ? 4 : 2) w4_stream(W4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // codes, A, scales, zero points; then the waves' sums
    __shared__ int is_last;
    constexpr int WN = w4_cols(TM) / 16, WK = WAVES / WN, CHUNK = w4_chunk(TM), ROW = CHUNK * 2, PR = ROW / 16;
    constexpr int PIECES = 16 * TM * PR / NT;      // of a chunk of a full tile, per thread
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK;
    const int l = lane & 15, g = lane >> 4;
    Part p;
    if (!find_part<TM>(a, p)) return;
    const int nk = p.nk, c0 = p.c0, c1 = p.c1, here = p.here;
    const char *qb = a.Q + uniform((int64_t)p.e * a.q_es + (int64_t)p.n0 * a.q_rs);
    const char *sb = a.S + uniform((int64_t)p.e * a.s_es + (int64_t)p.n0 * a.s_rs);
    const char *zb = ZP ? a.Z + uniform((int64_t)p.e * a.z_es + (int64_t)p.n0 * a.z_rs) : nullptr;
    const char *ab = a.A + uniform((int64_t)(p.begin + p.m0) * a.a_rs);

    // LDS: [wave] code unit, A (a_lds bytes), scales, zero points
    const int a_bytes = here * ROW;
    const bool resident = (int64_t)(c1 - c0) * a_bytes <= a.a_lds;   // all of this piece of A
    char *lq = lds + wave * UNIT_LDS, *la = lds + WAVES * UNIT_LDS, *lsc = la + a.a_lds, *lzp = lsc + 16 * WN * a.s_pitch;

    // Piece i (16 bytes) of row r of a unit at r * 128 + 16 * (i ^ (r & 7)): lane i
    // row 8 h + i / 8, position i % 8 of load h.
    const int q_row = lane >> 3, q_piece = (lane & 7) ^ q_row;
    const uint32_t q_off[2] = {(uint32_t)min(16 * wn + q_row, p.cols - 1) * (uint32_t)a.q_rs,
                               (uint32_t)min(16 * wn + q_row + 8, p.cols - 1) * (uint32_t)a.q_rs};
    const int q_bytes = (nk + 1) / 2;
    // A piece that crosses the row's end is read whole, ending there, and moved down
    // when it is stored (rows of at least 16 bytes; shorter ones byte by byte).
    u32x4 pq[2];
    auto piece_q = [&](int c) { return c * (CHUNK / 2) + wk * (UNIT / 2) + 16 * q_piece; };
    auto load_q = [&](int c) __attribute__((always_inline)) {
        const int at = max(min(piece_q(c), q_bytes - 16), 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (q_bytes >= 16) {
                pq[h] = *reinterpret_cast<const u32x4_any *>(qb + q_off[h] + at);
            } else {
                pq[h] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll 1
                for (int j = q_bytes - 1; j >= 0; --j) {
                    pq[h] = u32x4{pq[h][0] << 8, pq[h][1] << 8 | pq[h][0] >> 24, pq[h][2] << 8 | pq[h][1] >> 24, pq[h][3] << 8 | pq[h][2] >> 24};
                    pq[h][0] |= *reinterpret_cast<const uint8_t *>(qb + q_off[h] + j);
                }
            }
        }
    };
    auto store_q = [&](int c) __attribute__((always_inline)) {
        const int by = min(piece_q(c) - max(min(piece_q(c), q_bytes - 16), 0), 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4 *>(lq + h * 1024 + lane * 16) = by > 0 ? down_bytes(pq[h], by) : pq[h];
    };
    // Chunk c of A: piece i of row r at r * ROW + 16 * (i ^ (r & 15))
    u32x4 pa[PIECES];
    auto load_a = [&](int c) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int i = min(u * NT + tid, here * PR - 1), r = i / PR, k = c * CHUNK + 8 * ((i % PR) ^ (r & 15));
            if (u * NT >= here * PR) break;
            // a piece past the end is read from the last whole one's place and moved down, where there is one
            const int at = min(k, max(nk - 8, 0));
            pa[u] = nk >= 8 ? *reinterpret_cast<const u32x4_any *>(ab + (int64_t)r * a.a_rs + 2 * (int64_t)at)
                            : load_part<2>(ab + (int64_t)r * a.a_rs, 2, nk);
        }
    };
    auto store_a = [&](int c, char *buf) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int i = u * NT + tid;
            if (u * NT >= here * PR) break;
            if (i >= here * PR) continue;
            const int k = c * CHUNK + 8 * ((i % PR) ^ (i / PR & 15)), by = min(k - min(k, max(nk - 8, 0)), 8);
            if (by > 0) pa[u] = down_bytes(pa[u], 2 * by);
            *reinterpret_cast<u32x4 *>(buf + i * 16) = pa[u];
        }
    };
    // Scales and zero points of the groups of `seg` chunks from c on
    auto stage_scales = [&](int c) __attribute__((always_inline)) {
        const int g0 = c * CHUNK / a.G, n = min(a.groups - g0, a.seg_groups);
        const int ps = (n * SB + 15) / 16, pz = (n + 15) / 16;
#pragma unroll 1
        for (int i = tid; i < 16 * WN * ps; i += NT) {
            const int r = i / ps, j = i % ps;
            const char *src = sb + (int64_t)min(r, p.cols - 1) * a.s_rs + (int64_t)(g0 + j * (16 / SB)) * a.s_cs;
            *reinterpret_cast<u32x4 *>(lsc + r * a.s_pitch + 16 * j) = load_part<SB>(src, a.s_cs, n - j * (16 / SB));
        }
        if (ZP) {
#pragma unroll 1
            for (int i = tid; i < 16 * WN * pz; i += NT) {
                const int r = i / pz, j = i % pz;
                const char *src = zb + (int64_t)min(r, p.cols - 1) * a.z_rs + (int64_t)(g0 + 16 * j) * a.z_cs;
                *reinterpret_cast<u32x4 *>(lzp + r * a.z_pitch + 16 * j) = load_part<1>(src, a.z_cs, n - 16 * j);
            }
        }
        return g0;
    };

    f32x4 acc[TM];
    int arow[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        arow[t] = min(16 * t + l, here - 1);       // rows past the tile: one of it again
    }
    // Group of 32-element step `step` of K: step / (G / 32), by the reciprocal
    // 2^32 / (G / 32) rounded up, exact while the product of the two stays below
    // 2^32 (K <= 2^20).
    auto group_of = [&](int step) { return min((int)(a.g_mul ? __umulhi((uint32_t)step, a.g_mul) : (uint32_t)step), a.groups - 1); };
    int seg_g0 = 0;
    auto compute = [&](int c, const char *buf) __attribute__((always_inline)) {
        const int k0 = c * CHUNK + wk * UNIT;
        const char *ls = lsc + (16 * wn + l) * a.s_pitch, *lz = lzp + (16 * wn + l) * a.z_pitch;
#pragma unroll
        for (int w = 0; w < 2; ++w) {              // 128 elements each
            if (k0 + 128 * w >= nk) break;
            uint32_t q[4];                         // lane row g: bytes 4 g .. + 3 of the step's 16
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint32_t *>(lq + l * 128 + 4 * g + 16 * ((4 * w + i) ^ (l & 7)));
            float s[GV], zp[GV], in[GV];           // (in: microscaled, the codes' part of the scale)
#pragma unroll
            for (int v = 0; v < GV; ++v) {
                const int gi = group_of(k0 / 32 + 4 * w + v * (4 / GV)) - seg_g0;
                if constexpr (SB == 1) {
                    const BlockScale b = block_scale<IN>(*reinterpret_cast<const uint8_t *>(ls + gi));
                    s[v] = b.out;
                    in[v] = b.in;
                } else if constexpr (SB == 4) s[v] = *reinterpret_cast<const float *>(ls + 4 * gi);
                else {
                    const uint16_t h = *reinterpret_cast<const uint16_t *>(ls + 2 * gi);
                    s[v] = a.s_kind == OUT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
                }
                zp[v] = ZP ? (float)*reinterpret_cast<const uint8_t *>(lz + gi) : 8.0f;
            }
            // groups past K (these elements hold its end): their sums are zero, but
            // zero times an infinite last scale would be NaN
            if (GV > 1 && k0 + 128 * (w + 1) > nk) {
#pragma unroll
                for (int v = 1; v < GV; ++v)
                    if (k0 + 128 * w + v * (128 / GV) >= nk) s[v] = 0.0f;
            }
            f32x4 blk[TM];                         // a group's sums
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int PER = 4 / GV;        // 32-wide steps of a group
                const u32x4 fb = SB == 1 ? decode_e2m1<IN>(q[i], in[i / PER]) : decode<IN>(q[i], zp[i / PER]);
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    const u32x4 fa = *reinterpret_cast<const u32x4 *>(buf + arow[t] * ROW + 16 * ((wk * 32 + 16 * w + 4 * i + g) ^ (arow[t] & 15)));
                    blk[t] = mfma<IN>(fa, fb, i % PER == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : blk[t]);
                }
                if (i % PER == PER - 1) {
#pragma unroll
                    for (int t = 0; t < TM; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[t][r] = fmaf(s[i / PER], blk[t][r], acc[t][r]);
                }
            }
        }
    };

    if (c0 < c1) load_q(c0);
    for (int c = c0; c < (resident ? c1 : min(c0 + 1, c1)); ++c) {
        load_a(c);
        store_a(c, la + (c - c0) * a_bytes);
    }
    int until = 0;                                 // chunks until the next scales
    for (int c = c0; c < c1; ++c) {
        if (until == 0) {                          // the first chunk, mostly the only time
            if (c > c0) __syncthreads();           // the scales before have been read
            seg_g0 = stage_scales(c);
            until = a.seg;
            __syncthreads();
        }
        --until;
        store_q(c);
        const bool more = c + 1 < c1;
        if (more) {
            load_q(c + 1);
            if (!resident) load_a(c + 1);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's codes are in LDS
        compute(c, resident ? la + (c - c0) * a_bytes : la);
        if (!resident && more) {
            __syncthreads();                       // chunk c has been read
            store_a(c + 1, la);
            __syncthreads();
        }
    }
    __syncthreads();                               // every wave has read its last chunk
    finish<TM>(p, acc, lds, &is_last, tid, wk, wn);
}

template <int IN, int TM, int GV, int SB>
hipError_t launch_t(const W4Args &a, int64_t units, hipStream_t s) {
    auto k = a.whole ? w4_whole<IN, TM, GV, SB, false> : w4_stream<IN, TM, GV, SB, false>;
    if constexpr (SB > 1) {
        if (a.Z) k = a.whole ? w4_whole<IN, TM, GV, SB, true> : w4_stream<IN, TM, GV, SB, true>;
    }
    if (a.lds_bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, a.lds_bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)units), dim3(NT), a.lds_bytes, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace dg
