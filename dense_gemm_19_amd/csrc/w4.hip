// w4.hip -- products with 4-bit weights and group scales, for one weight matrix
// or for the experts of a mixture:
//
//   C[m][n] = act(sum over k of A[m][k] * s[n][k/G] * (q[n][k] - z[n][k/G]))
//
// Codes and zero points are whole numbers of at most 255, exact in FP16 and
// BF16, so they go to the matrix cores as they are; each scale group's sum is
// formed in FP32 there and then enters the FP32 accumulator times its scale,
// once.  No weight is rounded.
//
// Bound by the bytes of the codes for few rows (half a byte per weight), by the
// vector ALUs that decode them for many.
#include "device_common.hpp"
#include "gemm_dtl.hpp"
#include "moe.hpp"
#include "moe_slot.hpp"

namespace dg {
namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
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

// 8 codes minus z as FP16 or BF16.  A byte q under 0x64 is the FP16 number 1024
// + q, so one packed add gives two differences, exactly.  BF16 has no packed
// arithmetic here: mixed FP16 -> FP32 multiply-adds, then the upper halves of two
// (a difference has at most 8 significant bits).
template <int IN>
__device__ __forceinline__ u32x4 decode(uint32_t x, float z) {
    const u32x2 e = code_bytes(x);
    u32x4 out;
    float unit = 1.0f;
    asm("" : "+s"(unit));   // keeps the multiply, so that conversion and add are one instruction
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, e[j / 2], j & 1 ? 0x04030402u : 0x04010400u));
        if (IN == IN_F16) {
            const _Float16 c = (_Float16)(-1024.0f - z);
            out[j] = __builtin_bit_cast(uint32_t, v + f16x2{c, c});
        } else {
            const float p = fmaf((float)v[0], unit, -1024.0f - z), q = fmaf((float)v[1], unit, -1024.0f - z);
            out[j] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, q), __builtin_bit_cast(uint32_t, p), 0x07060302u);
        }
    }
    return out;
}

// 8 codes as BF16 numbers, z not yet subtracted.  As E4M3 a byte 0 .. 15 is that
// many times 2^-9 (its subnormals and first normals lie evenly), so one
// conversion with a scale of 2^9 gives two of them, exactly: 9 instructions where
// decode takes 21.
__device__ __forceinline__ u32x4 decode_codes(uint32_t x) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const u32x2 e = code_bytes(x);
    const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(e[0], 512.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(e[0], 512.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(e[1], 512.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(e[1], 512.0f, true)};
    return u32x4{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                 __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
}
// -z for every element of a fragment (z <= 255: exact in BF16)
__device__ __forceinline__ u32x4 minus_zero_point(float z) {
    const uint32_t b = __builtin_bit_cast(uint32_t, -z), p = __builtin_amdgcn_perm(b, b, 0x07060302u);
    return u32x4{p, p, p, p};
}

// 16 bytes from p on: elements of BYTES bytes `stride` apart, of which only the
// first `left` may be read; zeros after them.
template <int BYTES>
__device__ __forceinline__ u32x4 load_part(const char *p, int64_t stride, int left) {
    if (stride == BYTES && left >= 16 / BYTES) return *reinterpret_cast<const u32x4_any *>(p);
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int j = min(left, 16 / BYTES) - 1; j >= 0; --j) {
        const char *q = p + j * stride;
        hi = hi << (8 * BYTES) | lo >> (64 - 8 * BYTES);
        lo = lo << (8 * BYTES) | (BYTES == 1   ? *reinterpret_cast<const uint8_t *>(q)
                                  : BYTES == 2 ? *reinterpret_cast<const uint16_t *>(q)
                                               : *reinterpret_cast<const uint32_t *>(q));
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// C[m][n] before the activation, by the definition, one element after another
// (for sums that came out infinite or NaN).
__device__ __forceinline__ float whole_sum(const W4Args &a, int e, int m, int n, int nk) {
    const char *q = a.Q + (int64_t)e * a.q_es + (int64_t)n * a.q_rs, *x = a.A + (int64_t)m * a.a_rs;
    float sum = 0.0f;
    for (int k0 = 0; k0 < nk; k0 += a.G) {
        const int gi = k0 / a.G;
        const float s = load_out(a.S + (int64_t)e * a.s_es + (int64_t)n * a.s_rs + (int64_t)gi * a.s_cs, a.s_kind);
        const int z = a.Z ? *reinterpret_cast<const uint8_t *>(a.Z + (int64_t)e * a.z_es + (int64_t)n * a.z_rs + (int64_t)gi * a.z_cs) : 8;
        float part = 0.0f;
        for (int k = k0; k < min(k0 + a.G, nk); ++k) {
            const int code = *reinterpret_cast<const uint8_t *>(q + k / 2) >> (4 * (k & 1)) & 15;
            part = fmaf(bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(x + 2 * (int64_t)k)), (float)(code - z), part);
        }
        sum = fmaf(s, part, sum);
    }
    return sum;
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

// A workgroup computes 16 * TM rows x 16 * WN columns over its chunks of K.  Its
// 8 waves are WK x WN: wave (wk, wn) takes 16 columns and unit wk of every chunk.
//  - Codes go to LDS as they lie, `depth` units ahead, by load-to-LDS instructions
//    (`q_direct`) that fetch whole cache lines, 8 rows of 128 bytes each.  With 64
//    bytes of 16 rows per instruction, straight to registers, 1 x 4096 x 14336
//    took 14.2 us.  A wave reads only what it loaded itself: no barrier.
//  - Scales and zero points of many groups go to LDS at once, before the loop
//    (`seg` chunks of them): loaded at each unit they were 16 lines for 32 bytes.
//  - A's rows go to LDS a chunk at a time, by load-to-LDS instructions (`direct`)
//    or through registers, as many chunks ahead as a_lds bytes hold of the rows
//    there are: few rows of a usual K are there whole.
//  - The waves' sums along K are added through LDS, in wave order.  With splits > 1
//    pieces of K (one matrix, few columns) the workgroups' sums meet in the
//    workspace as in the dense kernels: the last to arrive adds them in the
//    order of K.
// Pieces of 16 bytes are XOR-swizzled by their row in LDS (fetched so from
// memory), so that the 16 rows of a fragment read fall on distinct banks.
// Loads return in order: waiting for a chunk of A waits for every older code
// load too, so min(depth - 1, chunks of A in LDS) units stay in flight.
// GV: scale groups that 128 K elements can touch (1, 2 or 4); SB: bytes of a scale.
template <int IN, int TM, int GV, int SB, bool ZP>
__global__ void __launch_bounds__(NT, TM == 1 ? 4 : 2) w4_stream(W4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // codes, A, scales, zero points; then the waves' sums
    __shared__ int is_last;
    constexpr int WN = w4_cols(TM) / 16, WK = WAVES / WN, CHUNK = w4_chunk(TM), ROW = CHUNK * 2;
    static_assert(WK * UNIT == CHUNK, "a unit per wave");
    constexpr int MR = 16 * TM;
    // Few BF16 rows are bound by the decoding: the codes go to the matrix cores as
    // they are and the zero points as a second product of the same rows.
    constexpr bool RAW = IN == IN_BF16 && TM == 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave % WK, wn = wave / WK;
    const int l = lane & 15, g = lane >> 4;

    // this workgroup's rows, columns, expert and piece of K
    int e = 0, begin = 0, rows = a.M, unit, nk = a.K, z = 0;
    if (a.offsets) {
        moe::Slot s;
        if (!moe::find_slot<MR>(a.offsets, a.o_s, a.E, a.M, a.slabs, blockIdx.x, s)) return;
        e = s.e; begin = s.begin; rows = s.rows; unit = s.unit;
        if (e == a.E) { e = 0; nk = 0; }   // rows of no expert: zero
    } else {
        unit = moe::xcd_run(blockIdx.x, gridDim.x);
        z = unit % a.splits;
        unit /= a.splits;
    }
    const int tiles_m = (rows + MR - 1) / MR;
    const int m0 = (unit % tiles_m) * MR, n0 = unit / tiles_m * 16 * WN;
    const int here = min(rows - m0, MR);           // rows of this tile
    const int c0 = z * a.chunks, c1 = min(c0 + a.chunks, (nk + CHUNK - 1) / CHUNK);

    const char *qb = a.Q + uniform((int64_t)e * a.q_es + (int64_t)n0 * a.q_rs);
    const char *sb = a.S + uniform((int64_t)e * a.s_es + (int64_t)n0 * a.s_rs);
    const char *zb = ZP ? a.Z + uniform((int64_t)e * a.z_es + (int64_t)n0 * a.z_rs) : nullptr;
    const char *ab = a.A + uniform((int64_t)(begin + m0) * a.a_rs);
    const int cols = min(16 * WN, a.N - n0);       // columns past N: the last one again

    // LDS: [wave][depth] code units, A (a_lds bytes), scales, zero points
    const uint32_t lds0 = dtl::lds_addr(lds);
    const int q_ring = wave * (a.depth * UNIT_LDS), a_ring = WAVES * a.depth * UNIT_LDS;
    const int a_bytes = here * ROW, bufs = min(a.a_lds / a_bytes, 64);   // A's ring: a buffer holds a chunk of the rows there are
    const int s_at = a_ring + a.a_lds, z_at = s_at + 16 * WN * a.s_pitch;

    // Piece p (16 bytes) of row r of a unit lies at r * 128 + 16 * (p ^ (r & 7)).
    // Load h of a unit fills rows 8 h .. 8 h + 7: lane i row 8 h + i / 8, position i % 8.
    const int q_row = lane >> 3, q_piece = (lane & 7) ^ q_row;   // (8 h + q_row) & 7 == q_row
    const uint32_t q_off[2] = {(uint32_t)min(16 * wn + q_row, cols - 1) * (uint32_t)a.q_rs,
                               (uint32_t)min(16 * wn + q_row + 8, cols - 1) * (uint32_t)a.q_rs};
    const int q_bytes = (nk + 1) / 2;
    u32x4 pend[2];   // a unit on its way through registers (codes not 16-byte aligned)
    // Fetch the unit of chunk c (a unit past K: its first line again, to keep the
    // count of loads) into slot `slot` of the ring.
    auto fetch = [&](int c, int slot) __attribute__((always_inline)) {
        const int at = c * (CHUNK / 2) + wk * (UNIT / 2);   // byte of the row
        if (a.q_direct) {
            const bool in = c < c1 && at < q_bytes;
            const int last = in ? q_bytes - at - 16 : 0;    // pieces past the row's end read its last one
            const char *base = qb + (in ? at : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                dtl::lds_load16(base, (in ? q_off[h] : 0u) + (uint32_t)min(16 * q_piece, last),
                                lds0 + q_ring + slot * UNIT_LDS + h * 1024);
        } else if (c < c1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) pend[h] = load_part<1>(qb + q_off[h] + at + 16 * q_piece, 1, q_bytes - at - 16 * q_piece);
        }
    };
    auto land = [&](int slot) __attribute__((always_inline)) {   // pend into its slot
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4 *>(lds + q_ring + slot * UNIT_LDS + h * 1024 + lane * 16) = pend[h];
    };

    // Chunk c of A into the buffer at byte `buf`: piece p of row r lies at r * ROW + 16 * (p ^ (r & 15)).
    constexpr int PR = ROW / 16;                   // pieces of a row
    auto stage = [&](int c, int buf) __attribute__((always_inline)) {
        if (a.direct) {
            const int last = nk / 8 - 1 - c * PR;  // pieces past K read the last one (cleared below)
#pragma unroll 1
            for (int j = wave; j * 64 < here * PR; j += WAVES) {
                const int i = j * 64 + lane, r = min(i / PR, here - 1), p = i % PR;
                dtl::lds_load16(ab + (int64_t)c * ROW, (uint32_t)r * (uint32_t)a.a_rs + 16 * min(p ^ (r & 15), last),
                                __builtin_amdgcn_readfirstlane(lds0 + a_ring + buf + j * 1024));
            }
        } else {
#pragma unroll 1
            for (int i = tid; i < here * PR; i += NT) {
                const int r = i / PR, k = c * CHUNK + 8 * ((i % PR) ^ (r & 15));
                *reinterpret_cast<u32x4 *>(lds + a_ring + buf + i * 16) = load_part<2>(ab + (int64_t)r * a.a_rs + 2 * (int64_t)k, 2, nk - k);
            }
        }
    };
    // The K elements past the end of a unit that direct loads of A left there
    auto clear = [&](int buf) __attribute__((always_inline)) {
        const int p0 = (nk % CHUNK) / 8, n = UNIT / 8 - p0 % (UNIT / 8);
#pragma unroll 1
        for (int j = tid; j < here * n; j += NT) {
            const int r = j / n, p = p0 + j % n;
            *reinterpret_cast<u32x4 *>(lds + a_ring + buf + r * ROW + 16 * (p ^ (r & 15))) = u32x4{0u, 0u, 0u, 0u};
        }
    };
    // Scales and zero points of groups g0 .. of `seg` chunks from c on
    const int groups = a.groups;
    auto stage_scales = [&](int c) __attribute__((always_inline)) {
        const int g0 = c * CHUNK / a.G, n = min(groups - g0, a.seg_groups);
        const int ps = (n * SB + 15) / 16, pz = (n + 15) / 16;
#pragma unroll 1
        for (int i = tid; i < 16 * WN * ps; i += NT) {
            const int r = i / ps, p = i % ps;
            const char *src = sb + (int64_t)min(r, cols - 1) * a.s_rs + (int64_t)(g0 + p * (16 / SB)) * a.s_cs;
            *reinterpret_cast<u32x4 *>(lds + s_at + r * a.s_pitch + 16 * p) = load_part<SB>(src, a.s_cs, n - p * (16 / SB));
        }
        if (ZP) {
#pragma unroll 1
            for (int i = tid; i < 16 * WN * pz; i += NT) {
                const int r = i / pz, p = i % pz;
                const char *src = zb + (int64_t)min(r, cols - 1) * a.z_rs + (int64_t)(g0 + 16 * p) * a.z_cs;
                *reinterpret_cast<u32x4 *>(lds + z_at + r * a.z_pitch + 16 * p) = load_part<1>(src, a.z_cs, n - 16 * p);
            }
        }
        return g0;
    };

    f32x4 acc[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    int arow[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) arow[t] = min(16 * t + l, here - 1);   // rows past the tile: one of it again

    // Group of 32-element step `step` of K: step / (G / 32), by the reciprocal
    // 2^32 / (G / 32) rounded up, exact while the product of the two stays below
    // 2^32 (K <= 2^20).
    auto group_of = [&](int step) { return min((int)(a.g_mul ? __umulhi((uint32_t)step, a.g_mul) : (uint32_t)step), groups - 1); };
    int seg_g0 = 0;
    auto compute = [&](int c, int slot, int buf) __attribute__((always_inline)) {
        const char *lq = lds + q_ring + slot * UNIT_LDS + l * 128 + 4 * g, *la = lds + a_ring + buf;
        const char *ls = lds + s_at + (16 * wn + l) * a.s_pitch, *lz = lds + z_at + (16 * wn + l) * a.z_pitch;
        const int k0 = c * CHUNK + wk * UNIT;
#pragma unroll
        for (int w = 0; w < 2; ++w) {              // 128 elements each
            if (k0 + 128 * w >= nk) break;
            uint32_t q[4];                         // lane row g: bytes 4 g .. + 3 of the step's 16
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint32_t *>(lq + 16 * ((4 * w + i) ^ (l & 7)));
            u32x4 fa[4][TM];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < TM; ++t)
                    fa[i][t] = *reinterpret_cast<const u32x4 *>(la + arow[t] * ROW + 16 * ((wk * 32 + 16 * w + 4 * i + g) ^ (arow[t] & 15)));
            float s[GV], zp[GV];
#pragma unroll
            for (int v = 0; v < GV; ++v) {
                const int gi = group_of(k0 / 32 + 4 * w + v * (4 / GV)) - seg_g0;
                if constexpr (SB == 4) s[v] = *reinterpret_cast<const float *>(ls + 4 * gi);
                else {
                    const uint16_t h = *reinterpret_cast<const uint16_t *>(ls + 2 * gi);
                    s[v] = a.s_kind == OUT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
                }
                zp[v] = ZP ? (float)*reinterpret_cast<const uint8_t *>(lz + gi) : 8.0f;
            }
            f32x4 blk[TM];                         // a group's sums
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int PER = 4 / GV;        // 32-wide steps of a group
                const bool first = i % PER == 0;
                const u32x4 fb = RAW ? decode_codes(q[i]) : decode<IN>(q[i], zp[i / PER]);
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    blk[t] = mfma<IN>(fa[i][t], fb, first ? f32x4{0.f, 0.f, 0.f, 0.f} : blk[t]);
                    if constexpr (RAW) blk[t] = mfma<IN>(fa[i][t], minus_zero_point(zp[i / PER]), blk[t]);
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

    // A, then codes, then scales: the loads return in this order
#pragma unroll 1
    for (int c = c0; c < min(c0 + bufs, c1); ++c) stage(c, (c - c0) * a_bytes);
    if (a.q_direct) {
#pragma unroll 1
        for (int d = 0; d < a.depth; ++d) fetch(c0 + d, d);
    } else {
        fetch(c0, 0);
    }
    int buf = 0, slot = 0;
    for (int c = c0; c < c1; ++c) {
        if ((c - c0) % a.seg == 0) {               // the first chunk, mostly the only time
            if (c > c0) wait_barrier();            // the scales before have been read
            seg_g0 = stage_scales(c);
            DG_VM(0);                              // and with them every load before
            wait_barrier();
        } else {
            // the unit at hand and, where A has a ring, this chunk of it have landed
            const int newer = c - c0 >= bufs ? min(a.depth - 1, bufs) : a.depth - 1;
            if (!a.q_direct) DG_VM(0);
            else if (newer == 1) DG_VM(2);
            else if (newer == 2) DG_VM(4);
            else DG_VM(6);
            if (c - c0 >= bufs) wait_barrier();  // every wave's part of chunk c is in LDS
        }
        if (a.direct && (c + 1) * CHUNK > nk && nk % UNIT != 0) {
            clear(buf);
            wait_barrier();
        }
        if (!a.q_direct) {
            land(slot);
            fetch(c + 1, 0);
        }
        asm volatile("" ::: "memory");             // codes and A are read from here on
        compute(c, slot, buf);
        if (c + bufs < c1) {
            wait_barrier();                        // chunk c has been read
            stage(c + bufs, buf);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot's reads are done
        if (a.q_direct) fetch(c + a.depth, slot);
        buf = buf + a_bytes == bufs * a_bytes ? 0 : buf + a_bytes;
        slot = slot + 1 == a.depth ? 0 : slot + 1;
    }

    // the waves' sums: register (t, r) of lane (l, g) is C[16 t + 4 g + r][16 wn + l]
    constexpr int REGS = TM * WN * 256;
    float *red = reinterpret_cast<float *>(lds);
    DG_VM(0);                                      // the last fetches write LDS too
    wait_barrier();
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wk * REGS + (wn * TM + t) * 256 + r * 64 + lane] = acc[t][r];
    __syncthreads();
    float v[REGS / NT];
#pragma unroll
    for (int u = 0; u < REGS / NT; ++u) {
        v[u] = red[u * NT + tid];
#pragma unroll
        for (int w = 1; w < WK; ++w) v[u] += red[w * REGS + u * NT + tid];
    }
    const W4Args &o = arguments();
    if (o.splits > 1) {
        float *part = o.ws + (int64_t)unit * o.splits * REGS + tid;
#pragma unroll
        for (int u = 0; u < REGS / NT; ++u)
            __hip_atomic_store(part + z * REGS + u * NT, v[u], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) is_last = take_last_ticket(o.counters + unit, o.splits);
        __syncthreads();
        if (!is_last) return;
#pragma unroll
        for (int u = 0; u < REGS / NT; ++u)
            v[u] = sum_partials(o.splits, [&](int q) {
                return __hip_atomic_load(part + q * REGS + u * NT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            });
        if (tid == 0) __hip_atomic_store(o.counters + unit, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int u = 0; u < REGS / NT; ++u) {
        const int i = u * NT + tid, la = i & 63, r = (i >> 6) & 3, t = (i >> 8) % TM, n = n0 + 16 * ((i >> 8) / TM) + (la & 15);
        const int m = m0 + 16 * t + 4 * (la >> 4) + r;
        if (m >= rows || n >= o.N) continue;
        // an infinite activation times q and times -z may cancel to NaN
        if (RAW && !(fabsf(v[u]) < __builtin_inff())) v[u] = whole_sum(o, e, begin + m, n, nk);
        store_out(o.C + (int64_t)(begin + m) * o.c_rs + (int64_t)n * o.c_cs, o.out_kind, activate(o.act, v[u]));
    }
}

template <int IN, int TM, int GV, int SB>
hipError_t launch_t(const W4Args &a, int64_t units, hipStream_t s) {
    const auto k = a.Z ? w4_stream<IN, TM, GV, SB, true> : w4_stream<IN, TM, GV, SB, false>;
    if (a.lds_bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, a.lds_bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)units), dim3(NT), a.lds_bytes, s, a);
    return hipGetLastError();
}

template <int IN, int TM, int SB>
hipError_t launch_g(const W4Args &a, int64_t units, hipStream_t s) {
    if (a.G % 128 == 0) return launch_t<IN, TM, 1, SB>(a, units, s);
    if (a.G == 64) return launch_t<IN, TM, 2, SB>(a, units, s);
    return launch_t<IN, TM, 4, SB>(a, units, s);
}

template <int IN, int SB>
hipError_t launch(int tm, const W4Args &a, int64_t units, hipStream_t s) {
    switch (tm) {
    case 1: return launch_g<IN, 1, SB>(a, units, s);
    case 2: return launch_g<IN, 2, SB>(a, units, s);
    case 3: return launch_g<IN, 3, SB>(a, units, s);
    case 4: return launch_g<IN, 4, SB>(a, units, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_w4(int in_kind, int tm, const W4Args &a, int64_t units, hipStream_t s) {
    const bool wide = a.s_kind == OUT_F32;
    if (in_kind == IN_BF16) return wide ? launch<IN_BF16, 4>(tm, a, units, s) : launch<IN_BF16, 2>(tm, a, units, s);
    return wide ? launch<IN_F16, 4>(tm, a, units, s) : launch<IN_F16, 2>(tm, a, units, s);
}

}  // namespace dg
