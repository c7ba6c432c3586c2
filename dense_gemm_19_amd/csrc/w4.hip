// w4.hip -- products with 4-bit weights and group scales, for one weight matrix
// or for the experts of a mixture:
//
//   C[m][n] = act(sum over k of A[m][k] * s[n][k/G] * (q[n][k] - z[n][k/G]))
//
// q - z is a whole number of at most 255, exact in FP16 and BF16, so it goes to
// the matrix cores as it is; each scale group's sum is formed in FP32 there and
// then enters the FP32 accumulator times its scale, once.  No weight is rounded.
#include "device_common.hpp"
#include "gemm_dtl.hpp"
#include "moe.hpp"
#include "moe_slot.hpp"

namespace dg {
namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int WAVES = 8, NT = 64 * WAVES;
constexpr int WIN = 128;             // K elements of a window: 64 bytes of a weight row
constexpr int CHUNK = WAVES * WIN;   // K elements of a chunk: one window per wave
constexpr int ROW = CHUNK * 2;       // bytes of a chunk's row of A in LDS

// 16 bytes at p, of which only the first `left` elements of BYTES bytes may be
// read; zeros after them.
template <int BYTES>
__device__ __forceinline__ u32x4 load_part(const char *p, int left) {
    if (left >= 16 / BYTES) return *reinterpret_cast<const u32x4_any *>(p);
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int j = left - 1; j >= 0; --j) {
        hi = hi << (8 * BYTES) | lo >> (64 - 8 * BYTES);
        lo = lo << (8 * BYTES) | (BYTES == 1 ? *reinterpret_cast<const uint8_t *>(p + j)
                                             : *reinterpret_cast<const uint16_t *>(p + 2 * j));
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

template <int IN>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 4 x 4 dwords across the four 16-lane rows of a wave: afterwards dword i of
// lane row g is what lane row i held in dword g.
__device__ __forceinline__ u32x4 across_rows(u32x4 d) {
    u32x2 t = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    d[0] = t[0]; d[2] = t[1];
    t = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    d[1] = t[0]; d[3] = t[1];
    t = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
    d[0] = t[0]; d[1] = t[1];
    t = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
    d[2] = t[0]; d[3] = t[1];
    return d;
}

// 8 codes (k in nibble k) minus z, in the order (k0 k4)(k1 k5)(k2 k6)(k3 k7):
// the pairs one mask finds; A's elements are put in the same order (a_order).
// 0x6400 | q is the FP16 number 1024 + q, and 0x6400 | 16 q is 1024 + 16 q, so
// one packed add or multiply-add gives two differences, exactly.
template <int IN>
__device__ __forceinline__ u32x4 decode(uint32_t x, float z) {
    const uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, one = 0x64006400u;
    const uint32_t h[4] = {(x & lo) | one, (x & hi) | one, ((x >> 8) & lo) | one, ((x >> 8) & hi) | one};
    u32x4 out;
    if (IN == IN_F16) {
        const _Float16 a = (_Float16)(-1024.0f - z), b = (_Float16)(-64.0f - z);
        const f16x2 a2 = {a, a}, b2 = {b, b}, s2 = {(_Float16)0.0625f, (_Float16)0.0625f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x2 v = __builtin_bit_cast(f16x2, h[j]);
            out[j] = __builtin_bit_cast(uint32_t, j & 1 ? __builtin_elementwise_fma(v, s2, b2) : v + a2);
        }
    } else {
        // BF16 has no packed arithmetic here: mixed FP16 -> FP32 multiply-adds, then the
        // upper halves of two (a difference has at most 8 significant bits)
        const float a = -1024.0f - z, b = -64.0f - z;
        float unit = 1.0f;
        asm("" : "+s"(unit));   // keeps the multiply, so that conversion and add are one instruction
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f16x2 v = __builtin_bit_cast(f16x2, h[j]);
            const float p = fmaf((float)v[0], j & 1 ? 0.0625f : unit, j & 1 ? b : a);
            const float q = fmaf((float)v[1], j & 1 ? 0.0625f : unit, j & 1 ? b : a);
            out[j] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, q), __builtin_bit_cast(uint32_t, p), 0x07060302u);
        }
    }
    return out;
}

// 8 codes as BF16 numbers, z not yet subtracted, in the order (k0 k2)(k4 k6)(k1
// k3)(k5 k7).  As E4M3 a byte 0 .. 15 is that many times 2^-9 (its subnormals
// and first normals lie evenly), so one conversion with a scale of 2^9 gives two
// of them, exactly: 7 instructions where decode takes 17.
__device__ __forceinline__ u32x4 decode_codes(uint32_t x) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t lo = x & 0x0f0f0f0fu, hi = (x >> 4) & 0x0f0f0f0fu;
    const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true)};
    return u32x4{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                 __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
}
// -z for every element of a fragment (z <= 255: exact in BF16)
__device__ __forceinline__ u32x4 minus_zero_point(float z) {
    const uint32_t b = __builtin_bit_cast(uint32_t, -z), p = __builtin_amdgcn_perm(b, b, 0x07060302u);
    return u32x4{p, p, p, p};
}

// A's elements in the order of decode_codes (SPLIT) or decode.
template <bool SPLIT>
__device__ __forceinline__ u32x4 a_order(u32x4 a) {
    if constexpr (SPLIT)
        return u32x4{__builtin_amdgcn_perm(a[1], a[0], 0x05040100u), __builtin_amdgcn_perm(a[3], a[2], 0x05040100u),
                     __builtin_amdgcn_perm(a[1], a[0], 0x07060302u), __builtin_amdgcn_perm(a[3], a[2], 0x07060302u)};

    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

// One window's codes, scales (SB bytes each; two 16-bit ones share a word) and
// zero points of NB column blocks, in flight.  GV: scale groups a window can
// touch (1, 2 or 4).
template <int NB, int GV, int SB> struct Window {
    u32x4 q[NB];                // lane row g: bytes 16 g .. + 15 of its column's 64
    uint32_t s[NB][GV * SB > 4 ? GV * SB / 4 : 1], z[NB];
};

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

// `BYTES` bytes at any alignment, into words.
template <int BYTES>
__device__ __forceinline__ void load_raw(uint32_t *w, const char *p) {
    if constexpr (BYTES == 1) w[0] = *reinterpret_cast<const uint8_t *>(p);
    else if constexpr (BYTES == 2) w[0] = *reinterpret_cast<const u16_any *>(p);
    else if constexpr (BYTES == 4) w[0] = *reinterpret_cast<const u32_any *>(p);
    else if constexpr (BYTES == 8) {
        const u32x2 v = *reinterpret_cast<const u32x2_any *>(p);
        w[0] = v[0]; w[1] = v[1];
    } else {
        const u32x4 v = *reinterpret_cast<const u32x4_any *>(p);
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    }
}

// A pointer that every lane shares, in scalar registers.
__device__ __forceinline__ const char *uniform(const char *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
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

// A workgroup computes 16 * TM rows x 16 * NB columns over its chunks of K.
//  - Codes go from memory to registers, D windows ahead of their use, each lane
//    16 bytes of one column: wave w takes window w of every chunk, so that the
//    8 waves together read 512-byte pieces of each weight row.
//  - A's rows go to LDS a chunk at a time, `bufs` chunks ahead, by load-to-LDS
//    instructions (`direct`; 16-byte chunks of A) or through registers.  A row's
//    16-byte pieces are XOR-swizzled by its number, so that the 16 rows of a
//    fragment read fall on distinct banks; only the rows there are take space.
//  - The waves' sums are added through LDS, in wave order.  With S > 1 pieces of
//    K (one matrix, few columns) the workgroups' sums meet in the workspace as
//    in the dense kernels: the last to arrive adds them in the order of K.
// Loads return in order, so that waiting for a chunk of A waits for every older
// code load too: the code loads a workgroup can keep in flight are those of
// `bufs` - 1 chunks, which is why few rows get up to 8 buffers.
template <int IN, int TM, int GV, int SB>
__global__ void __launch_bounds__(NT, TM == 1 ? 4 : 2) w4_stream(W4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // A ring; afterwards the waves' sums
    __shared__ int is_last;
    constexpr int D = TM == 1 ? (GV * SB < 8 ? 4 : 3) : TM == 2 || (TM == 3 && GV * SB < 16) ? 2 : 1;   // windows in flight
    // Few BF16 rows are bound by the decoding: the codes go to the matrix cores as
    // they are and the zero points as a second product into the same sums.
    constexpr bool RAW = IN == IN_BF16 && TM == 1;
    constexpr int NB = w4_cols(TM) / 16;   // 16-column blocks of a workgroup
    constexpr int MR = 16 * TM;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    const int m0 = (unit % tiles_m) * MR, n0 = unit / tiles_m * 16 * NB;
    const int here = min(rows - m0, MR);           // rows of this tile
    const int c0 = z * a.chunks, c1 = min(c0 + a.chunks, (nk + CHUNK - 1) / CHUNK);
    const int windows = (nk + WIN - 1) / WIN, whole = nk / WIN;

    const char *qb = uniform(a.Q + (int64_t)e * a.q_es + (int64_t)n0 * a.q_rs);
    const char *sb = uniform(a.S + (int64_t)e * a.s_es + (int64_t)n0 * a.s_rs);
    const char *zb = a.Z ? uniform(a.Z + (int64_t)e * a.z_es + (int64_t)n0 * a.z_rs) : nullptr;
    const char *ab = uniform(a.A + (int64_t)(begin + m0) * a.a_rs);
    uint32_t col[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) col[b] = min(n0 + 16 * b + l, a.N - 1) - n0;   // columns past N: the last one again
    const int groups = a.groups;

    f32x4 acc[TM][NB];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    using W = Window<NB, GV, SB>;
    // group of part i of window w's GV parts
    auto group_of = [&](int w, int i) { 
        // (32-wide step) / (G / 32), by the reciprocal 2^32 / (G / 32) rounded up:
        // exact while the product of the two stays below 2^32 (K <= 2^20)
        const uint32_t step = (uint32_t)(4 * w + i * (4 / GV));
        return min((int)(a.g_mul ? __umulhi(step, a.g_mul) : step), groups - 1);
    };
    auto scales_apart = [&](W &x, int w) __attribute__((always_inline)) {   // one by one
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t v[GV];
            x.z[b] = 0u;
#pragma unroll
            for (int i = 0; i < GV; ++i) {
                const int gi = group_of(w, i);
                load_raw<SB>(v + i, sb + (int64_t)gi * a.s_cs + col[b] * (uint32_t)a.s_rs);
                if (zb) x.z[b] |= (uint32_t)*reinterpret_cast<const uint8_t *>(zb + (int64_t)gi * a.z_cs + col[b] * (uint32_t)a.z_rs) << (8 * i);
            }
#pragma unroll
            for (int i = 0; i < GV; ++i) {
                if constexpr (SB == 4) x.s[b][i] = v[i];
                else if (i % 2 == 0) x.s[b][i / 2] = v[i] | v[i + 1 < GV ? i + 1 : i] << 16;
            }
        }
    };
    auto load = [&](W &x, int w) __attribute__((always_inline)) {   // a whole window
        if (w >= whole) return;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            x.q[b] = *reinterpret_cast<const u32x4_any *>(qb + (int64_t)w * (WIN / 2) + (col[b] * (uint32_t)a.q_rs + 16 * g));
        if (GV > 1 && !a.s_vec) {
            scales_apart(x, w);
            return;
        }
        const int g0 = group_of(w, 0);
#pragma unroll
        for (int b = 0; b < NB; ++b) load_raw<GV * SB>(x.s[b], sb + (int64_t)g0 * a.s_cs + col[b] * (uint32_t)a.s_rs);
        if (zb) {
#pragma unroll
            for (int b = 0; b < NB; ++b) load_raw<GV>(&x.z[b], zb + (int64_t)g0 * a.z_cs + col[b] * (uint32_t)a.z_rs);
        }
    };

    // chunk c of A into buffer c % bufs: piece p of row r holds K elements 8 (p ^ (r % 16)) .. + 7
    const uint32_t lds0 = dtl::lds_addr(lds);
    const int bytes = a.rows_lds * ROW;            // of a buffer
    auto stage = [&](int c, int buf) __attribute__((always_inline)) {   // buf: its byte offset
        if (a.direct) {
            const int last = nk / 8 - 1 - c * (CHUNK / 8);   // pieces past K read the last one (cleared below)
#pragma unroll 1
            for (int j = wave; j < 2 * here; j += WAVES) {
                const int r = j >> 1, p = (j & 1) * 64 + lane;
                dtl::lds_load16(ab + (int64_t)r * a.a_rs + (int64_t)c * ROW, 16 * min(p ^ (r & 15), last),
                                __builtin_amdgcn_readfirstlane(lds0 + buf + j * 1024));
            }
        } else {
#pragma unroll 1
            for (int j = tid; j < here * 128; j += NT) {
                const int r = j >> 7, k = c * CHUNK + 8 * ((j & 127) ^ (r & 15));
                *reinterpret_cast<u32x4 *>(lds + buf + j * 16) = load_part<2>(ab + (int64_t)r * a.a_rs + 2 * (int64_t)k, nk - k);
            }
        }
    };
    // K elements of a window's end that the direct loads could not leave out
    auto clear = [&](int buf) __attribute__((always_inline)) {
        const int p0 = (nk % CHUNK) / 8, n = 16 - p0 % 16;
        for (int j = tid; j < here * n; j += NT) {
            const int r = j / n, p = p0 + j % n;
            *reinterpret_cast<u32x4 *>(lds + buf + r * ROW + 16 * (p ^ (r & 15))) = u32x4{0u, 0u, 0u, 0u};
        }
    };

    int arow[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) arow[t] = min(16 * t + l, here - 1);   // rows past the tile: one of it again
    auto compute = [&](W &x, int buf) __attribute__((always_inline)) {
        const char *la = lds + buf;
#pragma unroll
        for (int b = 0; b < NB; ++b) x.q[b] = across_rows(x.q[b]);
        f32x4 blk[TM][NB];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            constexpr int PER = 4 / GV;               // 32-wide steps of a group
            const int part = i / PER;
            u32x4 fa[TM];
#pragma unroll
            for (int t = 0; t < TM; ++t)
                fa[t] = a_order<RAW>(*reinterpret_cast<const u32x4 *>(la + arow[t] * ROW + 16 * ((16 * wave + 4 * i + g) ^ (arow[t] & 15))));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float zp = zb ? (float)((x.z[b] >> (8 * part)) & 255u) : 8.0f;
                const u32x4 fb = RAW ? decode_codes(x.q[b][i]) : decode<IN>(x.q[b][i], zp);
#pragma unroll
                for (int t = 0; t < TM; ++t) {
                    blk[t][b] = mfma<IN>(fa[t], fb, i % PER == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : blk[t][b]);
                    if (RAW) blk[t][b] = mfma<IN>(fa[t], minus_zero_point(zp), blk[t][b]);
                }
            }
            if (i % PER == PER - 1) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float s;
                    if constexpr (SB == 4) {
                        s = __builtin_bit_cast(float, x.s[b][part]);
                    } else {
                        const uint16_t h = (uint16_t)(x.s[b][part / 2] >> (16 * (part & 1)));
                        s = a.s_kind == OUT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
                    }
#pragma unroll
                    for (int t = 0; t < TM; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[t][b][r] = fmaf(s, blk[t][b][r], acc[t][b][r]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // one step's codes at a time in registers
        }
    };

    // The loads of a window: NB of codes, NB of scales, NB of zero points (more
    // where the scales go one by one: the waits are then stricter than needed).
    W x[D];
    const int w0 = WAVES * c0 + wave;
#pragma unroll 1
    for (int c = c0; c < min(c0 + a.bufs, c1); ++c) stage(c, (c - c0) * bytes);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (c0 + d < c1) load(x[d], w0 + WAVES * d);
    int buf = 0, last_buf = 0;   // of the chunk at hand; of the last one
    for (int cc = c0; cc < c1; cc += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int c = cc + d, w = WAVES * c + wave;
            if (c >= c1) break;
            if (a.direct && (c == c0 || c - c0 >= a.bufs)) {
                // Chunk c has landed once no more loads are in flight than this
                // wave certainly issued after it: the windows of the prologue
                // (the first chunk: with it every buffer's), or the window
                // loaded at the end of the chunk before.
                if (c == c0 && c0 + D <= c1 && w0 + WAVES * (D - 1) < whole) {
                    if (zb) DG_VM(3 * NB * D); else DG_VM(2 * NB * D);
                } else if (c > c0 && c - 1 + D < c1 && w + WAVES * (D - 1) < whole) {
                    if (zb) DG_VM(3 * NB); else DG_VM(2 * NB);
                } else {
                    DG_VM(0);
                }
            }
            wait_barrier();      // every wave's part of chunk c is in LDS
            if (w < whole) compute(x[d], buf);
            if (c + a.bufs < c1) {
                wait_barrier();  // chunk c has been read
                stage(c + a.bufs, buf);
            }
            last_buf = buf;
            buf = buf + bytes == a.bufs * bytes ? 0 : buf + bytes;
            __builtin_amdgcn_sched_barrier(0);   // the loads reuse this window's registers
            if (c + D < c1) load(x[d], w + WAVES * D);
        }
    }
    // The window that K ends in: it lies in the last chunk, whose rows are still
    // in LDS, with what lies past K to be cleared where the loads were direct.
    if (whole < windows && c1 * CHUNK > whole * WIN && c0 < c1) {
        if (a.direct) {
            clear(last_buf);
            wait_barrier();
        }
        if (wave == whole % WAVES) {
            const int q0 = whole * (WIN / 2) + 16 * g, left = (nk + 1) / 2 - q0;
#pragma unroll
            for (int b = 0; b < NB; ++b) x[0].q[b] = load_part<1>(qb + col[b] * (uint32_t)a.q_rs + q0, left);
            scales_apart(x[0], whole);
            compute(x[0], last_buf);
        }
    }

    // the waves' sums: register (t, b, r) of lane (l, g) is C[16 t + 4 g + r][16 b + l]
    constexpr int REGS = TM * NB * 256;
    float *red = reinterpret_cast<float *>(lds);
    wait_barrier();
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[((wave * TM + t) * NB + b) * 256 + r * 64 + lane] = acc[t][b][r];
    __syncthreads();
    float v[REGS / NT];
#pragma unroll
    for (int u = 0; u < REGS / NT; ++u) {
        v[u] = red[u * NT + tid];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v[u] += red[w * REGS + u * NT + tid];
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
        const int i = u * NT + tid, la = i & 63, r = (i >> 6) & 3, b = (i >> 8) % NB, t = (i >> 8) / NB;
        const int m = m0 + 16 * t + 4 * (la >> 4) + r, n = n0 + 16 * b + (la & 15);
        if (m >= rows || n >= o.N) continue;
        // an infinite activation times q and times -z may cancel to NaN
        if (RAW && !(fabsf(v[u]) < __builtin_inff())) v[u] = whole_sum(o, e, begin + m, n, nk);
        store_out(o.C + (int64_t)(begin + m) * o.c_rs + (int64_t)n * o.c_cs, o.out_kind, activate(o.act, v[u]));
    }
}

template <int IN, int TM, int GV, int SB>
hipError_t launch_t(const W4Args &a, int64_t units, hipStream_t s) {
    const int ring = a.bufs * a.rows_lds * ROW, sums = WAVES * TM * w4_cols(TM) * 64, lds = ring > sums ? ring : sums;
    auto k = w4_stream<IN, TM, GV, SB>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)units), dim3(NT), lds, s, a);
    return hipGetLastError();
}

template <int IN, int TM, int SB>
hipError_t launch_g(const W4Args &a, int64_t units, hipStream_t s) {
    if (a.G % WIN == 0) return launch_t<IN, TM, 1, SB>(a, units, s);
    if (a.G == WIN / 2) {
        if constexpr (TM <= (SB == 4 ? 2 : 3)) return launch_t<IN, TM, 2, SB>(a, units, s);   // (more would spill)
        else return hipErrorInvalidValue;
    }
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

int w4_max_tm(int group, int s_kind) { return group == WIN / 2 ? (s_kind == OUT_F32 ? 2 : 3) : 4; }

hipError_t launch_w4(int in_kind, int tm, const W4Args &a, int64_t units, hipStream_t s) {
    const bool wide = a.s_kind == OUT_F32;
    if (in_kind == IN_BF16) return wide ? launch<IN_BF16, 4>(tm, a, units, s) : launch<IN_BF16, 2>(tm, a, units, s);
    return wide ? launch<IN_F16, 4>(tm, a, units, s) : launch<IN_F16, 2>(tm, a, units, s);
}

}  // namespace dg
