// w4.hip -- products with 4-bit weights and group scales, for one weight matrix
// or for the experts of a mixture:
//
//   C[m][n] = act(sum over k of A[m][k] * s[n][k/G] * (q[n][k] - z[n][k/G]))
//
// q - z is a whole number of at most 255, exact in FP16 and BF16, so it goes to
// the matrix cores as it is; each scale group's sum is formed in FP32 there and
// then enters the FP32 accumulator times its scale, once.  No weight is rounded.
#include "device_common.hpp"
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
constexpr int WIN = 128;   // K elements of a window: 64 bytes of a weight row

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
// the pairs one mask finds; A's elements are put in the same order (pair_order).
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

__device__ __forceinline__ u32x4 pair_order(u32x4 a) {
    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

// One window of a wave: 16 * NB columns, 16 * TM rows of A.  GV: scale groups a
// window can touch (1, 2 or 4).
template <int TM, int NB, int GV, int SB> struct Window {
    u32x4 q[NB];                // lane row g: bytes 16 g .. + 15 of its column's 64
    uint32_t s[NB][GV * SB > 4 ? GV * SB / 4 : 1], z[NB];   // raw scales of SB bytes each, zero points
    u32x4 a[TM][4];             // K 32 i + 8 g .. + 7
};

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

// A workgroup computes 16 * TM rows x 16 * NB columns; its 8 waves take the
// windows of K in turn (wave w: windows w, w + 8, ...), so that together they
// read whole 512-byte pieces of each weight row, and add up their sums through
// LDS, always in wave order.
template <int IN, int TM, int NB, int GV, int SB>
__global__ void __launch_bounds__(NT) w4_stream(W4Args a) {
    extern __shared__ float red[];   // [WAVES][TM * NB * 4][64]
    constexpr int D = 2;   // windows in flight
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = lane & 15, g = lane >> 4;

    // this workgroup's rows, columns and expert
    int e = 0, begin = 0, rows = a.M, unit, nk = a.K;
    if (a.offsets) {
        moe::Slot s;
        if (!moe::find_slot<16 * TM>(a.offsets, a.o_s, a.E, a.M, a.slabs, blockIdx.x, s)) return;
        e = s.e; begin = s.begin; rows = s.rows; unit = s.unit;
        if (e == a.E) { e = 0; nk = 0; }   // rows of no expert: zero
    } else {
        unit = moe::xcd_run(blockIdx.x, gridDim.x);
    }
    const int tiles_m = (rows + 16 * TM - 1) / (16 * TM);
    const int m0 = (unit % tiles_m) * 16 * TM, n0 = unit / tiles_m * 16 * NB;

    const char *qb = a.Q + (int64_t)e * a.q_es + (int64_t)n0 * a.q_rs;
    const char *sb = a.S + (int64_t)e * a.s_es + (int64_t)n0 * a.s_rs;
    const char *zb = a.Z ? a.Z + (int64_t)e * a.z_es + (int64_t)n0 * a.z_rs : nullptr;
    const char *ab = a.A + (int64_t)(begin + m0) * a.a_rs;
    uint32_t col[NB], row[TM];
#pragma unroll
    for (int b = 0; b < NB; ++b) col[b] = min(n0 + 16 * b + l, a.N - 1) - n0;   // columns past N: the last one again
#pragma unroll
    for (int i = 0; i < TM; ++i) row[i] = (uint32_t)(min(m0 + 16 * i + l, rows - 1) - m0) * (uint32_t)a.a_rs;
    const int groups = (a.K + a.G - 1) / a.G;

    f32x4 acc[TM][NB];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    using W = Window<TM, NB, GV, SB>;
    // group of part i of window w's GV parts
    auto group_of = [&](int w, int i) { return min((w * WIN + i * (WIN / GV)) / a.G, groups - 1); };
    auto load_scales = [&](W &x, int w, bool whole) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const char *sp = sb + col[b] * (uint32_t)a.s_rs, *zp = zb + (zb ? col[b] * (uint32_t)a.z_rs : 0u);
            x.z[b] = 0u;
            if (GV == 1 || (whole && a.s_vec)) {   // the groups are adjacent
                const int g0 = group_of(w, 0);
                load_raw<GV * SB>(x.s[b], sp + (int64_t)g0 * a.s_cs);
                if (zb) load_raw<GV>(&x.z[b], zp + (int64_t)g0 * a.z_cs);
            } else {
                uint32_t v[GV];
#pragma unroll
                for (int i = 0; i < GV; ++i) {
                    const int gi = group_of(w, i);
                    load_raw<SB>(v + i, sp + (int64_t)gi * a.s_cs);
                    if (zb) x.z[b] |= (uint32_t)*reinterpret_cast<const uint8_t *>(zp + (int64_t)gi * a.z_cs) << (8 * i);
                }
                if constexpr (SB == 4) {
#pragma unroll
                    for (int i = 0; i < GV; ++i) x.s[b][i] = v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < GV; i += 2) x.s[b][i / 2] = v[i] | v[i + 1 < GV ? i + 1 : i] << 16;
                }
            }
        }
    };
    auto load = [&](W &x, int w) __attribute__((always_inline)) {   // a whole window
#pragma unroll
        for (int b = 0; b < NB; ++b)
            x.q[b] = *reinterpret_cast<const u32x4_any *>(qb + (int64_t)w * (WIN / 2) + (col[b] * (uint32_t)a.q_rs + 16 * g));
        load_scales(x, w, true);
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x.a[t][i] = *reinterpret_cast<const u32x4_any *>(ab + (int64_t)w * (WIN * 2) + (row[t] + 64 * i + 16 * g));
    };
    // the window that K ends in: whole chunks or the bytes up to the end
    auto load_tail = [&](W &x, int w) __attribute__((always_inline)) {
        const int q0 = w * (WIN / 2) + 16 * g, q_left = (nk + 1) / 2 - q0;
#pragma unroll
        for (int b = 0; b < NB; ++b) x.q[b] = load_part<1>(qb + col[b] * (uint32_t)a.q_rs + q0, q_left);
        load_scales(x, w, false);
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = w * WIN + 32 * i + 8 * g;
                x.a[t][i] = load_part<2>(ab + row[t] + 2 * (int64_t)k, nk - k);
            }
    };
    auto compute = [&](const W &x) __attribute__((always_inline)) {
        u32x4 fa[TM][4];
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[t][i] = pair_order(x.a[t][i]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const u32x4 q = across_rows(x.q[b]);
            f32x4 blk[TM];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int part = i * GV / 4;
                const float z = zb ? (float)((x.z[b] >> (8 * part)) & 255u) : 8.0f;
                const u32x4 fb = decode<IN>(q[i], z);
                const bool first = i % (4 / GV) == 0, last = (i + 1) % (4 / GV) == 0;
#pragma unroll
                for (int t = 0; t < TM; ++t) blk[t] = mfma<IN>(fa[t][i], fb, first ? f32x4{0.f, 0.f, 0.f, 0.f} : blk[t]);
                if (last) {
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
                        for (int r = 0; r < 4; ++r) acc[t][b][r] = fmaf(s, blk[t][r], acc[t][b][r]);
                }
            }
        }
    };

    const int whole = nk / WIN;
    W x[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (wave + WAVES * d < whole) load(x[d], wave + WAVES * d);
    for (int w = wave; w < whole; w += WAVES * D) {
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (w + WAVES * d < whole) {
                compute(x[d]);
                __builtin_amdgcn_sched_barrier(0);   // the loads reuse this window's registers
                if (w + WAVES * (d + D) < whole) load(x[d], w + WAVES * (d + D));
            }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (nk % WIN != 0 && wave == whole % WAVES) {
        load_tail(x[0], whole);
        compute(x[0]);
    }

    // the waves' sums: register (t, b, r) of lane (l, g) is C[16 t + 4 g + r][16 b + l]
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[((wave * TM + t) * NB + b) * 256 + r * 64 + lane] = acc[t][b][r];
    __syncthreads();
    constexpr int REGS = TM * NB * 256;
    for (int i = tid; i < REGS; i += NT) {
        float v = red[i];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += red[w * REGS + i];
        const int la = i & 63, r = (i >> 6) & 3, b = (i >> 8) % NB, t = (i >> 8) / NB;
        const int m = m0 + 16 * t + 4 * (la >> 4) + r, n = n0 + 16 * b + (la & 15);
        if (m < rows && n < a.N)
            store_out(a.C + (int64_t)(begin + m) * a.c_rs + (int64_t)n * a.c_cs, a.out_kind, activate(a.act, v));
    }
}

template <int IN, int TM, int NB, int GV, int SB>
hipError_t launch_t(const W4Args &a, int64_t units, hipStream_t s) {
    constexpr int lds = WAVES * TM * NB * 1024;
    static_assert(lds <= 64 * 1024, "dynamic LDS without an attribute");
    hipLaunchKernelGGL((w4_stream<IN, TM, NB, GV, SB>), dim3((unsigned)units), dim3(NT), lds, s, a);
    return hipGetLastError();
}

template <int IN, int TM, int NB, int SB>
hipError_t launch_g(const W4Args &a, int64_t units, hipStream_t s) {
    if (a.G % WIN == 0) return launch_t<IN, TM, NB, 1, SB>(a, units, s);
    if (a.G == WIN / 2) return launch_t<IN, TM, NB, 2, SB>(a, units, s);
    return launch_t<IN, TM, NB, 4, SB>(a, units, s);
}

template <int IN, int SB>
hipError_t launch(int tm, const W4Args &a, int64_t units, hipStream_t s) {
    constexpr int NB = W4_COLS / 16;
    return tm == 1 ? launch_g<IN, 1, NB, SB>(a, units, s) : launch_g<IN, 2, NB, SB>(a, units, s);
}

}  // namespace

hipError_t launch_w4(int in_kind, int tm, const W4Args &a, int64_t units, hipStream_t s) {
    const bool wide = a.s_kind == OUT_F32;
    if (in_kind == IN_BF16) return wide ? launch<IN_BF16, 4>(tm, a, units, s) : launch<IN_BF16, 2>(tm, a, units, s);
    return wide ? launch<IN_F16, 4>(tm, a, units, s) : launch<IN_F16, 2>(tm, a, units, s);
}

}  // namespace dg
