// moe_route.hip -- tokens to expert order and back: the stable counting sort of
// the router's choices, the copy of token rows into expert order, the weighted
// sum of the experts' rows back in token order, and that sum's gradient.
#include <algorithm>

#include "device_common.hpp"
#include "moe.hpp"

namespace dg {
namespace {

// 16 bytes at any 1-byte aligned address: gfx950 loads and stores global
// memory at any alignment, so rows of odd length keep whole-chunk accesses.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

// ------------------------------------------------------------------ sort

constexpr int SORT_W = SORT_T / 64;

// The key of id i: its expert, or -1 (dropped).
__device__ __forceinline__ int sort_key(const SortArgs &a, int i) {
    const char *p = a.ids + (a.k > 0 ? (int64_t)(i / a.k) * a.i_rs + (int64_t)(i % a.k) * a.i_cs : i * a.i_cs);
    const int64_t v = a.wide ? *reinterpret_cast<const int64_t *>(p) : *reinterpret_cast<const int32_t *>(p);
    return v >= 0 && v < a.E ? (int)v : -1;
}

// The lanes whose key equals this lane's, among the active ones with a key.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
    uint64_t m = __ballot(key >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? set : ~set;
    }
    return m;
}

// A wave's run of ids: at most STEPS steps of 64, whose keys stay in registers
// from the count to the placing (every load is issued before any use).  Its end is
// kept as a length: the last id may be number 2^31 - 2, and numbers past it wrap.
template <int STEPS>
struct Run {
    int key[STEPS];
    int i0, len;

    // ids [at, at + each) of a workgroup's ids [b, e), as far as there are any
    __device__ void load(const SortArgs &a, int b, int e, int at, int each, int lane) {
        at = min(at, e - b);
        i0 = b + at;
        len = min(each, e - i0);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) key[s] = 64 * s + lane < len ? sort_key(a, i0 + 64 * s + lane) : -1;
    }
    // cnt[key] += 1 per id (integer counts: the order does not matter)
    __device__ void count(int *cnt) const {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (key[s] >= 0) atomicAdd(cnt + key[s], 1);
    }
    // The places of the run's ids, in order, next[key] being the place of the
    // wave's next id of each expert: the ids of one step with the same key take
    // consecutive places in lane order.
    __device__ void place(const SortArgs &a, int *next, int lane) const {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (64 * s >= len) break;
            const uint64_t m = same_key(key[s], a.bits);
            const int rank = __popcll(m & ((1ull << lane) - 1));
            int at = -1;
            if (key[s] >= 0) at = __hip_atomic_load(next + key[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) + rank;
            __builtin_amdgcn_wave_barrier();   // every lane has read before the last of each key writes
            if (key[s] >= 0 && (m >> lane) == 1)
                __hip_atomic_store(next + key[s], at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            __builtin_amdgcn_wave_barrier();
            if (64 * s + lane < len) {
                const int i = i0 + 64 * s + lane;
                a.pos[i] = at;
                if (at >= 0) a.order[at] = i;
            }
        }
    }
};

// Exclusive scan of v[0..E) by one wave; returns the total.
__device__ __forceinline__ int wave_scan(int *v, int E, int lane) {
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane, x = e < E ? v[e] : 0;
        int s = x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int t = __shfl_up(s, d);
            if (lane >= d) s += t;
        }
        if (e < E) v[e] = carry + s - x;
        carry += __shfl(s, 63);
    }
    return carry;
}

// Bound by latency (512 ids over 64 experts: 3.4 to 4.2 us, of which a launch
// takes 1.5).  One workgroup sorts everything: each wave counts its own run of ids, the
// counts become starting places (experts first, then waves within an expert,
// which keeps the sort stable), and each wave places its run.
template <int STEPS>
__global__ void __launch_bounds__(SORT_T) moe_sort_one(SortArgs a) {
    extern __shared__ int lds[];              // cnt[SORT_W][E], total[E]
    int *total = lds + SORT_W * a.E;
    __shared__ int kept;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = ((a.n + SORT_T - 1) / SORT_T) * 64;   // ids per wave, whole steps
    Run<STEPS> r;
    r.load(a, 0, a.n, wave * run, run, lane);
    for (int i = tid; i < SORT_W * a.E; i += SORT_T) lds[i] = 0;
    __syncthreads();
    r.count(lds + wave * a.E);
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < SORT_W; ++w) s += lds[w * a.E + e];
        total[e] = s;
    }
    __syncthreads();
    if (wave == 0) {
        const int t = wave_scan(total, a.E, lane);
        if (lane == 0) kept = t;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = total[e];
        a.offsets[e] = s;
#pragma unroll
        for (int w = 0; w < SORT_W; ++w) {
            const int c = lds[w * a.E + e];
            lds[w * a.E + e] = s;
            s += c;
        }
    }
    if (tid == 0) a.offsets[a.E] = kept;
    for (int i = kept + tid; i < a.n; i += SORT_T) a.order[i] = -1;
    __syncthreads();
    r.place(a, lds + wave * a.E, lane);
}

// The three-launch sort.  Workgroup b owns a contiguous part of the ids (the
// parts differ by one id at most, and none is shorter than E).  Its part of
// pos, which it alone writes in the last launch, carries its E counts between
// the launches, so that the sort needs no scratch memory: counts
// (moe_sort_count), starting places (moe_sort_scan), then the places
// themselves (moe_sort_place).
__device__ __forceinline__ int block_start(const SortArgs &a, int b) {
    return b * (a.n / a.blocks) + min(b, a.n % a.blocks);
}

__global__ void __launch_bounds__(SORT_T) moe_sort_count(SortArgs a) {
    extern __shared__ int lds[];
    const int i0 = block_start(a, blockIdx.x), i1 = block_start(a, blockIdx.x + 1);
    int key[SORT_BLOCK / SORT_T];
#pragma unroll
    for (int s = 0; s < SORT_BLOCK / SORT_T; ++s) {
        const int i = i0 + s * SORT_T + threadIdx.x;
        key[s] = i < i1 ? sort_key(a, i) : -1;
    }
    for (int e = threadIdx.x; e < a.E; e += SORT_T) lds[e] = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SORT_BLOCK / SORT_T; ++s)
        if (key[s] >= 0) atomicAdd(lds + key[s], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += SORT_T) a.pos[i0 + e] = lds[e];
}

// One workgroup: each thread walks one expert's column of the count table over
// its run of blocks, SCAN_U counts at a time.
constexpr int SCAN_U = 16;
__global__ void __launch_bounds__(SORT_T) moe_sort_scan(SortArgs a) {
    extern __shared__ int lds[];              // part[parts][E], total[E]
    const int tid = threadIdx.x, lane = tid & 63;
    const int cols = min(a.E, SORT_T), parts = SORT_T / cols;
    int *total = lds + parts * a.E;
    __shared__ int kept;
    const int part = tid / cols, per = (a.blocks + parts - 1) / parts;
    const int b0 = min(part * per, a.blocks), b1 = part < parts ? min(b0 + per, a.blocks) : b0;
    // column e of blocks [b, b + SCAN_U): all loads, then f(block, count) in order
    auto column = [&](int e, int b, auto f) __attribute__((always_inline)) {
        int c[SCAN_U];
#pragma unroll
        for (int u = 0; u < SCAN_U; ++u) c[u] = b + u < b1 ? a.pos[block_start(a, b + u) + e] : 0;
#pragma unroll
        for (int u = 0; u < SCAN_U; ++u)
            if (b + u < b1) f(b + u, c[u]);
    };
    for (int e = tid % cols; e < a.E && part < parts; e += cols) {
        int s = 0;
        for (int b = b0; b < b1; b += SCAN_U) column(e, b, [&](int, int c) { s += c; });
        lds[part * a.E + e] = s;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = 0;
        for (int q = 0; q < parts; ++q) s += lds[q * a.E + e];
        total[e] = s;
    }
    __syncthreads();
    if (tid < 64) {
        const int t = wave_scan(total, a.E, lane);
        if (lane == 0) kept = t;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = total[e];
        a.offsets[e] = s;
        for (int q = 0; q < parts; ++q) {
            const int c = lds[q * a.E + e];
            lds[q * a.E + e] = s;
            s += c;
        }
    }
    if (tid == 0) a.offsets[a.E] = kept;
    __syncthreads();
    for (int e = tid % cols; e < a.E && part < parts; e += cols) {
        int s = lds[part * a.E + e];
        for (int b = b0; b < b1; b += SCAN_U)
            column(e, b, [&](int at, int c) {
                a.pos[block_start(a, at) + e] = s;
                s += c;
            });
    }
}

__global__ void __launch_bounds__(SORT_T) moe_sort_place(SortArgs a) {
    extern __shared__ int lds[];              // cnt[SORT_W][E]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b0 = block_start(a, blockIdx.x), b1 = block_start(a, blockIdx.x + 1);
    const int run = (b1 - b0 + SORT_T - 1) / SORT_T * 64;
    Run<SORT_BLOCK / SORT_T> r;
    r.load(a, b0, b1, wave * run, run, lane);
    const int kept = a.offsets[a.E];
    for (int i = tid; i < SORT_W * a.E; i += SORT_T) lds[i] = 0;
    __syncthreads();
    r.count(lds + wave * a.E);
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = a.pos[b0 + e];
#pragma unroll
        for (int w = 0; w < SORT_W; ++w) {
            const int c = lds[w * a.E + e];
            lds[w * a.E + e] = s;
            s += c;
        }
    }
    for (int64_t i = (int64_t)kept + blockIdx.x * SORT_T + tid; i < a.n; i += (int64_t)a.blocks * SORT_T) a.order[i] = -1;
    __syncthreads();   // every count of this workgroup's part of pos has been read
    r.place(a, lds + wave * a.E, lane);
}

// The two-launch sort, where a count table in the stream's workspace is at hand
// and small: the counts go there, and every workgroup of the last launch adds the
// columns of the table itself, whole (the experts' totals) and up to its own
// part, instead of waiting for one workgroup that does it for all.  Bound by the
// latencies of two launches (262144 ids over 256 experts: 13.3 us, three launches
// 17.5 us; 30208 over 8: 10.5 and 16.3 us).
template <int BLOCK>
__global__ void __launch_bounds__(SORT_T) moe_sort_table(SortArgs a) {
    extern __shared__ int lds[];
    const int i0 = block_start(a, blockIdx.x), i1 = block_start(a, blockIdx.x + 1);
    int key[BLOCK / SORT_T];
#pragma unroll
    for (int s = 0; s < BLOCK / SORT_T; ++s) {
        const int i = i0 + s * SORT_T + threadIdx.x;
        key[s] = i < i1 ? sort_key(a, i) : -1;
    }
    for (int e = threadIdx.x; e < a.E; e += SORT_T) lds[e] = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < BLOCK / SORT_T; ++s)
        if (key[s] >= 0) atomicAdd(lds + key[s], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += SORT_T) a.table[(int64_t)blockIdx.x * a.E + e] = lds[e];
}

template <int BLOCK>
__global__ void __launch_bounds__(SORT_T) moe_sort_place_table(SortArgs a) {
    extern __shared__ int lds[];              // cnt[SORT_W][E], all[parts][E], before[parts][E]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, me = blockIdx.x;
    const int b0 = block_start(a, me), b1 = block_start(a, me + 1);
    const int run = (b1 - b0 + SORT_T - 1) / SORT_T * 64;
    const int cols = min(a.E, SORT_T), parts = SORT_T / cols;
    int *all = lds + SORT_W * a.E, *before = all + parts * a.E;
    __shared__ int kept;
    Run<BLOCK / SORT_T> r;
    r.load(a, b0, b1, wave * run, run, lane);
    // the table's columns, SCAN_U counts in flight per thread
    const int part = tid / cols, per = (a.blocks + parts - 1) / parts;
    const int t0 = min(part * per, a.blocks), t1 = part < parts ? min(t0 + per, a.blocks) : t0;
    for (int e = tid % cols; e < a.E && part < parts; e += cols) {
        int s = 0, sb = 0;
        for (int b = t0; b < t1; b += SCAN_U) {
            int c[SCAN_U];
#pragma unroll
            for (int u = 0; u < SCAN_U; ++u) c[u] = b + u < t1 ? a.table[(int64_t)(b + u) * a.E + e] : 0;
#pragma unroll
            for (int u = 0; u < SCAN_U; ++u) {
                s += c[u];
                sb += b + u < me ? c[u] : 0;
            }
        }
        all[part * a.E + e] = s;
        before[part * a.E + e] = sb;
    }
    for (int i = tid; i < SORT_W * a.E; i += SORT_T) lds[i] = 0;
    __syncthreads();
    r.count(lds + wave * a.E);
    for (int e = tid; e < a.E; e += SORT_T) {
        int s = 0, sb = 0;
        for (int q = 0; q < parts; ++q) {
            s += all[q * a.E + e];
            sb += before[q * a.E + e];
        }
        all[e] = s;
        before[e] = sb;
    }
    __syncthreads();
    if (wave == 0) {
        const int t = wave_scan(all, a.E, lane);
        if (lane == 0) kept = t;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += SORT_T) {
        if (me == 0) a.offsets[e] = all[e];
        int s = all[e] + before[e];
#pragma unroll
        for (int w = 0; w < SORT_W; ++w) {
            const int c = lds[w * a.E + e];
            lds[w * a.E + e] = s;
            s += c;
        }
    }
    if (me == 0 && tid == 0) a.offsets[a.E] = kept;
    for (int64_t i = (int64_t)kept + (int64_t)me * SORT_T + tid; i < a.n; i += (int64_t)a.blocks * SORT_T) a.order[i] = -1;
    __syncthreads();
    r.place(a, lds + wave * a.E, lane);
}

// ------------------------------------------------------------------ row chunks

// A row's elements in chunks of 16 bytes.  VEC rows are contiguous: one access
// of 16 bytes at any alignment for a whole chunk, element accesses for the
// row's last, partial one; other rows take element accesses throughout.
template <int EB> struct Chunk {
    static constexpr int N = 16 / EB;
    union { u32x4 v; uint8_t b[16]; uint16_t h[8]; uint32_t w[4]; };

    __device__ void get(int e, const char *p) {
        if (EB == 1) b[e] = *reinterpret_cast<const uint8_t *>(p);
        else if (EB == 2) h[e] = *reinterpret_cast<const uint16_t *>(p);
        else w[e] = *reinterpret_cast<const uint32_t *>(p);
    }
    __device__ void put(int e, char *p) const {
        if (EB == 1) *reinterpret_cast<uint8_t *>(p) = b[e];
        else if (EB == 2) *reinterpret_cast<uint16_t *>(p) = h[e];
        else *reinterpret_cast<uint32_t *>(p) = w[e];
    }
    // elements c * N .. of the row at p, `left` of them inside the row
    __device__ void load(const char *p, int64_t cs, int c, int left, int vec) {
        p += (int64_t)c * N * cs;
        if (vec && left >= N) {
            v = *reinterpret_cast<const u32x4_any *>(p);
        } else {
            v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e < left) get(e, p + e * cs);
        }
    }
    // STREAM: past the caches
    template <bool STREAM = false>
    __device__ void store(char *p, int64_t cs, int c, int left, int vec) const {
        p += (int64_t)c * N * cs;
        if (vec && left >= N) {
            if (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(p));
            else *reinterpret_cast<u32x4_any *>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e < left) put(e, p + e * cs);
        }
    }
};

// Chunks of floats of an element kind (OutKind).
template <int KIND> struct Vals {
    static constexpr int EB = KIND == OUT_F32 ? 4 : 2, N = 16 / EB;
    static __device__ float get(const Chunk<EB> &c, int e) {
        if (KIND == OUT_F32) return __builtin_bit_cast(float, c.w[e]);
        return KIND == OUT_BF16 ? bf16_bits_to_f32(c.h[e]) : f16_bits_to_f32(c.h[e]);
    }
    static __device__ void set(Chunk<EB> &c, int e, float x) {
        if (KIND == OUT_F32) c.w[e] = __builtin_bit_cast(uint32_t, x);
        else c.h[e] = KIND == OUT_BF16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x);
    }
};

// Lanes that share a row: the power of two that holds its chunks, at most a wave.
int lanes_of(int chunks) {
    int l = 1;
    while (l < chunks && l < 64) l *= 2;
    return l;
}

constexpr int NT = 256;
constexpr int GATHER_U = 4;   // chunks of a row that a lane holds at once

// ------------------------------------------------------------------ gather

// Xs[r] = X[order[r] / k].  A copy, bound by the bytes (16384 rows of 4096 BF16 45.0
// us, 4.5 TB/s; 32768 rows, past the caches (a.stream), 80.3 us, 5.0 TB/s; a plain
// copy of 1 GiB reaches 5.15): `lanes` lanes walk one piece (GATHER_U * lanes chunks)
// of a row, all of its loads before its stores.
template <int EB, bool STREAM>
__global__ void __launch_bounds__(NT) moe_gather_rows(GatherArgs a, int lanes, int pieces) {
    constexpr int CN = Chunk<EB>::N;
    const int64_t u = ((int64_t)blockIdx.x * NT + threadIdx.x) / lanes;
    const int64_t r = u / pieces;
    if (r >= a.n) return;
    const int c0 = (int)(u % pieces) * GATHER_U * lanes + threadIdx.x % lanes;
    const int o = *reinterpret_cast<const int *>(a.order + r * a.o_s);
    const int t = o >= 0 ? o / a.k : -1;
    const bool in = t >= 0 && t < a.T;
    const char *src = a.X + (int64_t)(in ? t : 0) * a.x_rs;
    char *dst = a.Y + r * a.y_rs;
    Chunk<EB> v[GATHER_U];
#pragma unroll
    for (int q = 0; q < GATHER_U; ++q) {
        const int c = c0 + q * lanes;
        v[q].v = u32x4{0u, 0u, 0u, 0u};
        if (in && c * CN < a.H) v[q].load(src, a.x_cs, c, a.H - c * CN, a.vec);
    }
#pragma unroll
    for (int q = 0; q < GATHER_U; ++q) {
        const int c = c0 + q * lanes;
        if (c * CN < a.H) v[q].template store<STREAM>(dst, a.y_cs, c, a.H - c * CN, a.vec);
    }
}

// ------------------------------------------------------------------ combine

constexpr int KU = 8;   // experts of a token handled together

__device__ __forceinline__ int pos_of(const CombineArgs &a, int64_t t, int j) {
    const int p = *reinterpret_cast<const int *>(a.pos + t * a.p_rs + j * a.p_cs);
    return p >= 0 && p < a.R ? p : -1;
}
__device__ __forceinline__ float weight_of(const CombineArgs &a, int64_t t, int j) {
    return a.w ? load_out(a.w + t * a.w_rs + j * a.w_cs, a.w_kind) : 1.0f;
}

// Y[t] = sum over j of w[t][j] * Ys[pos[t][j]], in FP32 in the order of j,
// rounded once (48 tokens of 8 experts, 2048 BF16: 4.7 us, bound by latency; 4096
// tokens 40 us, 3.7 TB/s).  A lane owns one chunk of a token's row and has the loads of
// up to KU experts' rows in flight; `pieces` runs of `lanes` chunks make a row.
template <int KIND>
__global__ void __launch_bounds__(NT) moe_combine_rows(CombineArgs a, int lanes, int pieces) {
    using V = Vals<KIND>;
    constexpr int CN = V::N;
    const int64_t u = ((int64_t)blockIdx.x * NT + threadIdx.x) / lanes;
    const int64_t t = u / pieces;
    const int c = (int)(u % pieces) * lanes + threadIdx.x % lanes, left = a.H - c * CN;
    if (t >= a.T || left <= 0) return;
    float sum[CN];
#pragma unroll
    for (int e = 0; e < CN; ++e) sum[e] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += KU) {
        int p[KU];
        float w[KU];
        Chunk<V::EB> y[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            p[j] = j0 + j < a.k ? pos_of(a, t, j0 + j) : -1;
            w[j] = j0 + j < a.k ? weight_of(a, t, j0 + j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KU; ++j)
            if (p[j] >= 0) y[j].load(a.Ys + (int64_t)p[j] * a.s_rs, a.s_cs, c, left, a.vec);
#pragma unroll
        for (int j = 0; j < KU; ++j)
            if (p[j] >= 0) {   // a dropped choice adds nothing, whatever its weight holds
#pragma unroll
                for (int e = 0; e < CN; ++e) sum[e] = fmaf(w[j], V::get(y[j], e), sum[e]);
            }
    }
    Chunk<V::EB> out;
#pragma unroll
    for (int e = 0; e < CN; ++e) V::set(out, e, sum[e]);
    out.store(a.Y + t * a.y_rs, a.y_cs, c, left, a.vec);
}

// ------------------------------------------------------------------ gradient of combine

constexpr int ZERO_ROWS_MAX = 1 << 16;   // rows per clearing workgroup: 8 KB of LDS bits

// Rows [r0, r1) of dYs that no pos names are set to zero: the workgroup marks
// the named ones in a bit map, then clears the others.
template <int EB>
__device__ __forceinline__ void clear_unnamed(const CombineArgs &a, uint32_t *bits, int b) {
    const int64_t r0 = (int64_t)b * a.zero_rows, r1 = min<int64_t>(r0 + a.zero_rows, a.R);
    for (int i = threadIdx.x; i < (a.zero_rows + 31) / 32; i += NT) bits[i] = 0;
    __syncthreads();
    const int64_t n = (int64_t)a.T * a.k;
    auto mark = [&](int64_t at) __attribute__((always_inline)) {
        if (at >= r0 && at < r1) atomicOr(bits + ((at - r0) >> 5), 1u << ((at - r0) & 31));
    };
    // pos whole, 16 bytes a load where it is one run (4 loads in flight)
    const int64_t quads = a.p_run ? n / 4 : 0;
    for (int64_t i0 = 0; i0 < quads; i0 += 4 * NT) {
        u32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t i = i0 + q * NT + threadIdx.x;
            v[q] = i < quads ? *reinterpret_cast<const u32x4_any *>(a.pos + 16 * i) : u32x4{~0u, ~0u, ~0u, ~0u};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) mark((int)v[q][e]);
    }
    for (int64_t i = 4 * quads + threadIdx.x; i < n; i += NT)
        mark(*reinterpret_cast<const int *>(a.p_run ? a.pos + 4 * i : a.pos + (i / a.k) * a.p_rs + (i % a.k) * a.p_cs));
    __syncthreads();
    Chunk<EB> zero;
    zero.v = u32x4{0u, 0u, 0u, 0u};
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int64_t r = r0 + wave; r < r1; r += NT / 64) {
        if (bits[(r - r0) >> 5] >> ((r - r0) & 31) & 1) continue;
        for (int c = lane; c * Chunk<EB>::N < a.H; c += 64)
            zero.store(a.dYs + r * a.d_rs, a.d_cs, c, a.H - c * Chunk<EB>::N, a.vec);
    }
}

// dYs[pos[t][j]] = w[t][j] * dY[t] and dw[t][j] = <dY[t], Ys[pos[t][j]]>, the
// token's row of dY read once for up to KU experts.  Bound by the bytes (4096
// tokens of 8 experts, 2048 BF16: 65 us, 4.4 TB/s).  WPT waves share a token
// (WPT = 1: `lanes` lanes do); the dot products are summed in FP32, over a
// lane's chunks, then the lanes, then the waves, always in that order.  The
// first zero_blocks workgroups clear the rows of dYs that no pos names.
template <int KIND, int WPT>
__global__ void __launch_bounds__(NT) moe_combine_grad_rows(CombineArgs a, int lanes) {
    using V = Vals<KIND>;
    constexpr int CN = V::N, EB = V::EB;
    __shared__ uint32_t bits[ZERO_ROWS_MAX / 32];
    __shared__ float part[NT / 64][KU];
    if ((int)blockIdx.x < a.zero_blocks) {
        clear_unnamed<EB>(a, bits, blockIdx.x);
        return;
    }
    const int64_t b = blockIdx.x - a.zero_blocks;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int span = WPT > 1 ? NT : lanes;                       // lanes of a token
    const int64_t t = WPT > 1 ? b : (b * NT + threadIdx.x) / lanes;
    const int me = threadIdx.x % span;
    const bool in = t < a.T;                                     // (WPT > 1: always)
    for (int j0 = 0; j0 < a.k; j0 += KU) {
        int p[KU];
        float w[KU], dot[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            p[j] = in && j0 + j < a.k ? pos_of(a, t, j0 + j) : -1;
            w[j] = in && j0 + j < a.k ? weight_of(a, t, j0 + j) : 0.0f;
            dot[j] = 0.0f;
            // kept in vector registers: 2 x KU row addresses as scalars would spill
            asm volatile("" : "+v"(p[j]));
        }
        const int whole = in && a.vec ? a.H / CN : 0;
        // whole chunks: all of a chunk's loads, then the products and stores
#pragma unroll 1
        for (int c = me; c < whole; c += span) {
            Chunk<EB> g, y[KU];
            g.load(a.Y + t * a.y_rs, EB, c, CN, 1);
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < KU; ++j)
                    if (p[j] >= 0) y[j].load(a.Ys + (int64_t)p[j] * a.s_rs, EB, c, CN, 1);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if (p[j] >= 0) {
                    Chunk<EB> d;
#pragma unroll
                    for (int e = 0; e < CN; ++e) {
                        const float x = V::get(g, e);
                        if (a.dw) dot[j] = fmaf(x, V::get(y[j], e), dot[j]);
                        V::set(d, e, w[j] * x);
                    }
                    d.store(a.dYs + (int64_t)p[j] * a.d_rs, EB, c, CN, 1);
                }
        }
        // the row's last elements, or all of them where a row is not contiguous
#pragma unroll 1
        for (int h = whole * CN + me; in && h < a.H; h += span) {
            const float x = load_out(a.Y + t * a.y_rs + h * a.y_cs, KIND);
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if (p[j] >= 0) {
                    if (a.dw) dot[j] = fmaf(x, load_out(a.Ys + (int64_t)p[j] * a.s_rs + h * a.s_cs, KIND), dot[j]);
                    store_out(a.dYs + (int64_t)p[j] * a.d_rs + h * a.d_cs, KIND, w[j] * x);
                }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int j = 0; j < KU; ++j)
            for (int s = (WPT > 1 ? 64 : lanes) / 2; s > 0; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
        if (WPT > 1) {
            __syncthreads();
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < KU; ++j) part[wave][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < KU && j0 + (int)threadIdx.x < a.k) {
                const int j = threadIdx.x;
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < WPT; ++q) s += part[q][j];
                store_out(a.dw + t * a.g_rs + (j0 + j) * a.g_cs, a.w_kind, s);
            }
        } else if (in && me == 0) {
#pragma unroll
            for (int j = 0; j < KU; ++j)
                if (j0 + j < a.k) store_out(a.dw + t * a.g_rs + (j0 + j) * a.g_cs, a.w_kind, dot[j]);
        }
    }
}

int64_t blocks(int64_t threads) { return (threads + NT - 1) / NT; }

}  // namespace

namespace {
// More than 64 KB of dynamic LDS (many experts) needs the kernel's attribute.
template <class Kernel>
hipError_t allow_lds(Kernel k, size_t bytes) {
    if (bytes <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
}  // namespace

hipError_t launch_moe_sort(const SortArgs &a, hipStream_t s) {
    hipError_t e;
    if (a.table) {
        const int cols = a.E < SORT_T ? a.E : SORT_T, parts = SORT_T / cols;
        const size_t lds = (size_t)(SORT_W + 2 * parts) * a.E * sizeof(int);
        const bool small = sort_table_block(a.n) == 2048;
        const auto count = small ? moe_sort_table<2048> : moe_sort_table<4096>;
        const auto place = small ? moe_sort_place_table<2048> : moe_sort_place_table<4096>;
        if ((e = allow_lds(place, lds)) != hipSuccess) return e;
        hipLaunchKernelGGL(count, dim3(a.blocks), dim3(SORT_T), a.E * sizeof(int), s, a);
        hipLaunchKernelGGL(place, dim3(a.blocks), dim3(SORT_T), lds, s, a);
        return hipGetLastError();
    }
    if (a.n <= SORT_ONE_MAX) {
        const size_t lds = (SORT_W + 1) * a.E * sizeof(int);
        const int steps = sort_steps(a.n);
        const auto k = steps == 1 ? moe_sort_one<1> : steps == 4 ? moe_sort_one<4> : moe_sort_one<SORT_ONE_MAX / SORT_T>;
        if ((e = allow_lds(k, lds)) != hipSuccess) return e;
        hipLaunchKernelGGL(k, dim3(1), dim3(SORT_T), lds, s, a);
        return hipGetLastError();
    }
    const int cols = a.E < SORT_T ? a.E : SORT_T, parts = SORT_T / cols;
    if ((e = allow_lds(moe_sort_place, SORT_W * a.E * sizeof(int))) != hipSuccess) return e;
    hipLaunchKernelGGL(moe_sort_count, dim3(a.blocks), dim3(SORT_T), a.E * sizeof(int), s, a);
    hipLaunchKernelGGL(moe_sort_scan, dim3(1), dim3(SORT_T), (parts + 1) * a.E * sizeof(int), s, a);
    hipLaunchKernelGGL(moe_sort_place, dim3(a.blocks), dim3(SORT_T), SORT_W * a.E * sizeof(int), s, a);
    return hipGetLastError();
}

// A launch holds fewer than 2^32 threads: rows of `per_row` threads go out in runs
// of at most 2^31, launch(first row, rows) each.
template <class Launch>
static hipError_t in_runs(int64_t rows, int64_t per_row, Launch launch) {
    const int64_t most = std::max<int64_t>(((int64_t)1 << 31) / per_row, 1);
    for (int64_t r = 0; r < rows; r += most) {
        launch(r, std::min(most, rows - r));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_moe_gather(const GatherArgs &all, hipStream_t s) {
    const int cn = 16 / all.esize, chunks = (all.H + cn - 1) / cn, lanes = lanes_of(chunks);
    const int pieces = (chunks + GATHER_U * lanes - 1) / (GATHER_U * lanes);
    return in_runs(all.n, (int64_t)pieces * lanes, [&](int64_t r, int64_t rows) {
        GatherArgs a = all;
        a.Y += r * a.y_rs;
        a.order += r * a.o_s;
        a.n = (int)rows;
        const dim3 g((unsigned)blocks(rows * pieces * lanes));
        switch (a.esize) {
        case 1: hipLaunchKernelGGL((a.stream ? moe_gather_rows<1, true> : moe_gather_rows<1, false>), g, dim3(NT), 0, s, a, lanes, pieces); break;
        case 2: hipLaunchKernelGGL((a.stream ? moe_gather_rows<2, true> : moe_gather_rows<2, false>), g, dim3(NT), 0, s, a, lanes, pieces); break;
        default: hipLaunchKernelGGL((a.stream ? moe_gather_rows<4, true> : moe_gather_rows<4, false>), g, dim3(NT), 0, s, a, lanes, pieces); break;
        }
    });
}

// Tokens from t on, `tokens` of them.
static CombineArgs tokens_from(CombineArgs a, int64_t t, int64_t tokens) {
    a.Y += t * a.y_rs;
    a.pos += t * a.p_rs;
    if (a.w) a.w += t * a.w_rs;
    if (a.dw) a.dw += t * a.g_rs;
    a.T = (int)tokens;
    return a;
}

hipError_t launch_moe_combine(int kind, const CombineArgs &all, hipStream_t s) {
    const int cn = kind == OUT_F32 ? 4 : 8, chunks = (all.H + cn - 1) / cn, lanes = lanes_of(chunks);
    const int pieces = (chunks + lanes - 1) / lanes;
    return in_runs(all.T, (int64_t)pieces * lanes, [&](int64_t t, int64_t tokens) {
        const CombineArgs a = tokens_from(all, t, tokens);
        const dim3 g((unsigned)blocks(tokens * pieces * lanes));
        switch (kind) {
        case OUT_F32: hipLaunchKernelGGL(moe_combine_rows<OUT_F32>, g, dim3(NT), 0, s, a, lanes, pieces); break;
        case OUT_F16: hipLaunchKernelGGL(moe_combine_rows<OUT_F16>, g, dim3(NT), 0, s, a, lanes, pieces); break;
        default: hipLaunchKernelGGL(moe_combine_rows<OUT_BF16>, g, dim3(NT), 0, s, a, lanes, pieces); break;
        }
    });
}

namespace {
template <int KIND>
hipError_t grad_kind(CombineArgs all, hipStream_t s) {
    const int chunks = (all.H + Vals<KIND>::N - 1) / Vals<KIND>::N, lanes = lanes_of(chunks);
    // clearing workgroups: 32, more where their rows would not fit the bit map
    all.zero_rows = (int)std::min<int64_t>(ZERO_ROWS_MAX, ((int64_t)all.R + 31) / 32);
    const int zero_blocks = all.zero_rows ? (int)(((int64_t)all.R + all.zero_rows - 1) / all.zero_rows) : 0;
    // a row of at least 128 chunks gives each of a workgroup's 4 waves 32 lanes of work
    // (48 tokens of 8 experts, 1024 BF16: 5.0 us, 9.1 with a wave a token; 768: 9.0,
    // 5.0 with four; 4096 tokens of 2: 768 16.1, 18.1 with four)
    const bool wide = chunks >= 128;
    const int64_t per_token = wide ? NT : lanes;
    auto launch = [&](CombineArgs a, int zeros, int64_t tokens) {
        a.zero_blocks = zeros;
        const dim3 g((unsigned)(zeros + blocks(tokens * per_token)));
        if (wide) hipLaunchKernelGGL((moe_combine_grad_rows<KIND, NT / 64>), g, dim3(NT), 0, s, a, lanes);
        else hipLaunchKernelGGL((moe_combine_grad_rows<KIND, 1>), g, dim3(NT), 0, s, a, lanes);
    };
    if (all.T * per_token <= (int64_t)1 << 31) {
        if (zero_blocks == 0 && all.T == 0) return hipSuccess;
        launch(all, zero_blocks, all.T);
        return hipGetLastError();
    }
    // (the clearing workgroups read the places of every token)
    if (zero_blocks) launch(all, zero_blocks, 0);
    return in_runs(all.T, per_token, [&](int64_t t, int64_t tokens) { launch(tokens_from(all, t, tokens), 0, tokens); });
}
}  // namespace

hipError_t launch_moe_combine_grad(int kind, const CombineArgs &a, hipStream_t s) {
    switch (kind) {
    case OUT_F32: return grad_kind<OUT_F32>(a, s);
    case OUT_F16: return grad_kind<OUT_F16>(a, s);
    default: return grad_kind<OUT_BF16>(a, s);
    }
}

}  // namespace dg
