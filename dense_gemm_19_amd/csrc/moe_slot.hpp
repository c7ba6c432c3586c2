// moe_slot.hpp -- from a workgroup to its expert and tile, by the offsets in
// device memory (shared by the experts' products).
#pragma once
#include "device_common.hpp"

namespace dg {
namespace moe {

// Workgroup b of `total` -> unit: each XCD (b % 8) takes a contiguous run of
// units, so that neighbouring tiles, which share operands, share an L2.
__device__ __forceinline__ int xcd_run(int b, int total) {
    const int x = b & 7, q = total >> 3, r = total & 7;
    return x * q + min(x, r) + (b >> 3);
}

// Inclusive sum over the wave's lanes up to this one.
__device__ __forceinline__ int lane_sum(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int t = __shfl_up(v, d);
        if (lane >= d) v += t;
    }
    return v;
}

// One expert's rows and this workgroup's unit within its tiles (wave-uniform).
// e == E: the rows that belong to no expert (from offsets[E] on).  above: rows
// of tiles of the groups before it.
struct Slot { int e, begin, rows, unit, above; };

// Rows [begin, end) of group e (e == E: the rest up to n).  Offsets are clamped
// into [0, n], so that no value of theirs reaches outside the operands.
__device__ __forceinline__ void group_rows(const char *off, int64_t o_s, int E, int n, int e, int &b, int &rows) {
    auto at = [&](int i) { return min(max(*reinterpret_cast<const int *>(off + i * o_s), 0), n); };
    b = e <= E ? at(e) : n;
    const int t = e < E ? at(e + 1) : n;
    rows = max(t - b, 0);
}

// The slot of workgroup b: groups in order, each with ceil(rows / BM) * tiles_n
// units (tiles_n: units per row of tiles).  False: b is past the last unit, or
// the offsets name more than the grid's `units`, which only overlapping groups
// can (n is at most 2^28, so that 64 groups' tile rows fit 32 bits).  Every wave
// does this by itself, so a call's scans grow with the square of E (4096 rows of 63
// experts, 512 -> 1024: 16.5 us where there are no others, 58 us among 256, 107 among
// 512, 273 among 1024, 893 among 2048), and E is bounded (MOE_MAX_SCANNED).
template <int BM>
__device__ __forceinline__ bool find_slot(const char *off, int64_t o_s, int E, int n, int tiles_n, int units, int b, Slot &s) {
    const int lane = threadIdx.x & 63;
    int begin, rows;
    group_rows(off, o_s, E, n, lane, begin, rows);
    int mine = lane <= E ? (rows + BM - 1) / BM : 0;
    int upto = lane_sum(mine, lane);
    int64_t total = __builtin_amdgcn_readlane(upto, 63);
    for (int e0 = 64; e0 <= E; e0 += 64) {   // more than 63 experts: the tiles of the rest
        int bb, rr;
        group_rows(off, o_s, E, n, e0 + lane, bb, rr);
        total += __builtin_amdgcn_readlane(lane_sum(e0 + lane <= E ? (rr + BM - 1) / BM : 0, lane), 63);
    }
    total *= tiles_n;
    if (b >= total || total > units) return false;
    const int u = xcd_run(b, (int)total);
    const int want = u / tiles_n;            // tile row among all groups'
    int base = 0, e0 = 0;
    while (true) {
        const uint64_t past = __ballot(base + upto > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            s.e = e0 + l;
            s.begin = __builtin_amdgcn_readlane(begin, l);
            s.rows = __builtin_amdgcn_readlane(rows, l);
            s.above = base + __builtin_amdgcn_readlane(upto - mine, l);
            s.unit = u - s.above * tiles_n;
            return true;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
        e0 += 64;
        if (e0 > E) return false;            // (never: want < total)
        group_rows(off, o_s, E, n, e0 + lane, begin, rows);
        mine = e0 + lane <= E ? (rows + BM - 1) / BM : 0;
        upto = lane_sum(mine, lane);
    }
}

}  // namespace moe
}  // namespace dg
