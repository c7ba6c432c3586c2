// moe.hpp -- argument blocks and launchers of the mixture-of-experts operators
// (host and device).  All strides are in bytes.
#pragma once
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "kernels.hpp"

namespace dg {

// The kernels walk an extent in 32 bits and may step past its end by less than a
// tile or a wave's chunks: 256 columns, 64 chunks of 16 elements.
constexpr int64_t MOE_MAX_EXTENT = INT32_MAX - 4095;

// ---------------------------------------------------------------- routing (moe_route.hip)

constexpr int MOE_MAX_EXPERTS = 2048;    // LDS counters of a sort workgroup: 16 waves x E
constexpr int MOE_MAX_ROWS = 1 << 28;     // of the experts' products: tile counts of 64 experts fit 32 bits
constexpr int MOE_MAX_SCANNED = 1 << 14; // experts of the products whose workgroups scan the offsets (find_slot)
constexpr int SORT_T = 1024;             // threads of a sort workgroup
constexpr int SORT_ONE_MAX = 16384;      // ids sorted by one workgroup; more take two launches or three
// Ids a thread of that workgroup holds at most: few where few ids allow it, for
// fewer registers and instructions to fetch (512 ids: 3.4 us, 3.9 with 16).
constexpr int sort_steps(int n) { return n <= SORT_T ? 1 : n <= 4 * SORT_T ? 4 : SORT_ONE_MAX / SORT_T; }
constexpr int SORT_BLOCK = 4096;         // ids per workgroup of the three-launch sort (at least E fit half of it)
// ids per workgroup of the two-launch sort: few ids want more workgroups (30208: 10.5
// us, 11.9 with 4096), many a smaller table (262144 over 256 experts: 14.7, 15.1 with 2048)
constexpr int sort_table_block(int64_t n) { return n <= 1 << 17 ? 2048 : 4096; }
// ids from which two launches are mostly quicker than one workgroup (64 experts: 6000
// ids 8.0 us, one workgroup 7.8; 8192 7.9 and 9.2; 16384 8.3 and 15.3; 8 experts: 8192
// 9.7 and 8.5)
constexpr int SORT_TABLE_MIN = 8192;
// counts that every workgroup of the two-launch sort reads at most (32768 of them:
// 16.3 us, three launches 21.7; 65536 would still be quicker, 22.8 and 30.4)
constexpr int SORT_TABLE_MAX = 1 << 15;

struct SortArgs {
    const char *ids; int64_t i_rs, i_cs;   // [T][k]
    int wide;                              // ids are 64-bit integers
    int k, n;                              // n = T * k
    int E, bits;                           // E < 2^bits + 1: every expert id fits `bits` bits
    int *offsets, *order, *pos;            // contiguous: [E + 1], [n], [T][k]
    int blocks;                            // workgroups of the two- and three-launch sorts
    int *table;                            // two launches: [blocks][E] counts, or null
};

struct GatherArgs {
    const char *X; int64_t x_rs, x_cs;     // [T][H]
    char *Y; int64_t y_rs, y_cs;           // [n][H]
    const char *order; int64_t o_s;        // [n] int32
    int T, k, n, H, esize;
    int vec;                               // both operands' rows are contiguous
    int stream;                            // stores past the caches
};

// combine (Y = sum of w * Ys) and its gradient (dYs = w * dY, dw = <dY, Ys>)
struct CombineArgs {
    const char *Ys; int64_t s_rs, s_cs;    // [R][H]
    char *Y; int64_t y_rs, y_cs;           // [T][H]: written by combine, read by its gradient
    const char *pos; int64_t p_rs, p_cs;   // [T][k] int32
    const char *w; int64_t w_rs, w_cs;     // [T][k], or null (weights of 1)
    int w_kind;                            // OutKind numbering
    char *dYs; int64_t d_rs, d_cs;         // gradient: [R][H]
    char *dw; int64_t g_rs, g_cs;          // gradient: [T][k] in w_kind, or null
    int T, k, R, H;
    int vec;                               // every operand's rows are contiguous
    int p_run;                             // pos is one contiguous run
    int zero_blocks, zero_rows;            // gradient: workgroups that clear unnamed rows, rows of each
};

hipError_t launch_moe_sort(const SortArgs &a, hipStream_t stream);
hipError_t launch_moe_gather(const GatherArgs &a, hipStream_t stream);
// kind: OutKind numbering of Ys, Y and dYs
hipError_t launch_moe_combine(int kind, const CombineArgs &a, hipStream_t stream);
hipError_t launch_moe_combine_grad(int kind, const CombineArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- expert products (moe_gemm.hpp)

// p describes one expert's product with the whole operands' pointers; the
// kernel adds the expert's offsets.  Forward: A's rows are grouped (M is the
// expert's row count), B moves by e_bs per expert.  Weight gradient (wgrad): K
// is the expert's row count, C moves by e_cs per expert.
struct MoeArgs {
    MfmaArgs p;
    const char *offsets; int64_t o_s;      // [E + 1] int32
    int E, n;                              // experts, grouped rows
    int units;                             // forward: workgroups of the grid
    int64_t e_bs, e_cs;                    // bytes per expert of B (forward) and C (wgrad)
};

// Loaders of the expert products.
//  MOE_DTL : direct HBM -> LDS loads (gemm_dtl.hpp): 16-byte aligned chunks.
//  MOE_VEC : register-staged 16-byte loads at any alignment; the operands are
//            contiguous along one of their dims, at least 8 long.
//  MOE_ELEM: element loads, any strides.
enum MoeLoad : int { MOE_DTL = 0, MOE_VEC = 1, MOE_ELEM = 2 };
constexpr int MOE_T192 = NUM_MFMA_TILES;   // MOE_DTL, forward: 192 x 256

// tile: MfmaTile or MOE_T192 (T64x128 here stands for the 32 x 128 tile of MOE_DTL).
// units: an upper bound of the work units (forward) or their number (wgrad).
hipError_t launch_moe_gemm_f16(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units,
                               hipStream_t stream);
hipError_t launch_moe_gemm_bf16(int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units,
                                hipStream_t stream);

// ---------------------------------------------------------------- 4-bit weights (w4.hip)

struct W4Args {
    const char *A; int64_t a_rs;           // [M][K] 16-bit, K-contiguous
    const char *Q; int64_t q_rs, q_es;     // [E][N][ceil(K/2)] bytes, K-contiguous
    const char *S; int64_t s_rs, s_cs, s_es;   // [E][N][ceil(K/G)]
    const char *Z; int64_t z_rs, z_cs, z_es;   // [E][N][ceil(K/G)] bytes, or null (8)
    int s_kind;                            // OutKind numbering
    char *C; int64_t c_rs, c_cs;
    int out_kind, act;
    int M, N, K, G, groups;                // groups = ceil(K / G)
    uint32_t g_mul;                        // ceil(2^32 / (G / 32)), 0 for G = 32
    const char *offsets; int64_t o_s; int E;   // offsets null: one group of all M rows
    int slabs;                             // column slabs of w4_cols(tm)
    int chunks, splits;                    // K in pieces of `chunks` chunks; splits > 1: one matrix only
    float *ws; int *counters;              // splits > 1: [tiles][splits][16 tm x w4_cols(tm)] sums, a counter per tile (0)
    int units;                             // workgroups of the grid
    int whole;                             // A and Q in aligned 16-byte pieces, scales and zero points in words that hold nothing else: w4_whole
    uint32_t s_mul, z_mul;                 // whole: ceil(2^32 / (pitch / 4)), to divide by it
    int depth;                             // whole: code units per wave in LDS (2 to 4)
    int a_lds;                             // LDS bytes for A: at least one chunk of 16 tm (or all M) rows
    int seg, seg_groups;                   // chunks whose scales are in LDS together, groups they touch at most
    int s_pitch, z_pitch;                  // bytes of a column's scales and zero points in LDS
    int lds_bytes;
};

// Geometry of the kernel by rows / 16 of a workgroup: columns, K elements of a
// chunk.  Few rows take narrow slabs, whose LDS
// lets two workgroups share a CU; more rows take shorter chunks, whose A fits.
constexpr int W4_MAX_TM = 3;
constexpr int w4_cols(int tm) { return tm == 1 ? 32 : 64; }
constexpr int w4_chunk(int tm) { return tm == 1 ? 1024 : 512; }

// tm: rows of a workgroup / 16, 1 to W4_MAX_TM (4, whose chunk of A leaves LDS
// no room for a second, took 26 us for 248 x 1452 x 2592 where 3 takes 14.2 to 21)
hipError_t launch_w4(int in_kind, int tm, const W4Args &a, int64_t units, hipStream_t stream);

}  // namespace dg
