// mx4.hpp -- argument blocks and launchers of the microscaled 4-bit (MXFP4) operators
// (host and device).  All strides are in bytes.
//
// A matrix of codes is [rows][ceil(K / 2)] bytes, rows contiguous; its scales are
// [rows][ceil(K / 32)] bytes with any strides.
#pragma once
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "kernels.hpp"

namespace dg {

// ---------------------------------------------------------------- quantiser (mx4_quant.hip)

constexpr int MX4_RUN = 4;         // 8-element chunks of a thread (rows kernels), or one
constexpr int MX4_TILE_M = 256;    // tile of the columns kernel: rows of X, and K
constexpr int MX4_TILE_K = 128;

struct Mx4QuantArgs {
    const char *X; int64_t x_es, x_rs, x_cs;   // [E][M][K]
    char *Q; int64_t q_es, q_rs;               // [E][M][ceil(K / 2)]
    char *S; int64_t s_es, s_rs, s_cs;         // [E][M][ceil(K / 32)]
    int x_kind;                                // OutKind numbering
    int M, K, E;
    int chunks;                                // of a row: 4 * ceil(K / 32)
    uint32_t chunk_mul;                        // ceil(2^32 / chunks), for chunks < 4096
    int run;                                   // 1 or MX4_RUN
    int tiles_m, tiles_k;                      // columns kernel
    int ceil;                                  // the scale at which nothing saturates
    int vec;                                   // columns kernel: rows of X are adjacent
};

// by_columns: X's rows are not contiguous.
hipError_t launch_mx4_quant(bool by_columns, const Mx4QuantArgs &a, int64_t units, hipStream_t stream);

struct Mx4DequantArgs {
    const char *Q; int64_t q_es, q_rs;
    const char *S; int64_t s_es, s_rs, s_cs;
    char *Y; int64_t y_es, y_rs, y_cs;         // [E][M][K]
    int y_kind;
    int M, K, E;
    int chunks, run;
    uint32_t chunk_mul;
    int vec;                                   // rows of Y are contiguous
};
hipError_t launch_mx4_dequant(const Mx4DequantArgs &a, int64_t units, hipStream_t stream);

// ---------------------------------------------------------------- products (mx4_gemm.hip)

// C[m][n] = act(sum over k of A[m][k] W[n][k]), W in MXFP4, A too or in 16 bits.
struct Mx4GemmArgs {
    const char *A; int64_t a_rs;               // [M][row_bytes] codes, or [M][K] 16-bit
    const char *SA; int64_t sa_rs, sa_cs;      // [M][blocks]; codes
    const char *Q; int64_t q_rs, q_es;         // [E][N][row_bytes]
    const char *S; int64_t s_rs, s_cs, s_es;   // [E][N][blocks]
    char *C; int64_t c_rs, c_cs;
    int out_kind, act;
    int vec4;                                  // rows of C are contiguous
    int M, N, K;                               // K of codes: 2 * row_bytes
    int row_bytes, blocks;                     // ceil(K / 2), ceil(K / 32)
    const char *offsets; int64_t o_s; int E;   // offsets null: one group of all M rows
    int tiles_n, ktiles;
    int group_m;
    int units;                                 // workgroups of the grid
    int splits, kt_per_split;                  // K in pieces (one matrix only)
    int s_words;                               // mx4_half.hip: scales at aligned words, K a multiple of 128
    int via;                                   // mx4_half.hip: any K and alignment, through registers
    int a_rows;                                // mx4_few.hip: rows of a 16-bit A that a workgroup stages in LDS, or 0
    float *ws; int *counters;
};

// Tiles of the products.
enum Mx4Tile : int { MX4_T256 = 0, MX4_T128 = 1, MX4_T64 = 2, NUM_MX4_TILES = 3 };
constexpr int mx4_tile_m(int t) { return t == MX4_T256 ? 256 : t == MX4_T128 ? 128 : 64; }
constexpr int mx4_tile_n(int t) { return t == MX4_T256 ? 256 : t == MX4_T128 ? 128 : 64; }

// Loads of the products.
//  MX4_DIRECT: codes from memory to LDS: rows begin at multiples of 4 bytes; scale bytes
//              adjacent, 8 of a row at least.
//  MX4_BYTES : codes through registers, 16 bytes at any alignment; scales as above.
//  MX4_ANY   : the same with scales byte by byte.
enum Mx4Load : int { MX4_DIRECT = 0, MX4_BYTES = 1, MX4_ANY = 2 };
hipError_t launch_mx4_gemm(int tile, int load, const Mx4GemmArgs &a, int64_t units, hipStream_t stream);

// The same by mx4_ring.hip, tiles of 256 and 128: K a multiple of 512, rows and scale rows
// at multiples of 16 bytes.
hipError_t launch_mx4_ring(int tile, const Mx4GemmArgs &a, int64_t units, hipStream_t stream);

// 16-bit A (mx4_half.hip): K 32 at least; without `via` a multiple of 8, A's rows at
// multiples of 16 bytes, W's at multiples of 4 and apart.
enum Mx4HalfTile : int { MX4_T128x256 = 0, MX4_T64x128 = 1 };
hipError_t launch_mx4_half(int in_kind, int tile, const Mx4GemmArgs &a, int64_t units, hipStream_t stream);

// Few rows (mx4_few.hip): any layout.  kind: MX4_CODES, or the type of a 16-bit A; tm, nf:
// tm 1 to 3 (codes: 1, 2, 4) for mx4_few_rows(tm) rows, x 16 nf columns, of a workgroup; pieces of K of kt_per_split units of 512.
constexpr int MX4_CODES = 3;               // beside IN_F16 and IN_BF16
constexpr int mx4_few_rows(int tm) { return tm == 3 ? 36 : 16 * tm; }   // of a workgroup (36: two steps of them fill LDS)
constexpr int mx4_few_sums(int tm, int nf) { return 256 * tm * nf; }   // of a workgroup: FP32, of whole 16 x 16 blocks
hipError_t launch_mx4_few(int kind, int tm, int nf, const Mx4GemmArgs &a, int64_t units, hipStream_t stream);

}  // namespace dg
