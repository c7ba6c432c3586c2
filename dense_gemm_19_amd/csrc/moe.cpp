// moe.cpp -- the entry points of the mixture-of-experts and 4-bit operators:
// validation, kernel selection and launch (see include/dg.h for the contracts).
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "entry.hpp"
#include "moe.hpp"

namespace dg {
namespace {

// ---------------------------------------------------------------- routing

dg_status sort_entry(const dg_view *ids, int32_t E, const dg_view *offsets, const dg_view *order, const dg_view *pos,
                     hipStream_t stream, Report *r) {
    Mat i, off, ord, p;
    if (E < 1 || E > MOE_MAX_EXPERTS) return DG_ERR_INVALID_ARG;
    DG_TRY(canonicalize(ids, &i));
    if (i.dtype != DG_I32 && i.dtype != DG_I64) return DG_ERR_DTYPE;
    const int64_t n = i.rows * i.cols;
    if (n > INT32_MAX) return DG_ERR_OVERFLOW;
    DG_TRY(index_vector(offsets, (int64_t)E + 1, &off));
    DG_TRY(index_vector(order, n, &ord));
    DG_TRY(canonicalize(pos, &p));
    if (p.dtype != DG_I32) return DG_ERR_DTYPE;
    if (p.rows != i.rows || p.cols != i.cols) return DG_ERR_SHAPE_MISMATCH;
    if (!contiguous(off) || !contiguous(ord) || !contiguous(p)) return DG_ERR_UNSUPPORTED_VIEW;
    if (spans_overlap(off, i) || spans_overlap(ord, i) || spans_overlap(p, i) || spans_overlap(off, ord) ||
        spans_overlap(off, p) || spans_overlap(ord, p))
        return DG_ERR_ALIAS;
    Device d;
    DG_TRY(ready({&i, &off, &ord, &p}, &d, r));
    SortArgs a;
    a.ids = i.ptr; a.i_rs = i.rs; a.i_cs = i.cs;
    a.wide = i.dtype == DG_I64;
    a.n = (int)n;
    a.k = i.rows <= 1 || (i.cols > 0 && i.rs == i.cols * i.cs) ? 0 : (int)i.cols;   // 0: one run of n ids
    if (a.k == 0 && i.cols == 1 && i.rows > 1) a.i_cs = i.rs;
    a.E = E;
    a.bits = 0;
    while ((1 << a.bits) < E) ++a.bits;
    a.offsets = reinterpret_cast<int *>(out_ptr(off));
    a.order = reinterpret_cast<int *>(out_ptr(ord));
    a.pos = reinterpret_cast<int *>(out_ptr(p));
    a.blocks = (int)cdiv(n, SORT_BLOCK);
    a.table = nullptr;
    WsLease lease;
    const int64_t table_blocks = cdiv(n, sort_table_block(n));
    if (n >= SORT_TABLE_MIN && table_blocks * E <= SORT_TABLE_MAX && !capturing(stream, r)) {
        a.blocks = (int)table_blocks;
        if (r) return r->say("two launches of %d workgroups, %d ids each", a.blocks, sort_table_block(n));
        if (lease_workspace(stream, (size_t)a.blocks * E * sizeof(int), 0, &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.table = reinterpret_cast<int *>(lease.ws);
    }
    if (r && n <= SORT_ONE_MAX) return r->say("one workgroup, up to %d ids a thread", sort_steps(a.n));
    if (r) return r->say("three launches of %d workgroups", a.blocks);
    return done(launch_moe_sort(a, stream), stream);
}

dg_status gather_entry(const dg_view *X, const dg_view *order, int32_t k, const dg_view *Xs, hipStream_t stream) {
    Mat x, o, y;
    if (k < 1) return DG_ERR_INVALID_ARG;
    DG_TRY(canonicalize(X, &x));
    DG_TRY(canonicalize(Xs, &y));
    if (!(is_float(x.dtype) || x.dtype == DG_F8E4M3 || x.dtype == DG_U8) || y.dtype != x.dtype) return DG_ERR_DTYPE;
    if (y.cols != x.cols) return DG_ERR_SHAPE_MISMATCH;
    DG_TRY(index_vector(order, y.rows, &o));
    if (x.rows > INT32_MAX || x.cols > MOE_MAX_EXTENT || y.rows > INT32_MAX) return DG_ERR_OVERFLOW;
    if (self_overlaps(y)) return DG_ERR_STRIDE;
    if (spans_overlap(y, x) || spans_overlap(y, o)) return DG_ERR_ALIAS;
    if (y.empty()) return DG_SUCCESS;
    Device d;
    DG_TRY(ready({&x, &o, &y}, &d, nullptr));
    GatherArgs a;
    a.X = x.ptr; a.x_rs = x.rs; a.x_cs = x.cs;
    a.Y = out_ptr(y); a.y_rs = y.rs; a.y_cs = y.cs;
    a.order = o.ptr; a.o_s = o.cs;
    a.T = (int)x.rows; a.k = k; a.n = (int)y.rows; a.H = (int)y.cols; a.esize = y.esize;
    a.vec = x.cols_contig() && y.cols_contig();
    // An output above 160 MB goes past the caches.  Alone a gather gains by that from
    // 96 MB on (16384 rows of 4096 BF16, 128 MB: 39.6 us instead of 45.0), but the
    // product that reads its output next gives it back while the last-level cache
    // still holds a good part of it.  Gather and product, 8 experts, 4096 -> 1024 and
    // -> 4096, past the caches and through them: 101 MB 153 and 449 us, 150 and 437;
    // 128 MB 239 and 565, 237 and 560; 187 MB 270 and 744, 283 and 747; 256 MB 394
    // and 1033, 405 and 1043.
    a.stream = y.rows * y.cols * y.esize > (int64_t)160 << 20;
    return done(launch_moe_gather(a, stream), stream);
}

// combine (grad false: Y is written) and its gradient (Y is dY, read)
dg_status combine_entry(const dg_view *Ys, const dg_view *pos, const dg_view *w, const dg_view *Y, const dg_view *dYs,
                        const dg_view *dw, bool grad, hipStream_t stream) {
    Mat s, p, wt, y, ds, dv;
    DG_TRY(canonicalize(Ys, &s));
    DG_TRY(canonicalize(pos, &p));
    DG_TRY(canonicalize(Y, &y));
    if (w) DG_TRY(canonicalize(w, &wt));
    if (grad) {
        DG_TRY(canonicalize(dYs, &ds));
        if (dw && !w) return DG_ERR_NULL;
        if (dw) DG_TRY(canonicalize(dw, &dv));
    }
    if (!is_float(s.dtype) || y.dtype != s.dtype || p.dtype != DG_I32) return DG_ERR_DTYPE;
    if (w && !is_float(wt.dtype)) return DG_ERR_DTYPE;
    if (grad && (ds.dtype != s.dtype || (dw && dv.dtype != wt.dtype))) return DG_ERR_DTYPE;
    if (y.cols != s.cols || p.rows != y.rows) return DG_ERR_SHAPE_MISMATCH;
    if (w && (wt.rows != p.rows || wt.cols != p.cols)) return DG_ERR_SHAPE_MISMATCH;
    if (grad && (ds.rows != s.rows || ds.cols != s.cols)) return DG_ERR_SHAPE_MISMATCH;
    if (dw && (dv.rows != p.rows || dv.cols != p.cols)) return DG_ERR_SHAPE_MISMATCH;
    if (s.rows > INT32_MAX || y.rows > INT32_MAX || y.cols > MOE_MAX_EXTENT || p.cols > MOE_MAX_EXTENT) return DG_ERR_OVERFLOW;
    // what is written overlaps neither itself nor any other view
    if (!grad) {
        if (self_overlaps(y)) return DG_ERR_STRIDE;
        if (spans_overlap(y, s) || spans_overlap(y, p) || spans_overlap(y, wt)) return DG_ERR_ALIAS;
        if (y.empty()) return DG_SUCCESS;
    } else {
        if (self_overlaps(ds) || self_overlaps(dv)) return DG_ERR_STRIDE;
        for (const Mat *o : {&ds, &dv})
            for (const Mat *m : {&s, &p, &wt, &y})
                if (spans_overlap(*o, *m)) return DG_ERR_ALIAS;
        if (spans_overlap(ds, dv)) return DG_ERR_ALIAS;
        if (ds.empty() && dv.empty()) return DG_SUCCESS;
    }
    Device d;
    DG_TRY(ready({&s, &p, &wt, &y, &ds, &dv}, &d, nullptr));
    CombineArgs a = {};
    a.Ys = s.ptr; a.s_rs = s.rs; a.s_cs = s.cs;
    a.Y = out_ptr(y); a.y_rs = y.rs; a.y_cs = y.cs;
    a.pos = p.ptr; a.p_rs = p.rs; a.p_cs = p.cs;
    if (w) { a.w = wt.ptr; a.w_rs = wt.rs; a.w_cs = wt.cs; a.w_kind = wt.dtype; }
    a.T = (int)y.rows; a.k = (int)p.cols; a.R = (int)s.rows; a.H = (int)s.cols;
    a.vec = s.cols_contig() && y.cols_contig();
    if (!grad) return done(launch_moe_combine(s.dtype, a, stream), stream);
    a.dYs = out_ptr(ds); a.d_rs = ds.rs; a.d_cs = ds.cs;
    if (dw) { a.dw = out_ptr(dv); a.g_rs = dv.rs; a.g_cs = dv.cs; }
    a.vec = a.vec && ds.cols_contig();
    a.p_run = p.cols_contig() && (p.rows <= 1 || p.rs == p.cols * p.esize);
    return done(launch_moe_combine_grad(s.dtype, a, stream), stream);
}

// ---------------------------------------------------------------- expert products

struct OpLayout {
    int mode = KMAJ;
    bool dtl = false, vec = false;   // what the loaders ask of the operand
};

// An operand whose rows (extent `rows`, `rs` bytes apart) are summed along k.
// aligned: every further base offset (experts) is a multiple of 16 bytes.
OpLayout layout(const char *ptr, int64_t rows, int64_t rs, int64_t k, int64_t ks, bool aligned) {
    OpLayout o;
    const bool base = reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && aligned;
    // lane offsets within a 256-row, 64-element tile stay below 2^31
    const bool near = 256 * rs + 64 * ks < ((int64_t)1 << 31);
    if (ks == 2 || k <= 1) {
        o.mode = KMAJ;
        o.vec = k >= 8;
        o.dtl = base && near && ks == 2 && rs % 16 == 0 && k % 8 == 0;
    } else if (rs == 2 || rows <= 1) {
        o.mode = MNMAJ;
        o.vec = rows >= 8;
        o.dtl = base && near && rs == 2 && ks % 16 == 0 && rows % 8 == 0;
    }
    return o;
}

// vec4 whatever the alignment: 4 element stores each took 74 us where these take
// 44 (30 experts of 880 x 1285 BF16).
Epilogue plain_epilogue(const Mat &c, int act) {
    Epilogue e = {};
    e.C = out_ptr(c);
    e.c_rs = c.rs;
    e.c_cs = c.cs;
    e.out_kind = c.dtype;
    e.alpha = 1.0f;
    e.beta = 0.0f;
    e.act = act;
    e.vec4 = c.cs == c.esize;
    return e;
}

hipError_t launch_product(int in_kind, int load, int tile, int b_mode, bool wgrad, const MoeArgs &a, int64_t units,
                          hipStream_t s) {
    return in_kind == IN_F16 ? launch_moe_gemm_f16(load, tile, b_mode, wgrad, a, units, s)
                             : launch_moe_gemm_bf16(load, tile, b_mode, wgrad, a, units, s);
}

int tile_rows(int load, int tile) { return tile == MOE_T192 ? 192 : load == MOE_DTL && tile == T64x128 ? 32 : mfma_tile_bm(tile); }
int tile_cols(int tile) { return tile == MOE_T192 ? 256 : mfma_tile_bn(tile); }

// The pieces of K that each tile is cut into where the tiles leave most of the
// device idle: `tiles` of them are expected, with `ktiles` K tiles; a piece keeps at least four.  Few tiles wait for one load after
// another: 12 rows of 4 experts, 3520 -> 192, took 24.0 us whole, 11.5 us cut.
// Adding the pieces takes about 3 us, what 8 K tiles of the 32 x 128 tile do (12 of
// them, 4 experts of 6 rows: 8.1 us whole, 9.6 cut).
// A captured call runs whole: the pieces' workspace may have to be allocated.
int pieces_of(int load, int tile, int64_t tiles, int64_t ktiles, const Device &d, hipStream_t stream, const Report *r) {
    if (tile == T256x256 || tile == MOE_T192 || (load != MOE_DTL && tile == T128x128) || ktiles < (tile == T64x128 ? 16 : 8)) return 1;
    const int64_t s = std::min(d.cus / std::max<int64_t>(tiles, 1), ktiles / 4);
    if (s < 2) return 1;
    return capturing(stream, r) ? 1 : (int)s;
}

// Launch `units` tiles in a.p.splits pieces each, on the stream's workspace.
dg_status launch_pieces(int in_kind, int load, int tile, int b_mode, bool wgrad, MoeArgs &a, int64_t units, int64_t bm, int64_t bn,
                        hipStream_t stream, Report *r) {
    if (units > INT32_MAX || !fits_a_launch(units * a.p.splits, tile == T256x256 || tile == MOE_T192 ? 512 : 256)) return DG_ERR_OVERFLOW;
    if (r)
        return r->say("%s loads, %dx%d tiles, K in %d pieces, %lld workgroups", load == MOE_DTL ? "direct" : load == MOE_VEC ? "vector" : "element",
                      (int)bm, (int)bn, a.p.splits, (long long)(units * a.p.splits));
    WsLease lease;
    if (a.p.splits > 1) {
        if (lease_workspace(stream, (size_t)units * a.p.splits * bm * bn * sizeof(float), (size_t)units, &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.p.ws = lease.ws;
        a.p.counters = lease.counters;
    }
    a.units = (int)(units * a.p.splits);
    return done(launch_product(in_kind, load, tile, b_mode, wgrad, a, units * a.p.splits, stream), stream);
}

dg_status moe_gemm_entry(const dg_view *A, const dg_view *offsets, const dg_view *W, const dg_view *C, int act,
                         hipStream_t stream, Report *r) {
    Mat x, off, c;
    Stack w;
    DG_TRY(canonicalize(A, &x));
    DG_TRY(canonicalize_stack(W, &w));
    DG_TRY(canonicalize(C, &c));
    if (!is_half(x.dtype) || w.one.dtype != x.dtype || !is_float(c.dtype)) return DG_ERR_DTYPE;
    if (w.E < 1 || w.one.rows != x.cols || c.rows != x.rows || c.cols != w.one.cols) return DG_ERR_SHAPE_MISMATCH;
    DG_TRY(index_vector(offsets, w.E + 1, &off));
    const int64_t n = x.rows, K = x.cols, N = c.cols;
    if (n > MOE_MAX_ROWS || K > MOE_MAX_EXTENT || N > MOE_MAX_EXTENT || w.E > MOE_MAX_SCANNED) return DG_ERR_OVERFLOW;
    if (act != DG_ACT_NONE && act != DG_ACT_RELU && act != DG_ACT_GELU_TANH) return DG_ERR_INVALID_ARG;
    if (self_overlaps(c)) return DG_ERR_STRIDE;
    if (spans_overlap(c, x) || spans_overlap(c, w.span) || spans_overlap(c, off)) return DG_ERR_ALIAS;
    if (c.empty()) return nothing(r);
    Device d;
    DG_TRY(ready({&x, &off, &w.span, &c}, &d, r));

    const OpLayout la = layout(x.ptr, n, x.rs, K, x.cs, true);
    const OpLayout lb = layout(w.one.ptr, N, w.one.cs, K, w.one.rs, w.es % 16 == 0 || w.E == 1);
    int load = MOE_ELEM;
    if (la.mode == KMAJ && la.vec && lb.vec) load = la.dtl && lb.dtl ? MOE_DTL : MOE_VEC;
    // The tile: by the mean row count of the experts that can have rows.  Direct, 32
    // x 128 up to a mean of 48 (8 experts, 4096 -> 14336: 16 rows each 178 us, 128 x
    // 128 178; 64 rows 243 and 188; between, whole 32-row tiles are as quick at 32
    // rows, 184 and 176, and behind at 40, 228 and 178: a bound of 24 would serve
    // even counts better).  Of the larger ones the quickest by what a K tile takes
    // in each (us, measured on long K; two 128 x 128 workgroups share a CU) and the
    // rounds that the expected tiles make: 64 experts of 234 rows, 4096 -> 512 FP16,
    // take 127 us as 256 x 256 tiles, 120.5 as 192 x 256; 13 experts of 366 rows,
    // 1088 -> 192, 25 us as 256 x 256, 16.6 as pieces of 128 x 128.
    // Expected tiles: an expert's last one is half full on average.
    const int64_t used = std::min(w.E, n), mean = n / std::max<int64_t>(used, 1), ktiles = cdiv(K, 64);
    auto expected = [&](int t) {
        const int64_t rows = tile_rows(load, t);
        return std::max(used, used / 2 + cdiv(n, rows)) * cdiv(N, tile_cols(t));
    };
    int tile = T64x64;
    if (load == MOE_DTL && mean <= 48) {
        tile = T64x128;
    } else if (load == MOE_DTL) {
        double best = 0.0;
        for (int t : {(int)T256x256, MOE_T192, (int)T128x128}) {
            const int64_t tiles = expected(t), S = pieces_of(load, t, tiles, ktiles, d, stream, r);
            const double k_us = t == T256x256 ? 1.78 : t == MOE_T192 ? 1.65 : tiles * S <= d.cus ? 0.8 : 1.3;
            // rounds: between their fraction and the next whole number, the expected
            // count being one of many (8 experts of exactly 2048 rows make one round
            // of 256 x 256 tiles where 1.06 are expected)
            const double r = (double)(tiles * S) / (t == T128x128 ? 2 * d.cus : d.cus);
            const double rounds = r <= 1.0 ? 1.0 : 0.5 * (r + std::ceil(r));
            const double us = k_us * rounds * cdiv(ktiles, S) + (S > 1 ? 3.0 : 0.0);
            if (best == 0.0 || us < best) {
                best = us;
                tile = t;
            }
        }
    } else if (load == MOE_VEC) {
        // 8 experts of 512 rows, 1001 -> 2047: 41 us, 55 as 64 x 64; of 128 rows, whose
        // 128 x 128 tiles leave CUs idle, 18 us, 29 as 128 x 128
        tile = mean <= 64 || expected(T128x128) < d.cus ? T64x64 : T128x128;
    }
    const int bm = tile_rows(load, tile), bn = tile_cols(tile);

    MoeArgs a = {};
    a.p.a = Operand{x.ptr, x.rs, x.cs, 1};
    a.p.b = Operand{w.one.ptr, w.one.cs, w.one.rs, 1};
    a.p.epi = plain_epilogue(c, act);
    a.p.N = (int)N; a.p.K = (int)K;
    a.p.tiles_n = (int)cdiv(N, bn);
    a.p.ktiles = (int)ktiles;
    a.p.splits = pieces_of(load, tile, expected(tile), ktiles, d, stream, r);
    a.p.group_m = tile == T256x256 || tile == MOE_T192 ? 4 : 8;
    a.offsets = off.ptr; a.o_s = off.cs;
    a.E = (int)w.E; a.n = (int)n;
    a.e_bs = w.es;
    // every group with rows (the experts and the rows of none) ends in a partial tile at most
    const int64_t units = ((n + std::min(w.E + 1, n) * (bm - 1)) / bm) * a.p.tiles_n;
    return launch_pieces(x.dtype == DG_F16 ? IN_F16 : IN_BF16, load, tile, lb.mode, false, a, units, bm, bn, stream, r);
}

dg_status moe_wgrad_entry(const dg_view *A, const dg_view *D, const dg_view *offsets, const dg_view *dW,
                          hipStream_t stream, Report *r) {
    Mat x, g, off;
    Stack w;
    DG_TRY(canonicalize(A, &x));
    DG_TRY(canonicalize(D, &g));
    DG_TRY(canonicalize_stack(dW, &w));
    if (!is_half(x.dtype) || g.dtype != x.dtype || !is_float(w.one.dtype)) return DG_ERR_DTYPE;
    if (w.E < 1 || g.rows != x.rows || w.one.rows != x.cols || w.one.cols != g.cols) return DG_ERR_SHAPE_MISMATCH;
    DG_TRY(index_vector(offsets, w.E + 1, &off));
    const int64_t n = x.rows, K = x.cols, N = g.cols;
    if (n > MOE_MAX_EXTENT || K > MOE_MAX_EXTENT || N > MOE_MAX_EXTENT || w.E > INT32_MAX / 2) return DG_ERR_OVERFLOW;
    if (stack_overlaps(w)) return DG_ERR_STRIDE;
    if (spans_overlap(w.span, x) || spans_overlap(w.span, g) || spans_overlap(w.span, off)) return DG_ERR_ALIAS;
    if (w.one.empty()) return nothing(r);
    Device d;
    DG_TRY(ready({&x, &g, &off, &w.span}, &d, r));

    // dW[e] is a product summed over rows: A's columns are its rows
    const OpLayout la = layout(x.ptr, K, x.cs, n, x.rs, true), lb = layout(g.ptr, N, g.cs, n, g.rs, true);
    int load = MOE_ELEM;
    if (x.cs == 2 && g.cs == 2 && K >= 8 && N >= 8)
        load = la.mode == MNMAJ && lb.mode == MNMAJ && la.dtl && lb.dtl ? MOE_DTL : MOE_VEC;
    // The largest tile that gives every CU one: 8 experts of 1024 rows, 2048 x 2048,
    // 82 us as 256 x 256 tiles, 103 as 128 x 128; 1024 x 1024 34 and 29.  Loads at any
    // alignment: 1001 x 1023 55 us as 64 x 64, 39 as 128 x 128; 513 x 511 of 256 rows
    // 10.4 and 13.9.
    int tile = load == MOE_ELEM ? T64x64 : T128x128;
    if (load == MOE_DTL && w.E * cdiv(K, 256) * cdiv(N, 256) >= d.cus) tile = T256x256;
    if (load == MOE_VEC && w.E * cdiv(K, 128) * cdiv(N, 128) < d.cus) tile = T64x64;
    const int bm = mfma_tile_bm(tile), bn = mfma_tile_bn(tile);

    MoeArgs a = {};
    a.p.a = Operand{x.ptr, x.cs, x.rs, 1};
    a.p.b = Operand{g.ptr, g.cs, g.rs, 1};
    a.p.epi = plain_epilogue(w.one, DG_ACT_NONE);
    a.p.M = (int)K; a.p.N = (int)N;
    a.p.tiles_m = (int)cdiv(K, bm); a.p.tiles_n = (int)cdiv(N, bn);
    a.p.group_m = tile == T256x256 ? 4 : 8;
    a.offsets = off.ptr; a.o_s = off.cs;
    a.E = (int)w.E; a.n = (int)n;
    a.e_cs = w.es;
    const int64_t tiles = (int64_t)a.p.tiles_m * a.p.tiles_n;
    if (tiles > INT32_MAX || tiles * w.E > INT32_MAX) return DG_ERR_OVERFLOW;
    a.p.splits = pieces_of(load, tile, tiles * w.E, cdiv(n / w.E, 64), d, stream, r);
    return launch_pieces(x.dtype == DG_F16 ? IN_F16 : IN_BF16, load, tile, lb.mode, true, a, tiles * w.E, bm, bn, stream, r);
}

// ---------------------------------------------------------------- 4-bit weights

dg_status w4_entry(const dg_view *A, const dg_view *offsets, const dg_view *Q, const dg_view *S, const dg_view *Z,
                   const dg_view *C, int32_t group, int act, bool experts, hipStream_t stream, Report *r) {
    Mat x, c, off;
    Stack q, s, z;
    DG_TRY(canonicalize(A, &x));
    DG_TRY(canonicalize(C, &c));
    if (experts) {
        DG_TRY(canonicalize_stack(Q, &q));
        DG_TRY(canonicalize_stack(S, &s));
        if (Z) DG_TRY(canonicalize_stack(Z, &z));
    } else {
        DG_TRY(canonicalize(Q, &q.one));
        DG_TRY(canonicalize(S, &s.one));
        if (Z) DG_TRY(canonicalize(Z, &z.one));
        for (Stack *t : {&q, &s, &z}) { t->E = 1; t->span = t->one; }
    }
    if (!is_half(x.dtype) || !is_float(c.dtype) || q.one.dtype != DG_U8 || !is_float(s.one.dtype)) return DG_ERR_DTYPE;
    if (Z && z.one.dtype != DG_U8) return DG_ERR_DTYPE;
    if (group < 32 || group % 32 != 0) return DG_ERR_INVALID_ARG;
    if (act != DG_ACT_NONE && act != DG_ACT_RELU && act != DG_ACT_GELU_TANH) return DG_ERR_INVALID_ARG;
    const int64_t M = x.rows, K = x.cols, N = c.cols, groups = cdiv(K, group);
    if (c.rows != M || q.one.rows != N || q.one.cols != cdiv(K, 2)) return DG_ERR_SHAPE_MISMATCH;
    if (q.E < 1 || s.E != q.E || s.one.rows != N || s.one.cols != groups) return DG_ERR_SHAPE_MISMATCH;
    if (Z && (z.E != q.E || z.one.rows != N || z.one.cols != groups)) return DG_ERR_SHAPE_MISMATCH;
    if (experts) DG_TRY(index_vector(offsets, q.E + 1, &off));
    if (M > (experts ? MOE_MAX_ROWS : MOE_MAX_EXTENT) || K > (1 << 20) || N > MOE_MAX_EXTENT || q.E > MOE_MAX_SCANNED) return DG_ERR_OVERFLOW;
    if (!x.cols_contig() || !q.one.cols_contig()) return DG_ERR_UNSUPPORTED_VIEW;
    // lane offsets within a workgroup's rows and columns are 32-bit
    const int64_t lim = W4_MAX_PITCH;
    if (x.rs >= lim || q.one.rs >= lim || s.one.rs >= lim || z.one.rs >= lim) return DG_ERR_OVERFLOW;
    if (self_overlaps(c)) return DG_ERR_STRIDE;
    for (const Mat *m : {&x, &q.span, &s.span, &z.span, &off})
        if (spans_overlap(c, *m)) return DG_ERR_ALIAS;
    if (c.empty()) return nothing(r);
    return w4_run(x, off, q, s, Z ? &z : nullptr, c, group, act, experts, false, stream, r);
}

}  // namespace

dg_status w4_run(const Mat &x, const Mat &off, const Stack &q, const Stack &s, const Stack *zeros, const Mat &c, int group, int act,
                 bool experts, bool mx, hipStream_t stream, Report *r) {
    const int64_t M = x.rows, K = x.cols, N = c.cols, groups = cdiv(K, group);
    const bool Z = zeros != nullptr;
    const Stack z = Z ? *zeros : Stack();
    Device d;
    DG_TRY(ready({&x, &off, &q.span, &s.span, &z.span, &c}, &d, r));

    W4Args a = {};
    a.A = x.ptr; a.a_rs = x.rs;
    a.Q = q.one.ptr; a.q_rs = q.one.rs; a.q_es = q.es;
    a.S = s.one.ptr; a.s_rs = s.one.rs; a.s_cs = s.one.cs; a.s_es = s.es;
    if (Z) { a.Z = z.one.ptr; a.z_rs = z.one.rs; a.z_cs = z.one.cs; a.z_es = z.es; }
    a.s_kind = s.one.dtype;
    a.C = out_ptr(c); a.c_rs = c.rs; a.c_cs = c.cs; a.out_kind = c.dtype; a.act = act;
    a.M = (int)M; a.N = (int)N; a.K = (int)K; a.G = group;
    a.groups = (int)groups;
    a.g_mul = group == 32 ? 0u : (uint32_t)((((uint64_t)1 << 32) + group / 32 - 1) / (group / 32));
    if (experts) { a.offsets = off.ptr; a.o_s = off.cs; }
    a.E = (int)q.E;
    auto pieces = [](const Mat &m, int64_t es) {   // rows of whole, aligned 16-byte pieces
        return reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && es % 16 == 0 && (m.rows <= 1 || m.rs % 16 == 0) &&
               m.cols * m.esize % 16 == 0;
    };
    // the words that hold any of them lie between the first and the last one
    auto words = [](const Stack &t) {
        return t.one.cs == t.one.esize && t.span.lo % 4 == 0 && t.span.hi % 4 == 0;
    };
    const bool usual = K > 0 && K % 32 == 0 && pieces(x, 0) && pieces(q.one, q.E > 1 ? q.es : 0) &&
                       words(s) && (!Z || words(z));

    // Rows of a tile: as few tiles as the largest allows, evenly filled (one
    // matrix), or by the mean count of the experts that can have rows (16 experts of
    // 0.5 to 1.5 times the mean, 4096 -> 7168, G 128: mean 8 83 us as 16 rows x 32
    // columns, 102 as 32 x 64; 12 126 and 104; 16 107 as 32 x 64, 116 as 48 x 64; 28
    // 145 and 123).
    int64_t tiles_m;
    int tm, rows;
    if (experts) {
        const int64_t mean = M / std::min(q.E, M);
        tm = mean <= 10 ? 1 : mean <= 24 ? 2 : 3;
        tiles_m = (M + std::min(q.E + 1, M) * (16 * tm - 1)) / (16 * tm);
        rows = 16 * tm;
    } else {
        tm = (int)cdiv(cdiv(M, cdiv(M, 16 * W4_MAX_TM)), 16);
        tiles_m = cdiv(M, 16 * tm);
        rows = (int)std::min<int64_t>(M, 16 * tm);
    }
    a.slabs = (int)cdiv(N, w4_cols(tm));
    // K in pieces where one matrix has too few slabs to fill the device and K is
    // above 4096: each piece keeps two chunks.  (The bound is a high one: cut from 4
    // chunks on, 1 x 1024 x 4096 takes 6.9 us instead of 7.9, 33 x 2048 x 4096 9.6
    // instead of 16.3.)  Experts' K is never cut: their tiles vary with the rows.  A
    // captured call runs whole: the pieces' workspace may have to be allocated.
    const int chunk = w4_chunk(tm);
    const int64_t chunks = cdiv(K, chunk), units = tiles_m * a.slabs;
    int64_t splits = 1;
    if (!experts && chunks * chunk > 4096 && 2 * units <= d.cus && !capturing(stream, r))
        splits = std::min<int64_t>(d.cus / units, chunks / 2);
    a.chunks = (int)std::max<int64_t>(cdiv(chunks, splits), 1);
    a.splits = (int)std::max<int64_t>(cdiv(chunks, a.chunks), 1);
    // LDS of the usual layout (w4_whole): scales and zero points in words, the pitch
    // an odd number of them, and rings of 2 to 4 chunks of A and the codes; experts'
    // rings hold so many of the mean count of rows, and one of a full tile.  Half of
    // a CU's LDS where 2 chunks of few rows fit and the grid has two workgroups for
    // a CU, else all.
    const int half = 80 * 1024 - 128, all = 160 * 1024 - 128;
    const int unit = 8 * 2048, a_buf = rows * chunk * 2;
    if (usual) {
        const int64_t need = std::min<int64_t>(groups, (int64_t)a.chunks * chunk / group + 5);   // from a multiple of 4 on
        auto pitch = [](int64_t bytes) { return (int)std::max<int64_t>((cdiv(bytes, 4) | 1) * 4, 12); };   // (the reciprocal of one word is 2^32)
        auto region = [&](int p) { return (w4_cols(tm) * p + 255) & ~255; };
        a.seg_groups = (int)need;
        a.s_pitch = pitch(need * s.one.esize + 3);
        a.z_pitch = Z ? pitch(need + 3) : 0;
        const int sz = region(a.s_pitch) + (Z ? region(a.z_pitch) : 0);
        const int64_t mean = experts ? std::min<int64_t>(M / std::min(q.E, M) + 1, rows) : rows;
        const int a_mean = (int)(mean * chunk * 2);
        auto fits = [&](int depth, int bufs, int cap) {
            a.depth = depth;
            a.a_lds = (cap - depth * unit - sz) & ~1023;   // (all there is: experts differ in rows)
            a.lds_bytes = depth * unit + a.a_lds + sz;
            return a.a_lds >= std::max(a_buf, bufs * a_mean);
        };
        const int most = std::min(4, std::max(a.chunks, 2));
        const bool pairs = tm == 1 && units * a.splits > d.cus;
        for (int n = most; n > 1 && pairs && !a.whole; --n) a.whole = fits(n, n, half);
        for (int n = most; n > 1 && !a.whole; --n) a.whole = fits(n, n, all);
        auto recip = [](int d) { return (uint32_t)((((uint64_t)1 << 32) + d - 1) / d); };
        a.s_mul = recip(a.s_pitch / 4);
        a.z_mul = Z ? recip(a.z_pitch / 4) : 0;
    }
    // Any other layout (w4_stream): a unit of codes per wave, scales for as many
    // chunks as fit, and all of A where that fits, else one chunk.
    if (!a.whole) {
        auto scales = [&](int64_t seg) {
            a.seg = (int)seg;
            a.seg_groups = (int)std::min<int64_t>(groups, seg * chunk / group + 2);
            a.s_pitch = (int)(cdiv(a.seg_groups * s.one.esize, 16) * 16 + 16);
            a.z_pitch = Z ? (int)(cdiv(a.seg_groups, 16) * 16 + 16) : 0;
            return w4_cols(tm) * (a.s_pitch + a.z_pitch);
        };
        int64_t seg = a.chunks;
        const int cap = tm == 1 && unit + scales(seg) + a_buf <= half ? half : all;
        while (seg > 1 && unit + scales(seg) + a_buf > cap) seg = cdiv(seg, 2);
        const int sz = scales(seg), left = (cap - unit - sz) / a_buf;
        a.a_lds = std::max(1, std::min(left, a.chunks)) * a_buf;
        // (the kernel's end adds the waves' sums in the same LDS: 8 KB each of 16 tm rows x 16 columns)
        a.lds_bytes = std::max(unit + sz + a.a_lds, tm * 8 * 1024);
    }
    if (a.lds_bytes > all) return DG_ERR_OVERFLOW;   // (no size gets here: one chunk's scales are at most 18 KB)
    if (!fits_a_launch(units * a.splits, 512)) return DG_ERR_OVERFLOW;
    if (r)
        return r->say("%s, %dx%d tiles, K in %d pieces, %lld workgroups of %d LDS bytes", a.whole ? "aligned words" : "any layout", 16 * tm,
                      w4_cols(tm), a.splits, (long long)(units * a.splits), a.lds_bytes);
    a.units = (int)(units * a.splits);
    WsLease lease;
    if (a.splits > 1) {
        if (lease_workspace(stream, (size_t)units * a.splits * 16 * tm * w4_cols(tm) * sizeof(float), (size_t)units, &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.ws = lease.ws;
        a.counters = lease.counters;
    }
    const int in_kind = x.dtype == DG_F16 ? IN_F16 : IN_BF16;
    return done(mx ? launch_w4_mx(in_kind, tm, a, units * a.splits, stream) : launch_w4(in_kind, tm, a, units * a.splits, stream), stream);
}

}  // namespace dg

extern "C" {

dg_status dg_moe_sort(const dg_view *ids, int32_t E, const dg_view *offsets, const dg_view *order, const dg_view *pos,
                      hipStream_t stream) {
    return dg::sort_entry(ids, E, offsets, order, pos, stream, nullptr);
}

dg_status dg_moe_gather(const dg_view *X, const dg_view *order, int32_t k, const dg_view *Xs, hipStream_t stream) {
    return dg::gather_entry(X, order, k, Xs, stream);
}

dg_status dg_moe_combine(const dg_view *Ys, const dg_view *pos, const dg_view *w, const dg_view *Y, hipStream_t stream) {
    return dg::combine_entry(Ys, pos, w, Y, nullptr, nullptr, false, stream);
}

dg_status dg_moe_combine_grad(const dg_view *dY, const dg_view *Ys, const dg_view *pos, const dg_view *w,
                              const dg_view *dYs, const dg_view *dw, hipStream_t stream) {
    return dg::combine_entry(Ys, pos, w, dY, dYs, dw, true, stream);
}

dg_status dg_moe_gemm(const dg_view *A, const dg_view *offsets, const dg_view *W, const dg_view *C, dg_act act,
                      hipStream_t stream) {
    return dg::moe_gemm_entry(A, offsets, W, C, (int)act, stream, nullptr);
}

dg_status dg_moe_gemm_wgrad(const dg_view *A, const dg_view *D, const dg_view *offsets, const dg_view *dW,
                            hipStream_t stream) {
    return dg::moe_wgrad_entry(A, D, offsets, dW, stream, nullptr);
}

dg_status dg_gemm_w4(const dg_view *A, const dg_view *Q, const dg_view *S, const dg_view *Z, const dg_view *C,
                     int32_t group, dg_act act, hipStream_t stream) {
    return dg::w4_entry(A, nullptr, Q, S, Z, C, group, (int)act, false, stream, nullptr);
}

dg_status dg_moe_gemm_w4(const dg_view *A, const dg_view *offsets, const dg_view *Q, const dg_view *S,
                         const dg_view *Z, const dg_view *C, int32_t group, dg_act act, hipStream_t stream) {
    return dg::w4_entry(A, offsets, Q, S, Z, C, group, (int)act, true, stream, nullptr);
}

dg_status dg_moe_sort_plan(const dg_view *ids, int32_t E, const dg_view *offsets, const dg_view *order, const dg_view *pos,
                           char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::sort_entry(ids, E, offsets, order, pos, nullptr, &r);
}

dg_status dg_moe_gemm_plan(const dg_view *A, const dg_view *offsets, const dg_view *W, const dg_view *C, char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::moe_gemm_entry(A, offsets, W, C, DG_ACT_NONE, nullptr, &r);
}

dg_status dg_moe_gemm_wgrad_plan(const dg_view *A, const dg_view *D, const dg_view *offsets, const dg_view *dW, char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::moe_wgrad_entry(A, D, offsets, dW, nullptr, &r);
}

dg_status dg_gemm_w4_plan(const dg_view *A, const dg_view *Q, const dg_view *S, const dg_view *Z, const dg_view *C,
                          int32_t group, char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::w4_entry(A, nullptr, Q, S, Z, C, group, DG_ACT_NONE, false, nullptr, &r);
}

dg_status dg_moe_gemm_w4_plan(const dg_view *A, const dg_view *offsets, const dg_view *Q, const dg_view *S,
                              const dg_view *Z, const dg_view *C, int32_t group, char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::w4_entry(A, offsets, Q, S, Z, C, group, DG_ACT_NONE, true, nullptr, &r);
}

}  // extern "C"
