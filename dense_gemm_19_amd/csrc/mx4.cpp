// mx4.cpp -- the entry points of the microscaled 4-bit (MXFP4) operators: validation,
// kernel selection and launch (see include/dg.h for the contracts).
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "entry.hpp"
#include "moe.hpp"
#include "mx4.hpp"

namespace dg {
namespace {

// A matrix, or a stack of them where the view is 3-D.
dg_status matrices(const dg_view *v, Stack *s) {
    if (v && v->ndim == 3) return canonicalize_stack(v, s);
    DG_TRY(canonicalize(v, &s->one));
    s->E = 1;
    s->span = s->one;
    return DG_SUCCESS;
}

// Codes and scales of E matrices of M x K.
dg_status codes_of(const Stack &q, const Stack &s, int64_t E, int64_t M, int64_t K) {
    if (q.one.dtype != DG_U8 || s.one.dtype != DG_U8) return DG_ERR_DTYPE;
    if (q.E != E || q.one.rows != M || q.one.cols != cdiv(K, 2)) return DG_ERR_SHAPE_MISMATCH;
    if (s.E != E || s.one.rows != M || s.one.cols != cdiv(K, 32)) return DG_ERR_SHAPE_MISMATCH;
    if (!q.one.cols_contig()) return DG_ERR_UNSUPPORTED_VIEW;
    return DG_SUCCESS;
}

// Workgroups of the kernels whose threads take `run` chunks of 8 elements each.
dg_status runs(const Device &d, int64_t E, int64_t M, int64_t K, int *chunks, uint32_t *mul, int *run, int64_t *units) {
    *chunks = (int)(4 * cdiv(K, 32));
    *mul = (uint32_t)((((uint64_t)1 << 32) + *chunks - 1) / *chunks);
    int64_t total;
    if (__builtin_mul_overflow(E, M, &total) || __builtin_mul_overflow(total, (int64_t)*chunks, &total)) return DG_ERR_OVERFLOW;
    // One chunk a thread where four leave most of the device idle: 1024 x 4096 quantised in
    // 3.9 us beside 5.0, 777 x 2055 read in 3.9 beside 5.5.
    *run = total < 4096 * (int64_t)std::max(d.cus, 1) ? 1 : MX4_RUN;
    *units = cdiv(total, 256 * *run);
    return fits_a_launch(*units, 256) ? DG_SUCCESS : DG_ERR_OVERFLOW;
}

dg_status quant_entry(const dg_view *X, const dg_view *Q, const dg_view *S, int mode, hipStream_t stream) {
    Stack x, q, s;
    DG_TRY(matrices(X, &x));
    DG_TRY(matrices(Q, &q));
    DG_TRY(matrices(S, &s));
    if (mode != DG_MX4_FLOOR && mode != DG_MX4_CEIL) return DG_ERR_INVALID_ARG;
    if (!is_float(x.one.dtype)) return DG_ERR_DTYPE;
    const int64_t M = x.one.rows, K = x.one.cols;
    DG_TRY(codes_of(q, s, x.E, M, K));
    if (M > MOE_MAX_EXTENT || K > MOE_MAX_EXTENT || x.E > INT32_MAX) return DG_ERR_OVERFLOW;
    if (stack_overlaps(q) || stack_overlaps(s)) return DG_ERR_STRIDE;
    if (spans_overlap(q.span, x.span) || spans_overlap(s.span, x.span) || spans_overlap(q.span, s.span)) return DG_ERR_ALIAS;
    if (x.E == 0 || x.one.empty()) return DG_SUCCESS;
    Device d;
    DG_TRY(ready({&x.span, &q.span, &s.span}, &d, nullptr));
    Mx4QuantArgs a = {};
    a.X = x.one.ptr; a.x_es = x.es; a.x_rs = x.one.rs; a.x_cs = x.one.cs;
    a.Q = out_ptr(q.one); a.q_es = q.es; a.q_rs = q.one.rs;
    a.S = out_ptr(s.one); a.s_es = s.es; a.s_rs = s.one.rs; a.s_cs = s.one.cs;
    a.x_kind = x.one.dtype;
    a.M = (int)M; a.K = (int)K; a.E = (int)x.E;
    a.ceil = mode == DG_MX4_CEIL;
    const bool by_columns = !x.one.cols_contig();
    int64_t units;
    if (by_columns) {
        a.vec = x.one.rows_contig();
        a.tiles_m = (int)cdiv(M, MX4_TILE_M);
        a.tiles_k = (int)cdiv(K, MX4_TILE_K);
        const int64_t tiles = (int64_t)a.tiles_m * a.tiles_k;
        if (tiles > INT32_MAX || __builtin_mul_overflow(tiles, x.E, &units) || !fits_a_launch(units, 512)) return DG_ERR_OVERFLOW;
    } else {
        DG_TRY(runs(d, x.E, M, K, &a.chunks, &a.chunk_mul, &a.run, &units));
    }
    return done(launch_mx4_quant(by_columns, a, units, stream), stream);
}

dg_status dequant_entry(const dg_view *Q, const dg_view *S, const dg_view *Y, hipStream_t stream) {
    Stack q, s, y;
    DG_TRY(matrices(Q, &q));
    DG_TRY(matrices(S, &s));
    DG_TRY(matrices(Y, &y));
    if (!is_float(y.one.dtype)) return DG_ERR_DTYPE;
    const int64_t M = y.one.rows, K = y.one.cols;
    DG_TRY(codes_of(q, s, y.E, M, K));
    if (M > MOE_MAX_EXTENT || K > MOE_MAX_EXTENT || y.E > INT32_MAX) return DG_ERR_OVERFLOW;
    if (stack_overlaps(y)) return DG_ERR_STRIDE;
    if (spans_overlap(y.span, q.span) || spans_overlap(y.span, s.span)) return DG_ERR_ALIAS;
    if (y.E == 0 || y.one.empty()) return DG_SUCCESS;
    Device d;
    DG_TRY(ready({&q.span, &s.span, &y.span}, &d, nullptr));
    Mx4DequantArgs a = {};
    a.Q = q.one.ptr; a.q_es = q.es; a.q_rs = q.one.rs;
    a.S = s.one.ptr; a.s_es = s.es; a.s_rs = s.one.rs; a.s_cs = s.one.cs;
    a.Y = out_ptr(y.one); a.y_es = y.es; a.y_rs = y.one.rs; a.y_cs = y.one.cs;
    a.y_kind = y.one.dtype;
    a.M = (int)M; a.K = (int)K; a.E = (int)y.E;
    a.vec = y.one.cols_contig();
    int64_t units;
    DG_TRY(runs(d, y.E, M, K, &a.chunks, &a.chunk_mul, &a.run, &units));
    return done(launch_mx4_dequant(a, units, stream), stream);
}

// A launch of the product of codes with codes.
struct CodesLaunch {
    Mx4GemmArgs a;
    int tile, load;
    bool ring;
};

// The launches of that product, two at most, appended to out[*n].  cut: K may be cut into
// pieces.  part: of the columns of a call.
dg_status codes_plan(const Mat &x, const Mat &sx, const Mat &off, const Stack &q, const Stack &s, const Mat &c, int act, bool experts,
                     const Device &d, bool cut, bool part, CodesLaunch *out, int *n) {
    const int64_t M = x.rows, N = c.cols, bytes = x.cols;
    Mx4GemmArgs a = {};
    a.A = x.ptr; a.a_rs = x.rs;
    a.SA = sx.ptr; a.sa_rs = sx.rs; a.sa_cs = sx.cols > 1 ? sx.cs : 1;
    a.Q = q.one.ptr; a.q_rs = q.one.rs; a.q_es = q.es;
    a.S = s.one.ptr; a.s_rs = s.one.rs; a.s_cs = s.one.cols > 1 ? s.one.cs : 1; a.s_es = s.es;
    a.C = out_ptr(c); a.c_rs = c.rs; a.c_cs = c.cs; a.out_kind = c.dtype; a.act = act;
    a.vec4 = c.cs == c.esize;
    a.M = (int)M; a.N = (int)N;
    a.row_bytes = (int)bytes;
    a.blocks = (int)cdiv(bytes, 16);
    if (experts) { a.offsets = off.ptr; a.o_s = off.cs; }
    a.E = (int)q.E;
    a.ktiles = (int)cdiv(bytes, 128);
    // Loads to LDS: rows at multiples of 4 bytes, none overlapping the next one, since
    // the last chunk of a row may reach into it; lane offsets within a tile are 32-bit.
    auto words = [&](const Mat &m, int64_t es) {
        return reinterpret_cast<uintptr_t>(m.ptr) % 4 == 0 && es % 4 == 0 &&
               (m.rows <= 1 || (m.rs % 4 == 0 && m.rs >= bytes && m.rs < ((int64_t)1 << 23)));
    };
    auto pieces = [&](const Mat &m, int64_t es) {
        return reinterpret_cast<uintptr_t>(m.ptr) % 16 == 0 && es % 16 == 0 && (m.rows <= 1 || (m.rs % 16 == 0 && m.rs < ((int64_t)1 << 23)));
    };
    int load = MX4_ANY;
    if (a.sa_cs == 1 && a.s_cs == 1 && a.blocks >= 8) load = words(x, 0) && words(q.one, q.E > 1 ? q.es : 0) ? MX4_DIRECT : MX4_BYTES;
    const int64_t used = experts ? std::min(q.E, M) : 1, mean = M / used;
    auto expected = [&](int t) {
        const int64_t bm = mx4_tile_m(t);
        return (experts ? std::max(used, used / 2 + cdiv(M, bm)) : cdiv(M, bm)) * cdiv(N, mx4_tile_n(t));
    };
    // The largest tile that gives three quarters of the CUs work, K = 4096: 256 over 128 at
    // 192 tiles (1536 x 8192: 40.1 us beside 46.6) and 256 (4096 x 4096: 43.4, 55.4), not at
    // 128 (2048 x 4096: 38.2, 29.5); 128 over 64 at 224 (256 x 14336: 21.9, 31.8) and 256
    // (1024 x 4096: 21.1, 27.3), not at 128 (512 x 4096: 16.3, 13.4).
    auto fills = [&](int t) { return 4 * expected(t) >= 3 * (int64_t)d.cus; };
    int tile = MX4_T64;
    if (load == MX4_DIRECT && mean > 128 && fills(MX4_T256)) tile = MX4_T256;
    else if (load != MX4_ANY && mean > 64 && fills(MX4_T128)) tile = MX4_T128;
    // A last round of tiles that half the CUs would sit out: the columns past the rounds
    // before it in smaller tiles, of a launch of their own (4096 x 14336 x 4096, 3 rounds and
    // a half: 149 us beside 155; 2048 x 8400 x 4096, 264 tiles: 55 beside 69), where they are
    // too few to take 256-tiles themselves (51200 x 1024: 200 of 800 tiles).  The first part is
    // not split again (263168 x 7680 would be in 30 parts, each with a last round of its own).
    const int64_t down = cdiv(M, 256), rounds = down * cdiv(N, 256) / d.cus, over = down * cdiv(N, 256) - rounds * d.cus;
    const int64_t first = rounds * d.cus / down * 256;   // columns of the whole rounds
    const int64_t rest = down * cdiv(N - first, 256);
    if (tile == MX4_T256 && !experts && !part && rounds >= 1 && over > 0 && 2 * over <= d.cus && first > 0 && 4 * rest < 3 * (int64_t)d.cus) {
        Stack q1 = q, s1 = s, q2 = q, s2 = s;
        Mat c1 = c, c2 = c;
        q1.one.rows = s1.one.rows = c1.cols = first;
        q2.one.rows = s2.one.rows = c2.cols = N - first;
        q2.one.ptr += first * q.one.rs;
        s2.one.ptr += first * s.one.rs;
        c2.ptr += first * c.cs;
        DG_TRY(codes_plan(x, sx, off, q1, s1, c1, act, false, d, cut, true, out, n));
        return codes_plan(x, sx, off, q2, s2, c2, act, false, d, cut, true, out, n);
    }
    const int64_t q_es = q.E > 1 ? q.es : 0, s_es = q.E > 1 ? s.es : 0;
    const bool ring = tile != MX4_T64 && bytes % 256 == 0 && a.sa_cs == 1 && a.s_cs == 1 && pieces(x, 0) && pieces(q.one, q_es) && pieces(sx, 0) &&
                      pieces(s.one, s_es);
    const int64_t bm = mx4_tile_m(tile), bn = mx4_tile_n(tile);
    a.tiles_n = (int)cdiv(N, bn);
    a.group_m = tile == MX4_T256 ? 4 : 8;
    int64_t units = experts ? ((M + std::min(q.E + 1, M) * (bm - 1)) / bm) * a.tiles_n : cdiv(M, bm) * a.tiles_n;
    // K in pieces where the tiles leave most of the device idle, which larger ones never do; a
    // captured call runs whole: the pieces' workspace may have to be allocated.
    int64_t splits = 1;
    if (!experts && tile == MX4_T64 && 2 * units <= d.cus && a.ktiles >= 4 && cut)
        splits = std::min<int64_t>(d.cus / units, a.ktiles / 2);
    a.kt_per_split = (int)cdiv(std::max(a.ktiles, 1), splits);
    a.splits = (int)cdiv(std::max(a.ktiles, 1), a.kt_per_split);
    if (units > INT32_MAX / a.splits || !fits_a_launch(units * a.splits, 512)) return DG_ERR_OVERFLOW;
    a.units = (int)(units * a.splits);
    out[(*n)++] = {a, tile, load, ring};
    return DG_SUCCESS;
}

// The product of codes with codes, its arguments checked.
dg_status codes_product(const Mat &x, const Mat &sx, const Mat &off, const Stack &q, const Stack &s, const Mat &c, int act, bool experts,
                        hipStream_t stream, Report *r) {
    Device d;
    DG_TRY(ready({&x, &sx, &off, &q.span, &s.span, &c}, &d, r));
    CodesLaunch todo[2];
    int n = 0;
    DG_TRY(codes_plan(x, sx, off, q, s, c, act, experts, d, !capturing(stream, r), false, todo, &n));
    if (r) {
        char text[2][128];
        for (int i = 0; i < n; ++i) {
            const CodesLaunch &l = todo[i];
            Report one = {text[i], sizeof text[i]};
            one.say("%s loads, %dx%d tiles, K in %d pieces, %d workgroups", l.ring ? "ring" : l.load == MX4_DIRECT ? "direct" : l.load == MX4_BYTES ? "vector" : "element",
                    mx4_tile_m(l.tile), mx4_tile_n(l.tile), l.a.splits, l.a.units);
        }
        return n > 1 ? r->say("%s; %s", text[0], text[1]) : r->say("%s", text[0]);
    }
    // The workspace comes before the first launch: without it nothing is written.  One of
    // the launches at most has pieces of K: the first of two has larger tiles.
    WsLease lease;
    for (int i = 0; i < n; ++i) {
        Mx4GemmArgs &a = todo[i].a;
        if (a.splits == 1) continue;
        const size_t tile = (size_t)mx4_tile_m(todo[i].tile) * mx4_tile_n(todo[i].tile);
        if (lease_workspace(stream, a.units * tile * sizeof(float), (size_t)(a.units / a.splits), &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.ws = lease.ws;
        a.counters = lease.counters;
        break;
    }
    for (int i = 0; i < n; ++i) {
        const CodesLaunch &l = todo[i];
        DG_TRY(done(l.ring ? launch_mx4_ring(l.tile, l.a, l.a.units, stream) : launch_mx4_gemm(l.tile, l.load, l.a, l.a.units, stream), stream));
    }
    return DG_SUCCESS;
}

// A 16-bit A that the kernel for few rows stages in LDS.
bool few_aligned(const Mat &x) { return reinterpret_cast<uintptr_t>(x.ptr) % 4 == 0 && (x.rows <= 1 || (x.rs % 4 == 0 && x.rs < 1 << 24)); }

// The product with codes where few rows meet every weight: 16-bit rows (sx null) or codes.
dg_status few_product(const Mat &x, const Mat *sx, const Mat &off, const Stack &q, const Stack &s, const Mat &c, int act, bool experts,
                      hipStream_t stream, Report *r) {
    Device d;
    DG_TRY(ready({&x, sx, &off, &q.span, &s.span, &c}, &d, r));
    const int64_t M = x.rows, N = c.cols, bytes = q.one.cols, K = sx ? 2 * bytes : x.cols;
    Mx4GemmArgs a = {};
    a.A = x.ptr; a.a_rs = x.rs;
    if (sx) { a.SA = sx->ptr; a.sa_rs = sx->rs; a.sa_cs = sx->cols > 1 ? sx->cs : 1; }
    a.Q = q.one.ptr; a.q_rs = q.one.rs; a.q_es = q.es;
    a.S = s.one.ptr; a.s_rs = s.one.rs; a.s_cs = s.one.cols > 1 ? s.one.cs : 1; a.s_es = s.es;
    a.C = out_ptr(c); a.c_rs = c.rs; a.c_cs = c.cs; a.out_kind = c.dtype; a.act = act;
    a.M = (int)M; a.N = (int)N; a.K = (int)K;
    a.row_bytes = (int)bytes;
    a.blocks = (int)cdiv(K, 32);
    if (experts) { a.offsets = off.ptr; a.o_s = off.cs; }
    a.E = (int)q.E;
    const int64_t used = experts ? std::min(q.E, M) : 1, mean = cdiv(M, used);
    const bool aligned = !sx && few_aligned(x);
    const int tm = mean > 32 ? sx ? 4 : 3 : mean > 16 ? 2 : 1;
    const int64_t rows = mx4_few_rows(tm);
    if (aligned) a.a_rows = (int)std::min<int64_t>(M, rows);
    const int64_t k_units = cdiv(bytes, 256), tiles = cdiv(N, 32) * used;
    const bool pieces = !experts && k_units >= 16 && !capturing(stream, r);
    // 32 columns to a workgroup halve the reads of A.  They pay where they still fill the
    // device (N = 14336, K = 4096, 16 rows: BF16 12.9 us beside 16.5, codes 10.4 beside 12.0)
    // or fill it with a long K in two pieces (N = 4096, K = 14336: 32 rows 17.5 beside 20,
    // 16 rows 14.1 beside 14.5, codes 11.1 beside 11.3; 16 rows of 16 experts, N = 7168, K =
    // 4096: 37 beside 50), and not for so few rows that A is little (N = 57344, 1 row: 29.6
    // beside 24.1; N = 4096, 8 rows: 13.3 beside 12.4).
    const bool wide = sx || aligned;
    const int nf = wide && M > 8 && (tiles >= d.cus || (pieces && 2 * tiles >= d.cus)) ? 2 : 1;
    a.tiles_n = (int)cdiv(N, 16 * nf);
    const int64_t units = (experts ? (M + std::min(q.E + 1, M) * (rows - 1)) / rows : cdiv(M, rows)) * a.tiles_n;
    // K in pieces where two of every tile fit the device at once and K is long (16 x 1024 x
    // 8192, 64 tiles: BF16 7.2 us whole, 6.6 in two, 6.3 in four; codes 6.8, 6.2, 5.8); a
    // short K loses (1 x 1024 x 4096: 3.9 whole, 4.6), and so do more tiles (256 of 16 x 4096 x
    // 14336: 14.8 whole, 18.2 in two).  A captured call runs whole, as above.
    int64_t splits = 1;
    if (pieces && 2 * units <= d.cus) splits = std::min<int64_t>(d.cus / units, k_units / 4);
    a.kt_per_split = (int)cdiv(std::max<int64_t>(k_units, 1), splits);
    a.splits = (int)cdiv(std::max<int64_t>(k_units, 1), a.kt_per_split);
    if (units > INT32_MAX / a.splits || !fits_a_launch(units * a.splits, 512)) return DG_ERR_OVERFLOW;
    a.units = (int)(units * a.splits);
    if (r) return r->say("few rows, %dx%d tiles, K in %d pieces, %d workgroups", (int)rows, 16 * nf, a.splits, a.units);
    WsLease lease;
    if (a.splits > 1) {
        if (lease_workspace(stream, (size_t)units * a.splits * mx4_few_sums(tm, nf) * sizeof(float), (size_t)units, &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.ws = lease.ws;
        a.counters = lease.counters;
    }
    return done(launch_mx4_few(sx ? MX4_CODES : x.dtype == DG_F16 ? IN_F16 : IN_BF16, tm, nf, a, a.units, stream), stream);
}

// The product of 16-bit rows with codes where many rows meet every weight (*taken; else
// nothing happens).
dg_status half_product(const Mat &x, const Mat &off, const Stack &q, const Stack &s, const Mat &c, int act, bool experts, hipStream_t stream,
                       Report *r, bool *taken) {
    const int64_t M = x.rows, N = c.cols, K = x.cols, bytes = q.one.cols;
    const int64_t used = experts ? std::min(q.E, M) : 1, mean = M / used;
    const int64_t s_cs = s.one.cols > 1 ? s.one.cs : 1, near = (int64_t)1 << 31;
    auto at = [](const Mat &m, int64_t es, int64_t n) { return reinterpret_cast<uintptr_t>(m.ptr) % n == 0 && es % n == 0 && (m.rows <= 1 || m.rs % n == 0); };
    *taken = mean > 48 && K >= 32 && 128 * x.rs + 2 * K < near && 256 * q.one.rs + bytes < near && 256 * s.one.rs + s.one.cols * s_cs < near;
    if (!*taken) return DG_SUCCESS;
    Device d;
    DG_TRY(ready({&x, &off, &q.span, &s.span, &c}, &d, r));
    auto expected = [&](int64_t bm, int64_t bn) { return (experts ? std::max(used, used / 2 + cdiv(M, bm)) : cdiv(M, bm)) * cdiv(N, bn); };
    const int tile = expected(128, 256) > d.cus / 2 ? MX4_T128x256 : MX4_T64x128;
    const int64_t bm = tile == MX4_T128x256 ? 128 : 64, bn = 2 * bm;
    const int64_t units = experts ? ((M + std::min(q.E + 1, M) * (bm - 1)) / bm) * cdiv(N, bn) : cdiv(M, bm) * cdiv(N, bn);
    // K in pieces of whole tiles of 256 where that fills idle CUs but each only once: of four
    // tiles (64 x 4096 x 4096: 14.7 us in two pieces, 12.6 in four, 14.2 in eight; 64 x 4096 x
    // 14336, 32 tiles of C: 71.9 whole, 26.7 in four, 21.8 in eight, 28.1 in 16), of two where
    // a tile of K takes longer (any address: 150 x 1000 x 4100 18.9 in eight, 21.8 in four) or
    // four pieces are not reached (309 x 160 x 1792: 10.3 in three, 11.0 whole; with four
    // tiles in all, 129 x 1024 x 1024, 10.9 in two, 10.4 whole).  A captured call runs whole,
    // as above.
    const int64_t ktiles = std::max<int64_t>(K / 256, 1);
    int64_t splits = 1;
    const bool via = !(K % 8 == 0 && at(x, 0, 16) && at(q.one, q.E > 1 ? q.es : 0, 4) && (N <= 1 || q.one.rs >= bytes));
    if (!experts && tile == MX4_T64x128 && 2 * units <= d.cus && ktiles >= 6 && !capturing(stream, r))
        splits = std::min<int64_t>(d.cus / units, std::max<int64_t>(ktiles / (via ? 2 : 4), std::min<int64_t>(4, ktiles / 2)));
    // Few rows leave too little work here where the pieces are few, too (64 x 1024 x 8192: 14.2
    // us beside 10.1 of the kernel for few rows; 64 x 4096 x 14336: 21.8 beside 26.8; 64 x
    // 14336 x 4096: 19.1 beside 30.5; 33 x 4096 x 14336: 21.1 beside 20.6).  At any address: 64 x
    // 14336 x 4100 35 us beside 51, 64 x 4096 x 4100 19.4 beside 17.3, 2048 x 4096 x 4100 93
    // beside 338.
    *taken = mean > 128 || 2 * splits * expected(bm, bn) >= d.cus;
    if (!*taken) return DG_SUCCESS;
    Mx4GemmArgs a = {};
    a.A = x.ptr; a.a_rs = x.rs;
    a.Q = q.one.ptr; a.q_rs = q.one.rs; a.q_es = q.es;
    a.S = s.one.ptr; a.s_rs = s.one.rs; a.s_cs = s_cs; a.s_es = s.es;
    a.C = out_ptr(c); a.c_rs = c.rs; a.c_cs = c.cs; a.out_kind = c.dtype; a.act = act;
    a.vec4 = c.cs == c.esize;
    a.M = (int)M; a.N = (int)N; a.K = (int)K;
    a.row_bytes = (int)bytes;
    a.blocks = (int)cdiv(K, 32);
    if (experts) { a.offsets = off.ptr; a.o_s = off.cs; }
    a.E = (int)q.E;
    a.via = via;
    a.s_words = K % 128 == 0 && s_cs == 1 && at(s.one, s.E > 1 ? s.es : 0, 4);
    a.tiles_n = (int)cdiv(N, bn);
    a.group_m = 8;
    a.kt_per_split = (int)cdiv(ktiles, splits);
    a.splits = (int)cdiv(ktiles, a.kt_per_split);
    if (units > INT32_MAX / a.splits || !fits_a_launch(units * a.splits, 512)) return DG_ERR_OVERFLOW;
    a.units = (int)(units * a.splits);
    if (r) return r->say("many rows%s, %dx%d tiles, K in %d pieces, %d workgroups", a.via ? " at any address" : "", (int)bm, (int)bn, a.splits, a.units);
    WsLease lease;
    if (a.splits > 1) {
        if (lease_workspace(stream, (size_t)units * a.splits * bm * bn * sizeof(float), (size_t)units, &lease) != hipSuccess) {
            (void)hipGetLastError();
            return DG_ERR_HIP;
        }
        a.ws = lease.ws;
        a.counters = lease.counters;
    }
    return done(launch_mx4_half(x.dtype == DG_F16 ? IN_F16 : IN_BF16, tile, a, a.units, stream), stream);
}

dg_status gemm_entry(const dg_view *A, const dg_view *SA, const dg_view *offsets, const dg_view *Q, const dg_view *S,
                     const dg_view *C, int act, bool experts, hipStream_t stream, Report *r) {
    Mat x, sx, c, off;
    Stack q, s;
    DG_TRY(canonicalize(A, &x));
    if (SA) DG_TRY(canonicalize(SA, &sx));
    DG_TRY(canonicalize(C, &c));
    if (experts) {
        DG_TRY(canonicalize_stack(Q, &q));
        DG_TRY(canonicalize_stack(S, &s));
    } else {
        DG_TRY(canonicalize(Q, &q.one));
        DG_TRY(canonicalize(S, &s.one));
        for (Stack *t : {&q, &s}) { t->E = 1; t->span = t->one; }
    }
    const bool codes = x.dtype == DG_U8;
    if (!(codes || is_half(x.dtype)) || !is_float(c.dtype)) return DG_ERR_DTYPE;
    if (codes && !SA) return DG_ERR_NULL;
    if (!codes && SA) return DG_ERR_INVALID_ARG;
    if (act != DG_ACT_NONE && act != DG_ACT_RELU && act != DG_ACT_GELU_TANH) return DG_ERR_INVALID_ARG;
    if (x.cols > MOE_MAX_EXTENT / 2) return DG_ERR_OVERFLOW;
    const int64_t M = x.rows, N = c.cols, K = codes ? 2 * x.cols : x.cols;
    if (c.rows != M || q.E < 1) return DG_ERR_SHAPE_MISMATCH;
    DG_TRY(codes_of(q, s, q.E, N, K));
    if (codes && sx.dtype != DG_U8) return DG_ERR_DTYPE;
    if (codes && (sx.rows != M || sx.cols != cdiv(K, 32))) return DG_ERR_SHAPE_MISMATCH;
    if (experts) DG_TRY(index_vector(offsets, q.E + 1, &off));
    if (M > (experts ? MOE_MAX_ROWS : MOE_MAX_EXTENT) || N > MOE_MAX_EXTENT || q.E > MOE_MAX_SCANNED) return DG_ERR_OVERFLOW;
    if (!x.cols_contig()) return DG_ERR_UNSUPPORTED_VIEW;
    if (!codes && (K > (1 << 20) || x.rs >= W4_MAX_PITCH || q.one.rs >= W4_MAX_PITCH || s.one.rs >= W4_MAX_PITCH)) return DG_ERR_OVERFLOW;
    if (self_overlaps(c)) return DG_ERR_STRIDE;
    for (const Mat *m : {&x, &sx, &q.span, &s.span, &off})
        if (spans_overlap(c, *m)) return DG_ERR_ALIAS;
    if (c.empty()) return nothing(r);
    const int64_t mean = cdiv(M, experts ? std::min(q.E, M) : 1);
    // Few rows: that kernel's waves share K and read A again for every 16 or 32 columns, which
    // pays up to 32 rows of codes (N = 14336, K = 4096: 14.8 us beside 16.3; 48: 17.9 beside
    // 16.5) and 16 of 16 bits (12.9 beside 17.6; 32: 18.0 beside 16.5), and up to 64 and 36 where
    // one workgroup to a CU takes all columns (64 rows of codes, 4096 x 4096: 8.4 us beside 9.6,
    // 4096 x 14336 18.7 beside 19.2, 1024 x 8192 8.2 beside 16.1; 32 of 16 bits, 4096 x 4096: 7.1
    // beside 15.0, 33, 4096 x 14336: 19.5 beside 20.6).
    const bool narrow = !experts && N <= 16 * 256;
    const int64_t few = codes ? narrow ? 64 : 32 : narrow && few_aligned(x) ? 36 : 16;
    if (mean <= few) return few_product(x, codes ? &sx : nullptr, off, q, s, c, act, experts, stream, r);
    if (codes) return codes_product(x, sx, off, q, s, c, act, experts, stream, r);
    bool done_here = false;
    const dg_status st = half_product(x, off, q, s, c, act, experts, stream, r, &done_here);
    if (done_here) return st;
    return w4_run(x, off, q, s, nullptr, c, 32, act, experts, true, stream, r);
}

}  // namespace
}  // namespace dg

extern "C" {

dg_status dg_quant_mx4(const dg_view *X, const dg_view *Q, const dg_view *S, dg_mx4_mode mode, hipStream_t stream) {
    return dg::quant_entry(X, Q, S, (int)mode, stream);
}

dg_status dg_dequant_mx4(const dg_view *Q, const dg_view *S, const dg_view *Y, hipStream_t stream) {
    return dg::dequant_entry(Q, S, Y, stream);
}

dg_status dg_gemm_mx4(const dg_view *A, const dg_view *SA, const dg_view *Q, const dg_view *S, const dg_view *C, dg_act act,
                      hipStream_t stream) {
    return dg::gemm_entry(A, SA, nullptr, Q, S, C, (int)act, false, stream, nullptr);
}

dg_status dg_moe_gemm_mx4(const dg_view *A, const dg_view *SA, const dg_view *offsets, const dg_view *Q, const dg_view *S,
                          const dg_view *C, dg_act act, hipStream_t stream) {
    return dg::gemm_entry(A, SA, offsets, Q, S, C, (int)act, true, stream, nullptr);
}

dg_status dg_gemm_mx4_plan(const dg_view *A, const dg_view *SA, const dg_view *Q, const dg_view *S, const dg_view *C, char *buf,
                           size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::gemm_entry(A, SA, nullptr, Q, S, C, DG_ACT_NONE, false, nullptr, &r);
}

dg_status dg_moe_gemm_mx4_plan(const dg_view *A, const dg_view *SA, const dg_view *offsets, const dg_view *Q, const dg_view *S,
                               const dg_view *C, char *buf, size_t len) {
    if (!buf && len) return DG_ERR_INVALID_ARG;
    dg::Report r = {buf, len};
    return dg::gemm_entry(A, SA, offsets, Q, S, C, DG_ACT_NONE, true, nullptr, &r);
}

}  // extern "C"
