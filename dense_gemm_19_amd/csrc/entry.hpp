// entry.hpp -- host helpers of the operators' entry points (mixture of experts, 4-bit
// weights, microscaled 4-bit operands): views of index vectors and of expert stacks,
// what a call checks of the device and stream, and the text of a plan.
#pragma once
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include <hip/hip_runtime_api.h>

#include "dg.h"
#include "runtime.hpp"
#include "view.hpp"

#define DG_TRY(expr) \
    do { const dg_status st_ = (expr); if (st_ != DG_SUCCESS) return st_; } while (0)

namespace dg {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }


inline bool is_float(dg_dtype t) { return t == DG_F32 || t == DG_F16 || t == DG_BF16; }
inline bool is_half(dg_dtype t) { return t == DG_F16 || t == DG_BF16; }

// A vector of `len` 32-bit integers ([len] or [1][len]).
inline dg_status index_vector(const dg_view *v, int64_t len, Mat *m) {
    DG_TRY(canonicalize(v, m));
    if (m->dtype != DG_I32) return DG_ERR_DTYPE;
    if (m->rows * m->cols != len || (len > 0 && m->rows != 1)) return DG_ERR_SHAPE_MISMATCH;
    return DG_SUCCESS;
}

// Elements one after another in row-major order.
inline bool contiguous(const Mat &m) { return m.empty() || (m.cols_contig() && (m.rows <= 1 || m.rs == m.cols * m.esize)); }

// A [E][rows][cols] view: one expert's matrix and the byte stride of experts.
// span: the same matrix with the byte span of all experts.
struct Stack {
    Mat one;
    int64_t E = 0, es = 0;
    Mat span;
};

inline dg_status canonicalize_stack(const dg_view *v, Stack *s) {
    if (!v) return DG_ERR_NULL;
    if (v->ndim != 3) return DG_ERR_NDIM;
    if (v->shape[0] < 0 || v->stride[0] < 0) return DG_ERR_STRIDE;
    dg_view m = *v;
    m.ndim = 2;
    for (int d = 0; d < 2; ++d) {
        m.shape[d] = v->shape[d + 1];
        m.stride[d] = v->stride[d + 1];
    }
    if (v->shape[0] == 0) m.shape[0] = 0;   // no experts: nothing is read
    DG_TRY(canonicalize(&m, &s->one));
    if (v->shape[0] == 0) s->one.rows = v->shape[1];
    if (v->stride[0] % s->one.esize != 0) return DG_ERR_STRIDE;
    s->E = v->shape[0];
    s->es = v->stride[0];
    s->span = s->one;
    int64_t reach;
    if (s->E > 0 && !s->one.empty()) {
        if (__builtin_mul_overflow(s->E - 1, s->es, &reach) ||
            __builtin_add_overflow(s->one.hi, (uintptr_t)reach, &s->span.hi))
            return DG_ERR_OVERFLOW;
    }
    return DG_SUCCESS;
}

// A written stack must not overlap itself: its matrices do not, and each starts
// past the end of the one before.
inline bool stack_overlaps(const Stack &s) {
    if (s.E == 0 || s.one.empty()) return false;
    return self_overlaps(s.one) || (s.E > 1 && s.es < (int64_t)(s.one.hi - s.one.lo));
}

// Where a call's plan is written instead of running it.
struct Report {
    char *buf;
    size_t len;
    __attribute__((format(printf, 2, 3))) dg_status say(const char *format, ...) {
        va_list args;
        va_start(args, format);
        if (len) std::vsnprintf(buf, len, format, args);
        va_end(args);
        return DG_SUCCESS;
    }
};

// Nothing to launch.
inline dg_status nothing(Report *r) { return r ? r->say("nothing to do") : DG_SUCCESS; }

// The current device (a plan needs none).
inline dg_status ready(std::initializer_list<const Mat *> ms, Device *d, const Report *r) {
    DG_TRY(current_device(d, !r));
    if (r) return DG_SUCCESS;
    if (!d->gfx950) return DG_ERR_ARCH;
    if (env_on("DG_CHECK_POINTERS"))
        for (const Mat *m : ms)
            if (m && m->ptr && m->hi > m->lo) DG_TRY(check_pointer(m->ptr));
    return DG_SUCCESS;
}

inline dg_status done(hipError_t e, hipStream_t stream) {
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return DG_ERR_HIP;
    }
    if (env_on("DG_SYNC_DEBUG") && (hipStreamSynchronize(stream) != hipSuccess || hipGetLastError() != hipSuccess))
        return DG_ERR_HIP;
    return DG_SUCCESS;
}

// The stream is being captured (or cannot be asked): no workspace is allocated.
// (A plan is that of a call that is not captured.)
inline bool capturing(hipStream_t stream, const Report *r) {
    if (r) return false;
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &cap) == hipSuccess) return cap != hipStreamCaptureStatusNone;
    (void)hipGetLastError();
    return true;
}

// A launch holds fewer than 2^32 threads.
inline bool fits_a_launch(int64_t workgroups, int64_t threads) { return workgroups < ((int64_t)1 << 32) / threads; }

inline char *out_ptr(const Mat &m) { return const_cast<char *>(m.ptr); }

}  // namespace dg
