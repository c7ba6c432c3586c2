// w4.hip -- products with 4-bit integer weights, group scales of 16 or 32 bits and
// zero points (kernels in w4.hpp).
#include "w4.hpp"

namespace dg {
namespace {

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
