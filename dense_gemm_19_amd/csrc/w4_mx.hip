// w4_mx.hip -- products of 16-bit activations with microscaled 4-bit weights (E2M1
// codes, an E8M0 scale byte for 32 of them): the kernels of w4.hpp with that decoding, for
// what neither mx4_few.hip nor mx4_half.hip takes: 17 to 48 rows (40 x 14336 x 4096: 19.1 us),
// 49 to 128 where those tiles leave half of the device idle, and any number where K is
// below 32 or rows lie 8 MiB apart and more.
#include "w4.hpp"

namespace dg {
namespace {

template <int IN>
hipError_t launch(int tm, const W4Args &a, int64_t units, hipStream_t s) {
    switch (tm) {
    case 2: return launch_t<IN, 2, 4, 1>(a, units, s);
    case 3: return launch_t<IN, 3, 4, 1>(a, units, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_w4_mx(int in_kind, int tm, const W4Args &a, int64_t units, hipStream_t s) {
    return in_kind == IN_BF16 ? launch<IN_BF16>(tm, a, units, s) : launch<IN_F16>(tm, a, units, s);
}

}  // namespace dg
