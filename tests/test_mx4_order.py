"""What an MXFP4 call does before its first launch, on the CPU: csrc/mx4.cpp and csrc/view.cpp compiled against
stand-ins that note launches and leases of the workspace and enqueue nothing.  Whatever can fail (here the lease) has to
come before anything is enqueued, since outputs stay untouched on error."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_19_amd", "csrc")

STAND_INS = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "entry.hpp"
#include "moe.hpp"
#include "mx4.hpp"

static bool fails;
namespace dg {
bool env_on(const char *) { return false; }
dg_status check_pointer(const void *) { return DG_SUCCESS; }
dg_status current_device(Device *d, bool) { *d = Device(); d->gfx950 = true; return DG_SUCCESS; }
hipError_t lease_workspace(hipStream_t, size_t bytes, size_t, WsLease *out) {
    std::printf("lease ");
    if (fails) return hipErrorOutOfMemory;
    static float ws[1];
    static int counters[1];
    out->ws = ws;
    out->counters = counters;
    return bytes ? hipSuccess : hipErrorInvalidValue;
}
static hipError_t launch(const char *what, const Mx4GemmArgs &a) {
    std::printf("%s%s ", what, a.splits > 1 ? a.ws && a.counters ? "-pieces" : "-without-workspace" : "");
    return hipSuccess;
}
hipError_t launch_mx4_gemm(int, int, const Mx4GemmArgs &a, int64_t, hipStream_t) { return launch("tile", a); }
hipError_t launch_mx4_ring(int, const Mx4GemmArgs &a, int64_t, hipStream_t) { return launch("ring", a); }
hipError_t launch_mx4_half(int, int, const Mx4GemmArgs &a, int64_t, hipStream_t) { return launch("half", a); }
hipError_t launch_mx4_few(int, int, int, const Mx4GemmArgs &a, int64_t, hipStream_t) { return launch("few", a); }
hipError_t launch_mx4_quant(bool, const Mx4QuantArgs &, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_mx4_dequant(const Mx4DequantArgs &, int64_t, hipStream_t) { return hipSuccess; }
dg_status w4_run(const Mat &, const Mat &, const Stack &, const Stack &, const Stack *, const Mat &, int, int, bool, bool, hipStream_t, Report *) {
    std::printf("w4 ");
    return DG_SUCCESS;
}
}  // namespace dg
extern "C" {
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

// argv: "codes" or "half", M, N, K, "fail" or "work"
int main(int, char **argv) {
    const bool codes = !std::strcmp(argv[1], "codes");
    const int64_t M = std::atoll(argv[2]), N = std::atoll(argv[3]), K = std::atoll(argv[4]), bytes = (K + 1) / 2, blocks = (K + 31) / 32;
    fails = !std::strcmp(argv[5], "fail");
    int64_t at = 1 << 20;
    auto view = [&](int64_t rows, int64_t cols, dg_dtype t, int64_t esize) {
        dg_view v = {};
        v.ptr = reinterpret_cast<decltype(v.ptr)>(at);
        v.dtype = t;
        v.ndim = 2;
        v.shape[0] = rows; v.shape[1] = cols;
        v.stride[0] = cols * esize; v.stride[1] = esize;
        at += (rows * cols * esize + 4095) / 4096 * 4096;
        return v;
    };
    const dg_view A = codes ? view(M, bytes, DG_U8, 1) : view(M, K, DG_BF16, 2), SA = view(M, blocks, DG_U8, 1), Q = view(N, bytes, DG_U8, 1),
                  S = view(N, blocks, DG_U8, 1), C = view(M, N, DG_F32, 4);
    std::printf("%s\n", dg_gemm_mx4(&A, codes ? &SA : nullptr, &Q, &S, &C, DG_ACT_NONE, nullptr) == DG_SUCCESS ? "success" : "error");
    return 0;
}
"""


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx4")
    src, exe = d / "calls.cpp", str(d / "calls")
    src.write_text(STAND_INS)
    subprocess.run(["g++", "-O0", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                    "-isystem/opt/rocm/include", os.path.join(CSRC, "mx4.cpp"), os.path.join(CSRC, "view.cpp"), str(src), "-o", exe], check=True)
    return lambda *args: subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True).stdout.split()


# few rows, tiles of codes, whole rounds of tiles with the other columns in a launch of their own whose K is cut, many rows
PIECES = [("codes", 16, 1000, 8192, ["few-pieces"]), ("half", 16, 1000, 8192, ["few-pieces"]), ("codes", 70, 130, 9000, ["tile-pieces"]),
          ("codes", 300, 33024, 1024, ["ring", "tile-pieces"]), ("codes", 300, 33024, 1000, ["tile", "tile-pieces"]),
          ("half", 100, 4096, 4096, ["half-pieces"])]


@pytest.mark.parametrize("kind,M,N,K,launches", PIECES)
def test_the_workspace_is_there_before_the_first_launch(call, kind, M, N, K, launches):
    assert call(kind, M, N, K, "work") == ["lease", *launches, "success"]


@pytest.mark.parametrize("kind,M,N,K,launches", PIECES)
def test_without_a_workspace_nothing_is_launched(call, kind, M, N, K, launches):
    assert call(kind, M, N, K, "fail") == ["lease", "error"]


@pytest.mark.parametrize("kind,M,N,K,launches", [("codes", 4096, 4200, 512, ["ring", "tile"]), ("codes", 4096, 14336, 4096, ["ring", "ring"]),
                                                 ("codes", 1, 64, 64, ["few"]), ("half", 2048, 4096, 4096, ["half"]), ("half", 40, 300, 100, ["w4"])])
def test_calls_without_pieces_need_none(call, kind, M, N, K, launches):
    assert call(kind, M, N, K, "fail") == [*launches, "success"]


@pytest.mark.parametrize("M,N,K,launches", [
    (4096, 14336, 4096, 2), (2048, 8400, 512, 2), (33000, 1024, 512, 2), (51200, 1024, 512, 1), (263168, 7680, 512, 1), (66000, 7700, 512, 1),
    (20000, 1024, 512, 2), (300, 33024, 512, 2)])
def test_a_last_round_is_one_launch_of_its_own_at_most(call, M, N, K, launches):
    # 128, 8, 129, 200, 1028, 258 (a round and more), 79 and 2 256-tiles behind the whole rounds' columns
    assert len(call("codes", M, N, K, "work")) - 1 - ("lease" in call("codes", M, N, K, "work")) == launches
