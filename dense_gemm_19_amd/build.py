"""Build libdg.so for gfx950 with hipcc (every source, every call).

    python -m dense_gemm_19_amd.build [-v] [--incremental]

Objects go to dense_gemm_19_amd/_build/; the library to dense_gemm_19_amd/libdg.so,
the tensor binding of its newer entry points (torch_bind.cpp) to
dense_gemm_19_amd/_dgtorch.so.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdg.so")
BIND = os.path.join(HERE, "_dgtorch.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops off: no packed FP32 instructions are emitted anywhere.
HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
# Per-source extra flags.  The FP8 kernels promote each matrix-core block sum on
# the vector ALUs; the VGPR form of the MFMA instructions lets those sums land
# where the ALUs can use them (no copies out of accumulation registers).
EXTRA_FLAGS = {"gemm_dtl_f8.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
               "gemm_dtl_f8s.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]

HIP_SOURCES = ["gemm_mfma.hip", "gemm_dtl_f16.hip", "gemm_dtl_bf16.hip", "gemm_dtl_f8.hip", "gemm_dtl_f8s.hip", "skinny.hip",
               "epilogue.hip", "calib.hip", "quant.hip", "noalloc.hip", "moe_gemm_f16.hip", "moe_gemm_bf16.hip", "w4.hip",
               "w4_mx.hip", "moe_route.hip", "mx4_quant.hip", "mx4_gemm.hip", "mx4_ring.hip", "mx4_half.hip", "mx4_few.hip"]
HOST_SOURCES = ["view.cpp", "plan.cpp", "dg.cpp", "gemm_dtl.cpp", "moe.cpp", "mx4.cpp"]


def _newest_header() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hpp", ".h"))]
    hs += [os.path.join(ROOT, "include", h) for h in os.listdir(os.path.join(ROOT, "include"))]
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, verbose: bool, incremental: bool = False) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if incremental and os.path.exists(obj):
        t = os.path.getmtime(obj)
        if t > os.path.getmtime(os.path.join(CSRC, src)) and t > _newest_header():
            return obj
    hip = src.endswith(".hip")
    flags = HIP_FLAGS + ["-Rpass-analysis=kernel-resource-usage"] if hip else HOST_FLAGS
    cmd = [HIPCC] + flags + EXTRA_FLAGS.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    lines = r.stderr.splitlines()
    # hipcc's host pass does not know the packed-fp32 feature; that note is harmless
    err = "\n".join(l for l in lines if "packed-fp32-ops" not in l and "kernel-resource-usage" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {src}\n{err}")
    if hip:
        spills = _scratch_kernels(lines)
        if spills:
            os.remove(obj)
            raise RuntimeError(f"{src}: kernels use scratch memory (register spills): {spills}")
    if err.strip() and verbose:
        print(err)
    return obj


def _scratch_kernels(remarks) -> list:
    """Kernels whose resource-usage remark reports scratch (spilled registers)."""
    out, name = [], None
    for l in remarks:
        if "remark: Function Name:" in l:
            name = l.split("Function Name:")[1].split("[")[0].strip()
        elif "ScratchSize [bytes/lane]:" in l and name:
            n = int(l.split("ScratchSize [bytes/lane]:")[1].split("[")[0].strip())
            if n > 0:
                out.append(f"{name} ({n} bytes/lane)")
    return out


def _bind_object(verbose: bool, incremental: bool) -> str:
    """torch_bind.cpp, compiled against torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    src, obj = os.path.join(CSRC, "torch_bind.cpp"), os.path.join(BUILD, "torch_bind.cpp.o")
    if incremental and os.path.exists(obj) and os.path.getmtime(obj) > max(
            os.path.getmtime(src), os.path.getmtime(os.path.join(ROOT, "include", "dg.h"))):
        return obj
    inc = [f"-isystem{p}" for p in cpp_extension.include_paths()] + ["-isystem/opt/rocm/include"]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(ROOT, "include"),
           "-isystem" + sysconfig.get_paths()["include"], *inc, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: torch_bind.cpp\n{r.stderr}")
    return obj


def _link_bind(obj: str, verbose: bool) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", f"-L{libs}", "-ltorch_python", "-ltorch_cpu",
           "-lc10_hip", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BIND)


def build(verbose: bool = False, jobs: int | None = None, incremental: bool = False) -> str:
    """Compile every source (or, with incremental=True, those newer than their
    object) and link libdg.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = HIP_SOURCES + HOST_SOURCES
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 4)))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(_bind_object, verbose, incremental)
        objs = list(ex.map(lambda s: _compile(s, verbose, incremental), srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libdg.so", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _link_bind(bind.result(), verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, incremental="--incremental" in sys.argv))
