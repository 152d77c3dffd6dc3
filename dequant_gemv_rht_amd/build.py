"""Build libwq.so for gfx950 with hipcc, in the source tree.

    python -m dequant_gemv_rht_amd.build          # compile every source, link
    python -m dequant_gemv_rht_amd.build --asm    # also keep the AMD assembly

Each source file compiles to its own object in parallel; the library lands
in ``dequant_gemv_rht_amd/_lib/libwq.so``.  ``csrc/binding.cpp``, the native
half of the Python binding, compiles against torch's headers with the host
compiler into ``_lib/_wqpy.so``; it holds no device code, and where torch's
headers or a host compiler are missing the library is built without it, with
a warning.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT, "libwq.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    f"--offload-arch={ARCH}",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


BINDING = "binding.cpp"
BINDING_LIB = os.path.join(OUT, "_wqpy.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".hip", ".cpp")) and f != BINDING)


def _replace(cmd, out: str, what: str) -> None:
    """Run `cmd` + an output file of this process's own, then put that in place of `out`."""
    tmp = out + ".tmp%d" % os.getpid()
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    os.replace(tmp, out)


def build_binding() -> str:
    import sysconfig

    import torch

    t = os.path.dirname(torch.__file__)
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(t, "lib")
    _replace([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
              "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
              *(a for i in inc for a in ("-isystem", i)), os.path.join(CSRC, BINDING), f"-L{lib}", "-ltorch_python",
              "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", f"-Wl,-rpath,{lib}"], BINDING_LIB, f"{BINDING}: g++")
    return BINDING_LIB


def _compile(src: str, asm: bool) -> str:
    obj = os.path.join(OUT, os.path.basename(src) + ".o")
    cmd = [HIPCC] + COMMON + ["-c", src, "-o", obj]
    if src.endswith(".hip"):
        cmd[1:1] = ["-x", "hip"]
        if os.path.basename(src) == "gemv_stream.hip":
            # the GEMV kernels' first seven arguments (the linears' first
            # workgroups) arrive preloaded in scalar registers
            cmd += ["-mllvm", "-amdgpu-kernarg-preload-count=7"]
        if asm:
            cmd += ["-save-temps=obj"]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=OUT)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(asm: bool = False, jobs: int | None = None) -> str:
    os.makedirs(OUT, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 4)))
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(lambda s: _compile(s, asm), srcs))
        _replace([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC"] + objs, LIB, "link")
        try:
            binding.result()
        except (RuntimeError, OSError, ImportError) as e:
            # the linears do not need it; the calls that do say so when used
            if os.path.exists(BINDING_LIB):
                os.remove(BINDING_LIB)
            warnings.warn(f"built without the cache, attention and rotary calls of the Python binding: {e}",
                          RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(asm="--asm" in sys.argv))
