"""The host code of the key-value cache, attention and rotary calls
(kv_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, driven by
``tests/host/kv_validator_check.cpp`` over extreme and defective arguments
(CPU only: no call gets as far as HIP).  The other objects are linked as
built; only the host file and the driver are instrumented."""

import glob
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dequant_gemv_rht_amd", "_lib")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
INC = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include")]


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-2000:]}\n{r.stderr[-2000:]}"
    return r


def test_kv_validator_under_asan_ubsan(tmp_path):
    objs = sorted(o for o in glob.glob(os.path.join(LIB, "*.o")) if os.path.basename(o) != "kv_api.cpp.o")
    if not objs:
        pytest.fail("the library's objects are not built: run python -m dequant_gemv_rht_amd.build")
    api, drv, exe = (str(tmp_path / n) for n in ("kv_api.o", "driver.o", "driver"))
    _run(["g++", "-std=c++17", "-g", "-O1", *SAN, *INC, "-c",
          os.path.join(ROOT, "dequant_gemv_rht_amd", "csrc", "kv_api.cpp"), "-o", api])
    _run(["g++", "-std=c++17", "-g", "-O1", *SAN, *INC, "-c",
          os.path.join(ROOT, "tests", "host", "kv_validator_check.cpp"), "-o", drv])
    _run(["g++", *SAN, drv, api, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    assert "checked" in _run([exe], env=env, timeout=600).stdout
