"""The host code of the slots, adapters and sampling calls (serve_api.cpp,
serve_plan.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, driven
by ``tests/host/serve_validator_check.cpp`` over extreme and defective
arguments (CPU only: no call gets as far as HIP)."""

import glob
import os

import pytest

from test_kv_sanitizers import INC, LIB, ROOT, SAN, _run


def test_serve_validator_under_asan_ubsan(tmp_path):
    mine = ("serve_api.cpp", "serve_plan.cpp")
    objs = sorted(o for o in glob.glob(os.path.join(LIB, "*.o")) if os.path.basename(o)[:-2] not in mine)
    if not objs:
        pytest.fail("the library's objects are not built: run python -m dequant_gemv_rht_amd.build")
    own = []
    for src in [os.path.join(ROOT, "dequant_gemv_rht_amd", "csrc", f) for f in mine] + [
            os.path.join(ROOT, "tests", "host", "serve_validator_check.cpp")]:
        own.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run(["g++", "-std=c++17", "-g", "-O1", *SAN, *INC, "-c", src, "-o", own[-1]])
    exe = str(tmp_path / "driver")
    _run(["g++", *SAN, *own, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    assert "checked" in _run([exe], env=env, timeout=600).stdout
