"""The host code of the serving operators around a step's attention under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU), built and run as test_sanitize_serve.py does it for the others."""
import os
import shutil
import subprocess
import sys

import pytest

import test_sanitize as base
import test_sanitize_serve as serve

SOURCES = serve.SOURCES + [os.path.join(base.CSRC, f) for f in ("serve_step_validate.cpp", "serve_step_plan.cpp",
                                                               "serve_step_api.cpp")]
SOURCES += [os.path.join(base.ROOT, "tests", "sanitize", "step_stub.cpp")]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_step_host_code_under_asan_ubsan(tmp_path):
    runtime = base._asan_runtime()
    if runtime is None:
        pytest.skip("g++ has no AddressSanitizer runtime")
    lib = str(tmp_path / "libwqstep_san.so")
    build = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=all", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(serve.ROCM, "include"),
         "-I", os.path.join(base.ROOT, "include"), "-I", base.CSRC, *SOURCES, "-o", lib], capture_output=True, text=True,
        timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    env = dict(os.environ)
    env["LD_PRELOAD"] = runtime + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:abort_on_error=1:verify_asan_link_order=0"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["WQ_HOST_LIBRARY"] = lib
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-rs", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_step_host.py"], cwd=base.ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout, out[-3000:]
