"""The serving operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU): serve_validate.cpp,
serve_plan.cpp and serve_api.cpp, which read caller-supplied descriptors and multiply their extents, are built with
g++ and both sanitizers into a library of their own (launchers are host stubs), and the argument tests run against
it in a child process.  What is refused there returns before any launch; what is accepted is planned."""
import os
import shutil
import subprocess
import sys

import pytest

import test_sanitize as base

ROOT, CSRC = base.ROOT, base.CSRC
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SOURCES = [os.path.join(CSRC, f) for f in ("serve_validate.cpp", "serve_plan.cpp", "serve_api.cpp", "wq_validate.cpp",
                                           "wq_plan.cpp")]
SOURCES += [os.path.join(ROOT, "tests", "sanitize", f) for f in ("serve_stub.cpp", "host_stub.cpp")]
TESTS = ["tests/test_serve_host.py", "tests/test_serve_host_edges.py"]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_serve_host_code_under_asan_ubsan(tmp_path):
    runtime = base._asan_runtime()
    if runtime is None:
        pytest.skip("g++ has no AddressSanitizer runtime")
    lib = str(tmp_path / "libwqserve_san.so")
    build = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=all", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
         "-I", os.path.join(ROOT, "include"), "-I", CSRC, *SOURCES, "-o", lib], capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    env = dict(os.environ)
    env["LD_PRELOAD"] = runtime + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:abort_on_error=1:verify_asan_link_order=0"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["WQ_HOST_LIBRARY"] = lib
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-rs", "-x", "-p", "no:cacheprovider", "-m", "not gpu", *TESTS],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
    assert " passed" in r.stdout and "skipped" not in r.stdout, out[-3000:]
