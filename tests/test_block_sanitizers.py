"""The host code of the block's operators (gdn_block_api.hip: validation, row
layouts, workspace carving and dispatch) built with AddressSanitizer and
UndefinedBehaviorSanitizer on the host and run without a GPU:
tests/sanitize/block_stubs.cpp stands in for the kernel launchers and checks
every device pointer they receive, tests/sanitize/block_driver.cpp calls every
entry point over a grid of problems."""

import os
import subprocess

import pytest

from .test_host_sanitizers import CLANG, CSRC, HIPCC, INC, SAN, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                    reason="ROCm compilers not found")
def test_block_host_code_under_asan_and_ubsan(tmp_path):
    d = str(tmp_path)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    common = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-I", INC, "-I", CSRC,
              "-I", SAN]
    host = [HIPCC, "-x", "hip", "--cuda-host-only", "-Wno-unused-command-line-argument"]
    _run(host + common + san + ["-c", os.path.join(CSRC, "gdn_block_api.hip"), "-o", "api.o"], d)
    _run(host + common + san + ["-c", os.path.join(SAN, "block_stubs.cpp"), "-o", "stubs.o"], d)
    _run([CLANG, "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined"] + common +
         ["-c", os.path.join(SAN, "block_driver.cpp"), "-o", "driver.o"], d)
    _run([CLANG, "-fsanitize=address,undefined", "api.o", "stubs.o", "driver.o",
          "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", "driver"], d)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([os.path.join(d, "driver")], cwd=d, capture_output=True, text=True,
                       env=env, timeout=300)
    print(r.stdout[-2000:])
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-5000:]
    assert " 0 failed" in r.stdout
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
