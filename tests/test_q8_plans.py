"""What the 8-bit matrices' host code makes and how large, under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): what a bind allocates, exceptions at the C entries,
and the workspaces that the rule for cutting products up asks for, operands at odd
addresses among them."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

NATIVE = os.path.join(ROOT, "tests", "native")
CSRC = os.path.join(ROOT, "sharded_shard_amd", "csrc")
ROCM_INCLUDE = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
FLAGS = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=undefined", "-ffp-contract=off", "-D__HIP_PLATFORM_AMD__",
         "-I" + ROCM_INCLUDE, "-Wall", "-Wextra", "-Wno-unused-parameter"]


def run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900, **kw)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-6000:])
    return r.stdout


def test_q8_plans_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path / "q8_plan_harness")
    srcs = [os.path.join(NATIVE, f) for f in ("q8_plan_harness.cpp", "fake_hip.cpp", "fake_launch.cpp")]
    srcs += [os.path.join(CSRC, f) for f in ("capi.cpp", "plan.cpp", "reshard.cpp", "host_adamw.cpp",
                                             "q8.cpp", "q8_cut.cpp")]
    # the launches' stand-ins, under another name the one of the rule that cuts products up:
    # the library's own is what is looked at here
    fakes = str(tmp_path / "fake_q8.o")
    run([gxx, *FLAGS, "-Dq8_cut=unused_q8_cut", "-c", os.path.join(NATIVE, "fake_q8.cpp"), "-o", fakes])
    run([gxx, *FLAGS, *srcs, fakes, "-pthread", "-o", out])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    env.pop("FSDP_FAULT", None)
    assert "ALL OK" in run([out], env=env)
