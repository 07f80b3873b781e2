"""Orthogonalisation plans without a GPU: what they refuse, and the host code of
several binds under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

NATIVE = os.path.join(ROOT, "tests", "native")
CSRC = os.path.join(ROOT, "sharded_shard_amd", "csrc")
capi = pytest.importorskip("sharded_shard_amd.capi")
NS = [(3.4445, -4.7750, 2.0315)] * 5

ROCM_INCLUDE = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")


def _harness(tmp_path, sources, host=("muon.cpp",)):
    """Build the sources with the library's host code under sanitizers and run them."""
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(ROCM_INCLUDE, "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = str(tmp_path / "harness")
    srcs = [os.path.join(NATIVE, f) for f in sources]
    srcs += [os.path.join(CSRC, f) for f in ("capi.cpp", "plan.cpp", "reshard.cpp", "host_adamw.cpp",
                                             "ortho.cpp") + tuple(host)]
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-ffp-contract=off", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE,
           "-Wall", "-Wextra", "-Wno-unused-parameter", *srcs, "-pthread", "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    env.pop("FSDP_FAULT", None)
    r = subprocess.run([out], capture_output=True, text=True, timeout=900, env=env)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-6000:])
    assert "ALL OK" in r.stdout


def test_a_plan_keeps_the_dtype_of_its_first_bind(tmp_path):
    _harness(tmp_path, ["ortho_plan_harness.cpp", "fake_hip.cpp", "fake_launch.cpp", "fake_muon.cpp"])


def test_plans_with_two_part_operands(tmp_path):
    _harness(tmp_path, ["ortho_fine_harness.cpp", "fake_hip.cpp", "fake_launch.cpp"], host=())


def test_products_are_named():
    from sharded_shard_amd.group import Orthogonalizer
    plans = [Orthogonalizer([(300, 400), (20, 30)], products=p) for p in ("fp16", "fp16x2")]
    assert plans[0].workspace_bytes < plans[1].workspace_bytes
    with pytest.raises(ValueError, match="fp16x2"):
        Orthogonalizer([(300, 400)], products="fp32")
    with pytest.raises(capi.FsdpError) as ei:
        capi.fsdp_ortho_plan_set_products(plans[0].plan, -1)
    assert ei.value.status == capi.FSDP_E_UNSUPPORTED
    few = [Orthogonalizer([(100, 4000)], products=p) for p in ("fp16", "fp16x2")]
    assert few[0].workspace_bytes == few[1].workspace_bytes


def test_every_step_has_three_coefficients():
    """Steps of other lengths whose numbers happen to make whole threes as well."""
    for bad in ([(1.5, -0.5), (0.0, 1.5, -0.5, 0.0)], [(1.5, -0.5, 0.0, 1.5, -0.5, 0.0), ()],
                [(1.0, 2.0)], [NS[0], (1.5,), (-0.5, 0.0, 1.5, -0.5, 0.0)]):
        with pytest.raises(ValueError, match="three"):
            capi.fsdp_ortho_plan_create([4], [8], bad)
    # any iterable of steps of any iterables
    capi.fsdp_ortho_plan_destroy(capi.fsdp_ortho_plan_create([4], [8], (iter(c) for c in NS)))


def _tops(coeffs):
    """The largest singular value after each step, from any in [0, 1]."""
    import numpy as np
    s, out = np.linspace(0.0, 1.0, 200001), []
    for a, b, c in coeffs:
        s = np.abs(a * s + b * s ** 3 + c * s ** 5)
        out.append(s.max())
    return out


def test_steep_schedules_are_accepted_as_far_as_the_range_allows():
    """The room that a step leaves for rounding is its own: handed on from step
    to step it refused schedules that stay far inside the range."""
    steep = [(8.205, -22.90, 16.46), (4.066, -2.861, 0.518)]
    assert max(_tops(steep)) < 2.1
    for coeffs in (steep, steep + [(1.0, 0.0, 0.0)] * 40, [(2.0, 0, 0), (1.95, 0, 0)] + [(1.0, 0, 0)] * 20):
        assert max(_tops(coeffs)) < 4.0
        capi.fsdp_ortho_plan_destroy(capi.fsdp_ortho_plan_create([4], [8], coeffs))
    # the second's 2 * 1.97 * 1.02 is 4.02
    for coeffs in ([(2.0, 0, 0), (2.0, 0, 0)], [(2.0, 0, 0), (1.97, 0, 0)] + [(1.0, 0, 0)] * 20,
                   [(4.0, 0, 0)], steep + [(2.3, 0, 0)], [(1.0, 0, 0)] * 9 + [(4.1, 0, 0)]):
        with pytest.raises(capi.FsdpError) as ei:
            capi.fsdp_ortho_plan_create([4], [8], coeffs)
        assert ei.value.status == capi.FSDP_E_UNSUPPORTED


@pytest.mark.parametrize("c", [1e-12, -1e-12, 1e-17, -1e-17, 1e-200, -1e-300, 5e-324])
def test_a_vanishing_fifth_order_term_does_not_hide_a_maximum(c):
    """15 s - 15 s^3 reaches 5.8 at s = 0.58 and returns to 0 at 1; so it does with
    c s^5 too small to count."""
    with pytest.raises(capi.FsdpError) as ei:
        capi.fsdp_ortho_plan_create([4], [8], [(15.0, -15.0, c)])
    assert ei.value.status == capi.FSDP_E_UNSUPPORTED
    # the same shape within the range: 2.6 at its largest
    capi.fsdp_ortho_plan_destroy(capi.fsdp_ortho_plan_create([4], [8], [(6.8, -6.8, c)]))


def test_bind_needs_an_address_for_every_matrix():
    """The C call reads n_mats of each array."""
    p = capi.fsdp_ortho_plan_create([5, 0, 7], [7, 4, 3], NS)
    ins, outs = [0x10000, 0, 0x20000], [0x30000, 0, 0x40001]
    for a, b in ((ins[:2], outs), (ins, outs[:1]), ([], []), (ins + [0x50000], outs + [0x60000])):
        with pytest.raises(ValueError, match="3 matrices"):
            capi.fsdp_ortho_bind(p, a, b, stream=0)
    with pytest.raises(capi.FsdpError) as ei:      # whole lists go on to the C checks
        capi.fsdp_ortho_bind(p, ins, outs, stream=0)
    assert ei.value.status == capi.FSDP_E_ALIGN
    capi.fsdp_ortho_plan_destroy(p)


def test_product_launchers_refuse_a_tile_that_they_do_not_have():
    """Before anything is launched: an unknown side ran as 64 x 64 tiles."""
    import ctypes
    gram = getattr(capi.lib, "_ZN4fsdp17launch_ortho_gramEiPKNS_9OrthoTileElS2_liPKNS_8OrthoMatEPvibP12ihipStream_t")
    gram.restype = ctypes.c_int
    gram.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_bool,
                     ctypes.c_void_p]
    hip_error_invalid_value = 1
    for side in (0, 32, 96, 160, 512, -64):
        for split in (1, 2):
            assert gram(side, None, 1, None, 1, split, None, None, 0, True, None) == hip_error_invalid_value


def test_plans_past_a_launch_are_refused():
    """A launch has less than 2^32 threads: 65536 x 2^20 elements are 2^23 blocks of
    256 at the start, two such matrices are one too many."""
    capi.fsdp_ortho_plan_destroy(capi.fsdp_ortho_plan_create([1 << 16], [1 << 20], NS[:1]))
    with pytest.raises(capi.FsdpError, match="too many tiles") as ei:
        capi.fsdp_ortho_plan_create([1 << 16] * 2, [1 << 20] * 2, NS[:1])
    assert ei.value.status == capi.FSDP_E_UNSUPPORTED
