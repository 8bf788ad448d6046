"""What the host code hands to the kernels, without a GPU.

The sources are compiled for the host alone, against a stand-in HIP runtime
(tests/launch_driver.cpp) that looks at every launch instead of running it,
with AddressSanitizer and UndefinedBehaviorSanitizer, and with uninitialised
variables filled with a pattern (-ftrivial-auto-var-init) that must reach no
kernel. The driver calls the layer and the feed-forward operators over shapes,
formats and forced paths, the feed-forward operators with arguments that they
refuse, and their size queries over the ends of the ranges.
"""

import os
import re
import subprocess

import pytest

import lora_fine_tuning_amd as L
from test_abi_sanitized import CSRC, ROOT, _tools

TESTS = os.path.join(ROOT, "tests")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    hipcc, _, rt = _tools()
    exe = str(tmp_path_factory.mktemp("launch") / "launch_driver")
    cmd = [hipcc, "-x", "hip", "--offload-host-only", "-fuse-cuid=none", "-no-hip-rt", "-O0", "-g", "-std=c++17",
           "-Xarch_host", "-ftrivial-auto-var-init=pattern", "-Xarch_host", "-fsanitize=address",
           "-Xarch_host", "-fsanitize=undefined", "-shared-libsan",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(TESTS, "launch_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    return exe, rt


def test_every_launch_gets_whole_parameters(driver):
    exe, rt = driver
    env = {k: v for k, v in os.environ.items() if not k.startswith("LORA4_")}
    env["LD_LIBRARY_PATH"] = rt + (":" + env["LD_LIBRARY_PATH"] if env.get("LD_LIBRARY_PATH") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0 and res.stdout.strip().endswith("ok"), res.stdout[-3000:] + res.stderr[-3000:]
    # the feed-forward kernels were all launched, the joint base of two projections among them
    for k in ("k_gemm_fwd_epi", "k_gemm_fwd_split", "k_epi_reduce", "k_small", "k_small_z", "k_act_dz", "k_col_part",
              "k_col_sum_slots", "k_gemm_dgrad", "k_gemm_nn", "k_gemm_tn2", "k_rmsnorm_fwd", "k_rmsnorm_bwd"):
        assert re.search(r"\d%s" % k, res.stdout), k


def test_every_entry_point_runs_under_sanitizers():
    """Each exported name is called by one of the two sanitized drivers."""
    calls = ""
    for name in ("abi_driver.c", "launch_driver.cpp"):
        with open(os.path.join(TESTS, name)) as f:
            calls += re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)
    assert [e for e in L.EXPORTS if not re.search(r"\b%s\(" % e, calls)] == []
