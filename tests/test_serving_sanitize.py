"""The serving calls' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitize.py does it for the solve: the
library's host code with the sanitizers, linked with a driver
(serving_sanitize_driver.cpp) whose calls all return before a launch.  CPU only."""
import os
import subprocess

import pytest

from test_abi_sanitize import ROOT, SAN, _tool


@pytest.mark.timeout(900)
def test_serving_host_code_under_sanitizers(tmp_path):
    from post_weight_quantization_07_amd import build as B
    hipcc, clangxx = _tool("hipcc"), _tool("clang++")
    if hipcc is None or clangxx is None:
        pytest.skip("hipcc / clang++ not available")
    flags = ["-O1", "-g", "-std=c++17", "-fPIC", f"--offload-arch={B.ARCH}", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", B.CSRC] + SAN
    jobs, objs = [], []
    for path in [os.path.join(B.CSRC, s) for s in B.SOURCES] + [os.path.join(ROOT, "tests", "serving_sanitize_driver.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(path) + ".o")))
        cmd = [hipcc, "-x", "hip", *flags, "-c", path, "-o", objs[-1]]
        jobs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for cmd, pr in jobs:
        out, _ = pr.communicate()
        assert pr.returncode == 0, f"{' '.join(cmd)}\n{out[-3000:]}"
    exe = str(tmp_path / "serving_sanitize")
    link = [clangxx, "-fsanitize=address,undefined", "-fno-sanitize-recover=all", *objs, "-o", exe,
            "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(link, capture_output=True, text=True)
    assert r.returncode == 0, f"{' '.join(link)}\n{r.stdout}\n{r.stderr}"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "all checks passed" in r.stdout and "runtime error" not in r.stderr
