"""The host code of the block-scaled e4m3 and routing entry points -- argument
checks, choice of kernel, shape and grid -- under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, no GPU): built with hipcc and driven by
tests/sanitize/experts_host_check.cpp over a grid of shapes; no call there reaches
a kernel launch.  Any sanitizer report aborts the driver."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_experts_host_paths_under_asan_ubsan(tmp_path):
    hipcc = "/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else shutil.which("hipcc")
    if hipcc is None:
        pytest.skip("hipcc not found")
    exe, csrc = str(tmp_path / "experts_host_check"), os.path.join(ROOT, "precision_integer_gemm_amd", "csrc")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-ffp-contract=off", "-I", os.path.join(ROOT, "include"), "-I", csrc]
    sources = [os.path.join(ROOT, "tests", "sanitize", "experts_host_check.cpp"), os.path.join(csrc, "fp8_block_api.hip"),
               os.path.join(csrc, "routing_api.hip")]
    jobs = [subprocess.Popen([hipcc, *flags, "-c", "-o", f"{exe}{i}.o", s], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            for i, s in enumerate(sources)]
    for job in jobs:
        out, _ = job.communicate(timeout=900)
        assert job.returncode == 0, out
    p = subprocess.run([hipcc, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-o", exe,
                        *[f"{exe}{i}.o" for i in range(len(sources))]], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert p.returncode == 0, (p.stdout + p.stderr)[-4000:]
    assert "all checks passed" in p.stdout
