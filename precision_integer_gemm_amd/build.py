"""Ahead-of-time build of the HIP library for gfx950 (MI355X).

    python -m precision_integer_gemm_amd.build

compiles csrc/lpgemm_api.hip (which includes every integer and unscaled fp8
kernel), csrc/mxfp4_api.hip (the microscaled 4-bit kernels),
csrc/fp8_block_api.hip (e4m3 with block scales) and csrc/routing_api.hip
(experts' routing) with hipcc into precision_integer_gemm_amd/_lpgemm.so, next
to this file, and the measurement probe csrc/ceiling_probe.hip into _ceiling.so
(loaded only by bench.py).  These need hipcc alone.  Where PyTorch for ROCm,
Python's headers and g++ are there, csrc/tensor_calls.cpp becomes the Python
module _tensor_calls.so, the short way of the float operators' tensor calls;
without it they take their longer way.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "lpgemm_api.hip")
MX_SRC = os.path.join(PKG, "csrc", "mxfp4_api.hip")
F8_SRC = os.path.join(PKG, "csrc", "fp8_block_api.hip")
ROUTE_SRC = os.path.join(PKG, "csrc", "routing_api.hip")
LIB = os.path.join(PKG, "_lpgemm.so")
CALLS_SRC = os.path.join(PKG, "csrc", "tensor_calls.cpp")
CALLS_LIB = os.path.join(PKG, "_tensor_calls.so")
PROBE_SRC = os.path.join(PKG, "csrc", "ceiling_probe.hip")
PROBE_LIB = os.path.join(PKG, "_ceiling.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the HIP library needs ROCm's hipcc")


def command(out: str, src: str, *mode: str) -> list[str]:
    return [
        hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", *mode, "-fPIC",
        # packed fp32 VALU forms are kept out of the generated code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        # the scaled epilogue's roundings are part of its definition: no
        # contraction of a multiply into a fused operation
        "-ffp-contract=off",
        "-Wall", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"),
        "-o", out, src,
    ]


def calls_missing() -> str | None:
    """What the Python module of the tensor calls cannot be built without and is not there."""
    import sysconfig
    try:
        import torch
    except ImportError:
        return "PyTorch"
    if torch.version.hip is None:
        return "PyTorch for ROCm"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None if shutil.which("g++") else "g++"


def calls_commands(obj: str, out: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of the Python module of the tensor calls: host
    code against PyTorch's headers, linked to the library beside it."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    headers = (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(rocm, "include"))
    return ([
        "g++", "-O2", "-std=c++17", "-c", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
        *(x for h in headers for x in ("-isystem", h)), "-o", obj, CALLS_SRC,
    ], [
        "g++", "-shared", "-o", out, obj, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip",
        "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
    ])


def run(cmd: list[str], what: str, verbose: bool) -> None:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = [l for l in (proc.stdout + proc.stderr).splitlines() if noise not in l]
    if proc.returncode != 0:
        raise RuntimeError(f"compiling {what} failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


def build(verbose: bool = False) -> str:
    objects = [LIB + "." + os.path.basename(src) + ".o" for src in (SRC, F8_SRC)]
    jobs = [(command(o, src, "-c"), os.path.basename(src)) for o, src in zip(objects, (SRC, F8_SRC))]
    jobs.append((command(PROBE_LIB + ".tmp", PROBE_SRC, "-shared"), os.path.basename(PROBE_SRC)))
    missing, calls_obj = calls_missing(), CALLS_LIB + ".o"
    with ThreadPoolExecutor(len(jobs) + 1) as pool:
        if missing is None:
            calls_compile, calls_link = calls_commands(calls_obj, CALLS_LIB + ".tmp")
            calls = pool.submit(run, calls_compile, os.path.basename(CALLS_SRC), verbose)
        for done in [pool.submit(run, cmd, what, verbose) for cmd, what in jobs]:
            done.result()
    # the remaining sources are compiled by the command that links; the objects come
    # first, since hipcc takes what follows a source for sources too
    run([*command(LIB + ".tmp", "", "-shared")[:-1], *objects, MX_SRC, ROUTE_SRC], "the library", verbose)
    os.replace(PROBE_LIB + ".tmp", PROBE_LIB)
    os.replace(LIB + ".tmp", LIB)
    for o in objects:
        os.remove(o)
    if missing is not None:
        if os.path.exists(CALLS_LIB):  # of another library
            os.remove(CALLS_LIB)
        print(f"{os.path.basename(CALLS_LIB)} is not built ({missing} is missing): the microscaled tensor calls take their longer way")
        return LIB
    calls.result()
    run(calls_link, "the tensor calls", verbose)
    os.replace(CALLS_LIB + ".tmp", CALLS_LIB)
    os.remove(calls_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
