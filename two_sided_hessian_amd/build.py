"""Build libbakron.so in-tree with hipcc for gfx950.

Each .hip file under csrc/ is compiled separately (in parallel) into
_build/ and linked into two_sided_hessian_amd/libbakron.so.  fast_calls.cpp
becomes two_sided_hessian_amd/_fast.so beside it, a Python module that calls
the library (host code only, torch's headers).  The library needs neither torch nor
that module: where it cannot be built, the build says so and goes on without it.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libbakron.so")
FAST = os.path.join(HERE, "_fast.so")
SOURCES = ["factor.hip", "solve.hip", "gptq.hip", "kfac.hip", "antidiag.hip", "capi.hip", "noalloc.hip",
           "q4.hip", "q4_prompt.hip", "q4_grad.hip", "q4_moe.hip", "q4_experts.hip",
           "moe_route.hip", "moe_rows.hip", "moe_gated.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # IEEE-correct fp32 division: the rounding decision x = w / s + z must be
    # reproducible bit for bit.
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    # no packed fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def fast_command(out: str) -> list:
    """The compiler's command line for fast_calls.cpp."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_path("include"), os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), "/opt/rocm/include"]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{p}" for p in include), os.path.join(CSRC, "fast_calls.cpp"), "-o", out, "-L" + os.path.join(root, "lib"),
            "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-ldl"]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for s in SOURCES:
        obj = os.path.join(BUILD, s.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [HIPCC] + FLAGS + ["-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, s), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    fast, fast_proc, why = FAST + ".tmp%d" % os.getpid(), None, ""
    try:
        fast_proc = subprocess.Popen(fast_command(fast), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except (ImportError, OSError) as e:   # no torch, or no host compiler
        why = str(e)
    failed = []
    for s, p in procs:
        out = p.communicate()[0].decode(errors="replace")
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
        if p.returncode != 0:
            failed.append((s, out))
        elif verbose and out.strip():
            print(out)
    if fast_proc is not None:
        why = fast_proc.communicate()[0].decode(errors="replace")
    if failed:
        if os.path.exists(fast):
            os.remove(fast)
        raise RuntimeError("hipcc failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    if fast_proc is not None and fast_proc.returncode == 0:
        os.replace(fast, FAST)
    else:
        for left in (fast, FAST):   # one of another build's might not fit this library
            if os.path.exists(left):
                os.remove(left)
        print(f"{os.path.basename(FAST)} is not built, its calls go through ctypes:\n{why}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
