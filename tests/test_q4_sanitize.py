"""The host code of the 4-bit layer calls under AddressSanitizer and
UndefinedBehaviorSanitizer (host side only), driven by
tests/sanitize/q4_check.cpp on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "two_sided_hessian_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANGXX = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(CLANGXX), reason="ROCm toolchain not found")
def test_q4_host_paths_under_asan_ubsan(tmp_path):
    objs, procs = [], []
    for f in sorted(f for f in os.listdir(CSRC) if f.startswith("q4") and f.endswith(".hip")):
        objs.append(str(tmp_path / f.replace(".hip", ".o")))
        procs.append((f, subprocess.Popen(
            [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xarch_host", "-fsanitize=address,undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, f), "-o", objs[-1]],
            stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for f, p in procs:
        out = p.communicate()[0]
        assert p.returncode == 0, f"{f}\n{out[-4000:]}"

    def run(cmd, **kw):
        r = subprocess.run(cmd, cwd=str(tmp_path), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
        assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-4000:]}"
        return r.stdout
    drv, exe = str(tmp_path / "q4_check.o"), str(tmp_path / "q4_check")
    run([CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=all", "-c", os.path.join(SAN, "q4_check.cpp"), "-o", drv])
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address,undefined", drv] + objs + ["-o", exe])
    out = run([exe], timeout=300, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                                           UBSAN_OPTIONS="print_stacktrace=1"))
    assert "Q4 SANITIZE OK" in out
