"""The host code of the FP8 linear, the rotary positions, the Q/K norms and the
QKV entries built with AddressSanitizer and UndefinedBehaviorSanitizer on the
host side only, linked with the unchanged kernel objects, and driven on the CPU
by tests/sanitize_operators.c: sizing and validation over extents up to
INT64_MAX."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang")
KERNELS = ("gemm_i8", "rotquant", "probes", "fp8", "gemm_fp8", "norm_rope")


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="no ROCm")
def test_operators_host_code_under_asan_ubsan(tmp_path):
    from w8a8_int8_rotated_amd import build as hb
    kernels = [os.path.join(ROOT, "_build", f + ".hip.o") for f in KERNELS]
    if not all(os.path.exists(k) for k in kernels):
        pytest.fail("kernel objects not built (run __graft_entry__.build())")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]

    def run(*cmd, **kw):
        r = subprocess.run(cmd, capture_output=True, text=True, **kw)
        assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
        return r.stdout

    api, lib, exe = (str(tmp_path / f) for f in ("api.o", "libconvrot.so", "sanitize_operators"))
    run(HIPCC, *[f for f in hb.COMMON if f != "-O3"], "-O1", "-g", *san, "-c",
        os.path.join(ROOT, "w8a8_int8_rotated_amd", "csrc", "convrot_api.hip"), "-o", api)
    # (a host link: the kernels are in the objects already)
    run(CLANG + "++", "-shared", "-fPIC", "-fsanitize=address,undefined", api, *kernels,
        f"-L{ROCM}/lib", "-lamdhip64", "-o", lib)
    run(CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined",
        "-fno-sanitize-recover=all", f"-I{ROOT}/include",
        os.path.join(ROOT, "tests", "sanitize_operators.c"), lib, f"-Wl,-rpath,{tmp_path}",
        f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe)
    # the HIP runtime keeps allocations for the life of the process
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    out = run(exe, env=env, timeout=300)
    assert " 0 failed checks" in out
