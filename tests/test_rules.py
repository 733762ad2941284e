"""The rules by which the library chooses among kernels with equal results, asked of the library
itself (built into a small program) on the CPU, on both sides of their borders."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang++")
OBJECTS = ("convrot_api", "layer_api", "gemm_i8", "rotquant", "probes", "fp8", "gemm_fp8",
           "norm_rope", "add_norm", "moe")


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("no ROCm")
    objs = [os.path.join(ROOT, "_build", f + ".hip.o") for f in OBJECTS]
    if not all(os.path.exists(o) for o in objs):
        pytest.fail("kernel objects not built (run __graft_entry__.build())")
    exe = str(tmp_path_factory.mktemp("rules") / "rules")
    r = subprocess.run([CLANG, "-O1", os.path.join(ROOT, "tests", "rules.cpp"), *objs,
                        f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(*questions):
        r = subprocess.run([exe], input="\n".join(questions), capture_output=True, text=True,
                           timeout=60)
        assert r.returncode == 0
        return [int(v) for v in r.stdout.split()]
    return ask


def test_own_choice(ask):
    """Experts' workgroups choose for themselves up to one round of three a CU, one token's too."""
    assert ask("own 1 384", "own 1 768", "own 4 768") == [1, 1, 1]
    assert ask("own 1 769", "own 1 4096", "own 2 1792", "own 4 769", "own 5 16") == [0] * 5


def test_few_rows(ask):
    """The INT8 product's kernel for few rows: any N up to 16 rows, to 2^20 up to 32, to 96 a CU up
    to 64."""
    assert ask("few 1 16", "few 16 4194304", "few 17 1048576", "few 32 1048576",
               "few 33 24576", "few 64 24576") == [1] * 6
    assert ask("few 17 1048592", "few 32 4194304", "few 33 24592", "few 64 32768",
               "few 65 16") == [0] * 5
