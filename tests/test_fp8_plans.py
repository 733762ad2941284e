"""The shapes that the GPU tests of the FP8 product run cover every kernel shape and
both kinds of launch plan, for either output type: the plans themselves, asked of the
library's own chooser (built into a small program) on the CPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CLANG = os.path.join(ROCM, "llvm", "bin", "clang++")
OBJECTS = ("convrot_api", "gemm_i8", "rotquant", "probes", "fp8", "gemm_fp8", "norm_rope")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("no ROCm")
    objs = [os.path.join(ROOT, "_build", f + ".hip.o") for f in OBJECTS]
    if not all(os.path.exists(o) for o in objs):
        pytest.fail("kernel objects not built (run __graft_entry__.build())")
    exe = str(tmp_path_factory.mktemp("plans") / "fp8_plans")
    r = subprocess.run([CLANG, "-O1", os.path.join(ROOT, "tests", "fp8_plans.cpp"), *objs,
                        f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(shapes, f32):
        text = "".join(f"{M} {K} {N} {int(f32)} {int(M <= 16)}\n" for M, K, N in shapes)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        lines = [tuple(ln.split()) for ln in r.stdout.splitlines()]
        assert len(lines) == len(shapes)
        return [(ln[0], *map(int, ln[1:])) for ln in lines]
    return ask


def test_few_rows_cover_every_width(plan):
    from test_gpu_fp8 import FEW_ROWS, SHAPES
    few = [(M, K, N) for M in (1, 8, 16) for K, N in FEW_ROWS] + [s for s in SHAPES if s[0] <= 16]
    for f32 in (False, True):
        got = plan(few, f32)
        assert {p[:2] for p in got} == {("few", 1), ("few", 2), ("few", 4)}
        # row blocks that the workgroup's tiles do not divide
        for rt in (2, 4):
            assert any(p[1] == rt and N // 16 % rt for p, (_, _, N) in zip(got, few))


def test_plans_cover_every_kernel(plan):
    from test_gpu_fp8 import PLANS, SHAPES, TAILS
    shapes = [s for s in (*SHAPES, *PLANS, *TAILS) if s[0] > 16]
    for f32 in (False, True):
        got = plan(shapes, f32)
        few = {p[1:] for p in got if p[0] == "few"}
        assert few == {(1, 1), (2, 1), (2, 2), (2, 4)}
        alone = {p[1:3] for p in got if p[0] == "tiles" and p[3] == 0}
        tails = {p[1:3] for p in got if p[0] == "tiles" and p[3] > 0}
        if f32:
            assert alone == {(128, 256), (128, 128), (128, 64)}
            assert tails == {(128, 128), (128, 64)}
        else:
            assert alone == {(256, 256), (256, 128), (128, 256), (256, 64), (128, 128), (128, 64)}
            assert tails == {(256, 128), (128, 256), (256, 64), (128, 128), (128, 64)}


def test_plans_are_whole(plan):
    """A first launch holds whole rows of the largest tiles and leaves some."""
    shapes = [(M, K, N) for M in (17, 333, 1024, 4096, 4133, 38656, 38657, 1 << 20)
              for N in (16, 272, 5376, 16128, 32768) for K in (128, 640, 5376)
              if M * K < 1 << 31]
    for f32 in (False, True):
        for s, p in zip(shapes, plan(shapes, f32)):
            if p[0] == "tiles":
                assert p[3] % 256 == 0 and p[3] < s[0], (s, p)
            else:
                assert p[1] in (1, 2) and p[2] in (1, 2, 4), (s, p)
