"""The row and MXFP4 operators from C: ``tests/c/rows_check.c`` as strict C99 and as
C++17 (warnings are errors), linked with the built library and run without a GPU."""
import os
import shutil
import subprocess

import pytest

from moe_expert_ffn_permute_b200.build import LIB, build

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))


@pytest.mark.parametrize("compiler,flags", [("gcc", ["-std=c99", "-pedantic"]),
                                            ("g++", ["-x", "c++", "-std=c++17"])], ids=["c99", "c++17"])
def test_c_program_against_the_header(tmp_path, compiler, flags):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not installed")
    build()
    exe, pkg = str(tmp_path / "rows_check"), os.path.dirname(LIB)
    r = subprocess.run([compiler, *flags, "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "rows_check.c"),
                        "-L", pkg, "-lmoe_b200", f"-Wl,-rpath,{pkg}", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip().endswith("abi ok"), r.stdout + r.stderr
