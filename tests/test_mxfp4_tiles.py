"""The product's tile arithmetic without a GPU: ``tests/c/tiles_check.cu``, built with
nvcc from the kernels' own header and run on the host."""
import os
import subprocess

from moe_expert_ffn_permute_b200.build import CSRC, FLAGS, NVCC

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))


def test_tiles_of_groups_of_any_size(tmp_path):
    exe = str(tmp_path / "tiles_check")
    flags = [f for f in FLAGS if f not in ("-Xcompiler", "-fPIC", "-shared")]
    r = subprocess.run([NVCC, *flags, "-I", CSRC, "-o", exe,
                        os.path.join(ROOT, "tests", "c", "tiles_check.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip().endswith("tiles ok"), r.stdout + r.stderr
