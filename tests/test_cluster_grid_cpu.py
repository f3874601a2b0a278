"""How many CTAs a persistent cluster kernel gets: found once per kernel and device, and
never taken from another kernel of the same type."""
import os
import subprocess

from combine_topk_ids_expert_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_grid_is_each_kernels_own(tmp_path):
    exe = str(tmp_path / "cluster_grid")
    # The shared runtime: the program's own definitions come before it.
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "lib64")
    files = [os.path.join(HERE, "c", f) for f in ("cluster_grid.cu", "cluster_grid_runtime.cpp")]
    r = subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "-cudart",
                        "shared", "-Xlinker", f"-rpath={lib}", *files, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
