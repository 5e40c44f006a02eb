"""Compiles the host check of the large products' plans with nvcc and runs it (no GPU needed)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def test_plans_exist_for_every_count_of_rows_and_segments(tmp_path):
    exe = str(tmp_path / "plans_check")
    csrc = os.path.join(ROOT, "segmented_gather_gemm_expand_b200", "csrc")
    r = subprocess.run([NVCC, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_100a,code=sm_100a",
                        "-I", os.path.join(ROOT, "include"), "-I", csrc, "-o", exe, os.path.join(ROOT, "tests", "plans_check.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
