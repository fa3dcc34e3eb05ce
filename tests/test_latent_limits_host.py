"""The largest calls of attention over latent rows, as include/cfa.h states them."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_units_of_a_call(tmp_path):
    from out_proj_block_gb300 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    exe = str(tmp_path / "limits")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "out_proj_block_gb300", "csrc"), "-I", cuda,
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "latent_limits_check.cpp"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
