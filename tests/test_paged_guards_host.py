"""What the paged-cache operators make of values out of range, without a GPU: the rules that
their kernels share with the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cuda_include():
    from out_proj_block_gb300 import build
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")


def run_check(tmp_path, name, *args, timeout=120):
    """Compiles tests/<name>.cpp with the host compiler and runs it with these arguments."""
    exe = str(tmp_path / name)
    csrc = os.path.join(ROOT, "out_proj_block_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", csrc, "-I", cuda_include(), "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe], check=True)
    out = subprocess.run([exe, *args], capture_output=True, text=True, timeout=timeout)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_refused_batches_and_pools(tmp_path):
    run_check(tmp_path, "paged_guards_check")


def test_layer_refuses_writing_over_what_it_reads(tmp_path):
    run_check(tmp_path, "paged_calls_check", "overlaps")


def test_words_are_cleared_before_the_call_returns(tmp_path):
    run_check(tmp_path, "paged_calls_check", "order")


def test_scales_that_pass_32_bits(tmp_path):
    run_check(tmp_path, "paged_calls_check", "scales")


def test_walk_through_long_requests(tmp_path):
    run_check(tmp_path, "paged_walk_check")


def test_describe_counts_every_byte(tmp_path):
    run_check(tmp_path, "paged_calls_check", "bytes")


def test_clocks_of_a_blocks_bytes(tmp_path):
    run_check(tmp_path, "paged_calls_check", "clocks")
