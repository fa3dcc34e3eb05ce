"""Latent-cache entry points without a GPU: argument checks that come before any device call, how the
attention is cut, and the oracle against closed forms."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cfa_oracle_latent as ref
from oracle import cfa_oracle_paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from out_proj_block_gb300 import build
    build.build()
    from out_proj_block_gb300 import cfa
    return cfa


@pytest.mark.parametrize("args,code", [
    ((0, 1, 32, 64), 1),                  # no requests
    ((1, 0, 32, 64), 1),                  # no tokens
    ((1, 1, 0, 64), 1),
    ((1, 1, 32, 0), 1),
    ((1, 1, 32, 8), 2),                   # page sizes
    ((1, 1, 32, 48), 2),
    ((1, 1, 32, 100), 2),
    ((1, 1, 32, (1 << 22) + 64), 2),
    ((1025, 1, 32, 64), 2),
    ((1, (1 << 17) + 1, 32, 64), 2),
    ((1, 1, 1025, 64), 2),
])
def test_create_rejects_bad_shapes(lib, args, code):
    assert lib._lib.cfa_latent_create(*args) is None
    assert lib.cfa_last_error() == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")
def test_create_without_gpu_reports_cuda_error(lib):
    assert lib._lib.cfa_latent_create(4, 4, 8, 64) is None
    assert lib.cfa_last_error() == lib.CFA_ERR_CUDA


def test_calls_reject_a_null_plan(lib):
    L, p, bad = lib._lib, ctypes.c_void_p(256), lib.CFA_ERR_INVALID_ARG
    assert L.cfa_latent_set_rope(None, 1e4, 0, 0, 1.0, 1.0, 32.0, 4096, 1.0) == bad
    assert L.cfa_latent_append(None, 1, p, 576, p, 1e-6, p, 192, p, p, 1, p, p, None) == bad
    assert L.cfa_latent_fold(None, 1, p, 192, p, p, None) == bad
    assert L.cfa_latent_unfold(None, 1, p, p, p, None) == bad
    assert L.cfa_latent_attention(None, 1, 1, p, p, p, 1, p, 1, p, 0.0, p, None, None) == bad
    assert L.cfa_latent_expanded(None, 1, 1, 1, p, 192, p, 256, p, 64, p, p, 0.0, p, None, None) == bad
    assert L.cfa_latent_layer(None, 1, 1, p, 576, p, 1e-6, p, 192, p, p, p, p, 1, p, 1, p, p, 0.0, p, p, p,
                              None, p, None) == bad
    assert L.cfa_latent_status(None) == bad
    buf = ctypes.create_string_buffer(64)
    assert L.cfa_latent_describe(None, buf, 64) == bad
    L.cfa_latent_destroy(None)  # no-op


def run_check(tmp_path, name, *args, timeout=120):
    """Compiles tests/<name>.cpp with the host compiler and runs it with these arguments."""
    from out_proj_block_gb300 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    exe = str(tmp_path / name)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "out_proj_block_gb300", "csrc"), "-I", cuda,
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe],
                   check=True)
    out = subprocess.run([exe, *args], capture_output=True, text=True, timeout=timeout)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


@pytest.mark.parametrize("check", ["overlaps", "ranges", "order", "bytes", "forms"])
def test_calls(tmp_path, check):
    run_check(tmp_path, "latent_calls_check", check)


def test_split_covers_every_block_once(tmp_path):
    run_check(tmp_path, "latent_split_check")


# ------------------------------------------------------------------ oracle pins


def test_oracle_rows():
    a = np.zeros((2, 576))
    a[0, :512], a[1, 3] = 2.0, 5.0
    a[:, 512] = 1.0
    g = np.arange(512.0)
    rows = ref.rows(a, g, 0.0, [0, 7], cfa_oracle_paged.frequencies(10000.0, 64))
    assert np.allclose(rows[0, :512], g) and rows[1, 3] == pytest.approx(3.0 * math.sqrt(512.0))
    assert np.array_equal(rows[0, 512:], a[0, 512:])
    assert rows[1, 512] == pytest.approx(math.cos(7.0)) and rows[1, 544] == pytest.approx(math.sin(7.0))


def test_oracle_forms_are_one():
    """Folding the queries, attending over the rows and folding back is attention over expanded
    keys and values."""
    rng = np.random.default_rng(1)
    H, n, L = 3, 4, 9
    W = rng.standard_normal((512, H * 256)) / 20
    q, rows = rng.standard_normal((n, H, 192)), rng.standard_normal((L, 576))
    kv = (rows[:, :512] @ W).reshape(L, H, 256)
    q_lat, _ = ref.fold(q, W)
    o, lse, _ = ref.attention(q_lat, [0, n], [L], [[0]], rows[None])
    out, _ = ref.unfold(o, W)
    want, wl, _ = ref.expanded(q, kv, rows[:, 512:], [0, n], [0, L])
    assert np.allclose(out, want) and np.allclose(lse, wl)


def test_oracle_rows_not_seen():
    rng = np.random.default_rng(2)
    rows, q = rng.standard_normal((1, 16, 576)), rng.standard_normal((5, 2, 576))
    out, lse, _ = ref.attention(q, [0, 5], [2], [[0]], rows)
    assert not out[:3].any() and np.all(lse[:3] == -math.inf)
    assert np.allclose(out[3], rows[0, 0, :512]) and np.isfinite(out[4]).all()
