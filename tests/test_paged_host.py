"""Paged-cache entry points without a GPU: argument checks that come before any
device call, the frequencies and tables of the oracle against closed forms."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cfa_oracle_paged as ref


@pytest.fixture(scope="module")
def lib():
    from out_proj_block_gb300 import build
    build.build()
    from out_proj_block_gb300 import cfa
    return cfa


@pytest.mark.parametrize("args,code", [
    ((0, 1, 32, 8, 128, 64), 1),          # no requests
    ((1, 0, 32, 8, 128, 64), 1),          # no tokens
    ((1, 1, 0, 1, 128, 64), 1),
    ((1, 1, 32, 0, 128, 64), 1),
    ((1, 1, 32, 5, 128, 64), 1),          # heads do not divide
    ((1, 1, 8, 16, 128, 64), 1),          # more key heads than heads
    ((1, 1, 32, 8, 128, 0), 1),
    ((1, 1, 32, 8, 96, 64), 2),           # head_dim
    ((1, 1, 32, 8, 256, 64), 2),
    ((1, 1, 32, 8, 128, 8), 2),           # page sizes
    ((1, 1, 32, 8, 128, 48), 2),
    ((1, 1, 32, 8, 128, 100), 2),
    ((1, 1, 32, 8, 128, (1 << 22) + 64), 2),
    ((1025, 1, 32, 8, 128, 64), 2),
    ((1, (1 << 17) + 1, 32, 8, 128, 64), 2),
    ((1, 1, 2048, 8, 128, 64), 2),
])
def test_create_rejects_bad_shapes(lib, args, code):
    assert lib._lib.cfa_paged_create(*args) is None
    assert lib.cfa_last_error() == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")
def test_create_without_gpu_reports_cuda_error(lib):
    assert lib._lib.cfa_paged_create(4, 4, 8, 2, 128, 64) is None
    assert lib.cfa_last_error() == lib.CFA_ERR_CUDA


def test_calls_reject_a_null_plan(lib):
    L, p = lib._lib, ctypes.c_void_p(256)
    bad = lib.CFA_ERR_INVALID_ARG
    assert L.cfa_paged_set_rope(None, 1e4, 64, 0, 0, 1.0, 1.0, 32.0, 4096, 1.0) == bad
    assert L.cfa_paged_tables(None, 1, 0, p, p, p, 1, p, p, 1, p, p, p, p, p, 1, None) == bad
    assert L.cfa_paged_append(None, 1, p, 128, p, 128, p, 128, p, p, 1, p, p, p, None) == bad
    assert L.cfa_paged_attention(None, 1, 1, p, 128, p, p, 0, p, 1, p, 1, p, p, 0.0, p, None,
                                 None) == bad
    assert L.cfa_paged_layer(None, 1, 1, p, 128, p, 128, p, 128, p, p, p, p, 0, p, 1, p, 1, p, p,
                             0.0, p, p, None, None) == bad
    assert L.cfa_paged_status(None) == bad
    buf = ctypes.create_string_buffer(64)
    assert L.cfa_paged_describe(None, buf, 64) == bad
    L.cfa_paged_destroy(None)  # no-op


def test_no_pages_status_has_a_name(lib):
    assert lib.cfa_status_string(lib.CFA_ERR_NO_PAGES) == "CFA_ERR_NO_PAGES"


# ------------------------------------------------------------------ oracle pins


def test_oracle_tables_by_hand():
    tables = np.full((3, 4), -1, dtype=np.int32)
    tables[0, :1] = [9]
    tables[2, :2] = [4, 5]
    got = ref.build_tables([3, 0, 8], [2, 0, 1], [7, 6, 1, 2], [1, 4], tables, 100, 4, 5)
    ok, t, lens, pool, cu, pos, slots = got
    assert ok and lens == [5, 0, 9] and pool == [3, 4] and cu == [0, 2, 2, 3]
    assert t[0].tolist() == [9, 6, -1, -1] and t[2].tolist() == [4, 5, 1, -1]
    assert pos == [103, 104, 108, 0, 0] and slots == [39, 24, 4, -1, -1]
    assert not ref.build_tables([3, 0, 8], [2, 0, 1], [7, 6], [1, 2], tables, 0, 4, 5)[0]


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 32))
    f = ref.frequencies(10000.0, 16)
    for inter in (False, True):
        y = ref.rotate(x, [0, 5, 1 << 20], f, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[:, :, 16:], x[:, :, 16:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # the two layouts are one rotation in another order of dims
    order = np.arange(32)
    order[:16] = np.arange(16).reshape(2, 8).T.reshape(-1)
    assert np.allclose(ref.rotate(x, [1, 2, 3], f, False)[:, :, order],
                       ref.rotate(x[:, :, order], [1, 2, 3], f, True))


def test_oracle_scaling_limits():
    plain = ref.frequencies(10000.0, 64)
    parts = ref.frequencies(10000.0, 64, "by_parts", 8.0, 1.0, 32.0, 4096)
    turns = [4096 * w / (2 * math.pi) for w in plain]
    for p, w, r in zip(parts, plain, turns):
        if r >= 32:
            assert p == pytest.approx(w)
        elif r <= 1:
            assert p == pytest.approx(w / 8)
        else:
            assert w / 8 < p < w
    assert ref.frequencies(10000.0, 64, "linear", 4.0)[3] == pytest.approx(plain[3] / 4)


def test_oracle_attention_of_equal_keys_is_the_mean():
    k = np.ones((2, 1, 16, 4))
    v = np.arange(2 * 16 * 4, dtype=np.float64).reshape(2, 1, 16, 4)
    q = np.ones((2, 1, 4))
    out, lse, _ = ref.attention(q, [0, 2], [3], [[1]], k, v, [0], 5)
    assert np.allclose(out[1, 0], np.concatenate((v[0, 0, :5], v[1, 0, :3])).mean(0))
    assert np.allclose(out[0, 0], np.concatenate((v[0, 0, :5], v[1, 0, :2])).mean(0))
    assert lse[1, 0] == pytest.approx(2.0 + math.log(8))
    out, lse, _ = ref.attention(q, [0, 2], [1], [[1]], k, v)
    assert np.all(out[0] == 0) and lse[0, 0] == -math.inf and np.allclose(out[1, 0], v[1, 0, 0])


# ------------------------------------------------------------------ how the attention is cut


def test_split_covers_every_block_once(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "paged_split_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(root, "out_proj_block_gb300", "csrc"),
                    os.path.join(root, "tests", "paged_split_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
