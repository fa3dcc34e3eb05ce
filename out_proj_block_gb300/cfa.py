"""Python binding of libcfa.so (see include/cfa.h): same names, argument marshalling only.

Every step of the decode path runs inside the CUDA library. This module only
checks tensor dtypes, devices, shapes and contiguity, turns tensors into
pointers and CUDA streams into handles, and maps status codes to exceptions.
Importing it raises ImportError if the library has not been built; there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes
import json
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcfa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with out_proj_block_gb300.build.build() "
        "(nvcc, sm_103a). There is no fallback path.")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i = ctypes.c_int

_lib.cfa_plan_create.restype = _vp
_lib.cfa_plan_create.argtypes = [_i, _i, _i, _i, _i]
_lib.cfa_plan_destroy.restype = None
_lib.cfa_plan_destroy.argtypes = [_vp]
_lib.cfa_decode_step.restype = _i
_lib.cfa_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]
_lib.cfa_decode_step_ex.restype = _i
_lib.cfa_decode_step_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(ctypes.c_int),
                                    ctypes.c_double, _vp, _vp]
_lib.cfa_decode_step_host.restype = _i
_lib.cfa_decode_step_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]
_lib.cfa_decode_step_noalloc.restype = _i
_lib.cfa_decode_step_noalloc.argtypes = [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]
_lib.cfa_plan_set_cluster_size.restype = _i
_lib.cfa_plan_set_cluster_size.argtypes = [_vp, _i]
_lib.cfa_plan_set_stages.restype = _i
_lib.cfa_plan_set_stages.argtypes = [_vp, _i]
_lib.cfa_plan_set_overlap.restype = _i
_lib.cfa_plan_set_overlap.argtypes = [_vp, _i]
_lib.cfa_plan_set_qkv_exchange.restype = _i
_lib.cfa_plan_set_qkv_exchange.argtypes = [_vp, _i]
_lib.cfa_plan_cluster_size.restype = _i
_lib.cfa_plan_cluster_size.argtypes = [_vp]
_lib.cfa_plan_describe.restype = _i
_lib.cfa_plan_describe.argtypes = [_vp, ctypes.c_char_p, _i]
_lib.cfa_plan_status.restype = _i
_lib.cfa_plan_status.argtypes = [_vp]
_lib.cfa_last_error.restype = _i
_lib.cfa_last_error.argtypes = []
_lib.cfa_status_string.restype = ctypes.c_char_p
_lib.cfa_status_string.argtypes = [_i]
_lib.cfa_selftest_wait_timeout.restype = _i
_lib.cfa_selftest_wait_timeout.argtypes = [_i, _vp]
_lib.cfa_rmsnorm.restype = _i
_lib.cfa_rmsnorm.argtypes = [_i, _i, _vp, _vp, ctypes.c_float, _vp, _vp]
_lib.cfa_mlp_create.restype = _vp
_lib.cfa_mlp_create.argtypes = [_i, _i, _i]
_lib.cfa_mlp_destroy.restype = None
_lib.cfa_mlp_destroy.argtypes = [_vp]
_lib.cfa_mlp_step.restype = _i
_lib.cfa_mlp_step.argtypes = [_vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp]
_lib.cfa_mlp_set_pipeline.restype = _i
_lib.cfa_mlp_set_pipeline.argtypes = [_vp, _i, _i]
_lib.cfa_mlp_set_path.restype = _i
_lib.cfa_mlp_set_path.argtypes = [_vp, _i]
_lib.cfa_mlp_status.restype = _i
_lib.cfa_mlp_status.argtypes = [_vp]
_lib.cfa_mlp_describe.restype = _i
_lib.cfa_mlp_describe.argtypes = [_vp, ctypes.c_char_p, _i]
_lib.cfa_stack_create.restype = _vp
_lib.cfa_stack_create.argtypes = [_i] * 7
_lib.cfa_stack_destroy.restype = None
_lib.cfa_stack_destroy.argtypes = [_vp]
_lib.cfa_stack_set_layer.restype = _i
_lib.cfa_stack_set_layer.argtypes = [_vp, _i] + [_vp] * 9
_lib.cfa_stack_step.restype = _i
_lib.cfa_stack_step.argtypes = [_vp, _vp, _vp, ctypes.c_double, ctypes.c_float, _i, _vp, _vp]
_lib.cfa_stack_step_graph.restype = _i
_lib.cfa_stack_step_graph.argtypes = [_vp, _vp, _vp, ctypes.c_double, ctypes.c_float, _i, _vp,
                                      _vp]
_lib.cfa_stack_status.restype = _i
_lib.cfa_stack_status.argtypes = [_vp]
_lib.cfa_mla_create.restype = _vp
_lib.cfa_mla_create.argtypes = [_i] * 5
_lib.cfa_mla_destroy.restype = None
_lib.cfa_mla_destroy.argtypes = [_vp]
_lib.cfa_mla_step.restype = _i
_lib.cfa_mla_step.argtypes = ([_vp] * 9 + [ctypes.POINTER(ctypes.c_int), ctypes.c_double,
                                           ctypes.c_float, _vp, _vp])
_lib.cfa_mla_status.restype = _i
_lib.cfa_mla_status.argtypes = [_vp]
_lib.cfa_mla_describe.restype = _i
_lib.cfa_mla_describe.argtypes = [_vp, ctypes.c_char_p, _i]
_lib.cfa_mla_set_row_splits.restype = _i
_lib.cfa_mla_set_row_splits.argtypes = [_vp, _i]
_lib.cfa_stack_describe.restype = _i
_lib.cfa_stack_describe.argtypes = [_vp, ctypes.c_char_p, _i]
_lib.cfa_plan_layout.restype = _i
_lib.cfa_plan_layout.argtypes = [_i] * 12 + [ctypes.c_char_p, _i]

_lib.cfa_paged_create.restype = _vp
_lib.cfa_paged_create.argtypes = [_i] * 6
_lib.cfa_paged_destroy.restype = None
_lib.cfa_paged_destroy.argtypes = [_vp]
_lib.cfa_paged_set_rope.restype = _i
_lib.cfa_paged_set_rope.argtypes = [_vp, ctypes.c_double, _i, _i, _i, ctypes.c_double,
                                    ctypes.c_double, ctypes.c_double, _i, ctypes.c_double]
_ll = ctypes.c_longlong
_lib.cfa_paged_tables.restype = _i
_lib.cfa_paged_tables.argtypes = ([_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _i] + [_vp] * 5
                                  + [_i, _vp])
_lib.cfa_paged_append.restype = _i
_lib.cfa_paged_append.argtypes = [_vp, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _i, _vp, _vp,
                                  _vp, _vp]
_lib.cfa_paged_attention.restype = _i
_lib.cfa_paged_attention.argtypes = [_vp, _i, _i, _vp, _ll, _vp, _vp, _i, _vp, _i, _vp, _i, _vp,
                                     _vp, ctypes.c_float, _vp, _vp, _vp]
_lib.cfa_paged_layer.restype = _i
_lib.cfa_paged_layer.argtypes = [_vp, _i, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp,
                                 _i, _vp, _i, _vp, _i, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp]
_lib.cfa_paged_status.restype = _i
_lib.cfa_paged_status.argtypes = [_vp]
_lib.cfa_paged_describe.restype = _i
_lib.cfa_paged_describe.argtypes = [_vp, ctypes.c_char_p, _i]

_lib.cfa_latent_create.restype = _vp
_lib.cfa_latent_create.argtypes = [_i] * 4
_lib.cfa_latent_destroy.restype = None
_lib.cfa_latent_destroy.argtypes = [_vp]
_lib.cfa_latent_set_rope.restype = _i
_lib.cfa_latent_set_rope.argtypes = [_vp, ctypes.c_double, _i, _i, ctypes.c_double, ctypes.c_double,
                                     ctypes.c_double, _i, ctypes.c_double]
_lib.cfa_latent_append.restype = _i
_lib.cfa_latent_append.argtypes = [_vp, _i, _vp, _ll, _vp, ctypes.c_float, _vp, _ll, _vp, _vp, _i, _vp,
                                   _vp, _vp]
_lib.cfa_latent_fold.restype = _i
_lib.cfa_latent_fold.argtypes = [_vp, _i, _vp, _ll, _vp, _vp, _vp]
_lib.cfa_latent_unfold.restype = _i
_lib.cfa_latent_unfold.argtypes = [_vp, _i, _vp, _vp, _vp, _vp]
_lib.cfa_latent_attention.restype = _i
_lib.cfa_latent_attention.argtypes = [_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, ctypes.c_float, _vp,
                                      _vp, _vp]
_lib.cfa_latent_expanded.restype = _i
_lib.cfa_latent_expanded.argtypes = [_vp, _i, _i, _i, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp,
                                     ctypes.c_float, _vp, _vp, _vp]
_lib.cfa_latent_layer.restype = _i
_lib.cfa_latent_layer.argtypes = [_vp, _i, _i, _vp, _ll, _vp, ctypes.c_float, _vp, _ll, _vp, _vp, _vp, _vp,
                                  _i, _vp, _i, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.cfa_latent_status.restype = _i
_lib.cfa_latent_status.argtypes = [_vp]
_lib.cfa_latent_describe.restype = _i
_lib.cfa_latent_describe.argtypes = [_vp, ctypes.c_char_p, _i]

CFA_OK = 0
CFA_ERR_INVALID_ARG = 1
CFA_ERR_UNSUPPORTED = 2
CFA_ERR_CUDA = 3
CFA_ERR_TIMEOUT = 4
CFA_ERR_ALIGNMENT = 5
CFA_ERR_NO_PAGES = 6

EXPORTED_SYMBOLS = (
    "cfa_plan_create", "cfa_plan_destroy", "cfa_decode_step", "cfa_decode_step_ex",
    "cfa_decode_step_host",
    "cfa_decode_step_noalloc",
    "cfa_plan_set_cluster_size", "cfa_plan_set_stages", "cfa_plan_set_overlap",
    "cfa_plan_set_qkv_exchange",
    "cfa_plan_cluster_size",
    "cfa_plan_describe", "cfa_plan_layout", "cfa_plan_status", "cfa_last_error",
    "cfa_status_string",
    "cfa_selftest_wait_timeout",
    "cfa_rmsnorm", "cfa_mlp_create", "cfa_mlp_destroy", "cfa_mlp_step", "cfa_mlp_status",
    "cfa_mlp_set_pipeline", "cfa_mlp_set_path",
    "cfa_mlp_describe", "cfa_stack_create", "cfa_stack_destroy", "cfa_stack_set_layer",
    "cfa_stack_step", "cfa_stack_step_graph", "cfa_stack_status", "cfa_stack_describe",
    "cfa_mla_create", "cfa_mla_destroy", "cfa_mla_step", "cfa_mla_status", "cfa_mla_describe",
    "cfa_mla_set_row_splits",
    "cfa_paged_create", "cfa_paged_destroy", "cfa_paged_set_rope", "cfa_paged_tables",
    "cfa_paged_append", "cfa_paged_attention", "cfa_paged_layer", "cfa_paged_status",
    "cfa_paged_describe",
    "cfa_latent_create", "cfa_latent_destroy", "cfa_latent_set_rope", "cfa_latent_append",
    "cfa_latent_fold", "cfa_latent_unfold", "cfa_latent_attention", "cfa_latent_expanded",
    "cfa_latent_layer", "cfa_latent_status", "cfa_latent_describe",
)


class CfaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {cfa_status_string(status)}" if what else cfa_status_string(status))


def cfa_status_string(status: int) -> str:
    return _lib.cfa_status_string(int(status)).decode()


def cfa_last_error() -> int:
    return int(_lib.cfa_last_error())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------- raw C-ABI calls


def cfa_plan_create(B: int, hidden: int, n_heads: int, head_dim: int, max_ctx: int) -> int:
    h = _lib.cfa_plan_create(B, hidden, n_heads, head_dim, max_ctx)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_plan_create")
    return h


def cfa_plan_destroy(plan: int) -> None:
    _lib.cfa_plan_destroy(plan)


def cfa_decode_step(plan, x, W_qkv, W_o, k_cache, v_cache, ctx_len: int, out, stream=None) -> int:
    return int(_lib.cfa_decode_step(plan, _ptr(x), _ptr(W_qkv), _ptr(W_o), _ptr(k_cache),
                                    _ptr(v_cache), int(ctx_len), _ptr(out), _stream(stream)))


def cfa_decode_step_ex(plan, x, W_qkv, W_o, k_cache, v_cache, ctx_lens, rope_theta: float,
                       out, stream=None) -> int:
    lens = (ctypes.c_int * len(ctx_lens))(*[int(v) for v in ctx_lens])
    return int(_lib.cfa_decode_step_ex(plan, _ptr(x), _ptr(W_qkv), _ptr(W_o), _ptr(k_cache),
                                       _ptr(v_cache), lens, float(rope_theta), _ptr(out),
                                       _stream(stream)))


def cfa_decode_step_host(plan, x_host, W_qkv, W_o, k_cache, v_cache, ctx_len: int, out_host,
                         stream=None) -> int:
    return int(_lib.cfa_decode_step_host(plan, _ptr(x_host), _ptr(W_qkv), _ptr(W_o),
                                         _ptr(k_cache), _ptr(v_cache), int(ctx_len),
                                         _ptr(out_host), _stream(stream)))


def cfa_decode_step_noalloc(B: int, hidden: int, n_heads: int, head_dim: int, max_ctx: int,
                            x, W_qkv, W_o, k_cache, v_cache, ctx_len: int, out,
                            stream=None) -> int:
    """The decode step for callers that cannot allocate device memory (see
    include/cfa.h); its scratch is a fixed array inside the library."""
    return int(_lib.cfa_decode_step_noalloc(B, hidden, n_heads, head_dim, max_ctx, _ptr(x),
                                            _ptr(W_qkv), _ptr(W_o), _ptr(k_cache),
                                            _ptr(v_cache), int(ctx_len), _ptr(out),
                                            _stream(stream)))


def cfa_plan_set_cluster_size(plan, C: int) -> int:
    return int(_lib.cfa_plan_set_cluster_size(plan, int(C)))


def cfa_plan_set_stages(plan, stages: int) -> int:
    return int(_lib.cfa_plan_set_stages(plan, int(stages)))


def cfa_plan_set_overlap(plan, enable: bool) -> int:
    return int(_lib.cfa_plan_set_overlap(plan, 1 if enable else 0))


def cfa_plan_set_qkv_exchange(plan, mode: int) -> int:
    return int(_lib.cfa_plan_set_qkv_exchange(plan, int(mode)))


def cfa_plan_cluster_size(plan) -> int:
    return int(_lib.cfa_plan_cluster_size(plan))


def cfa_plan_describe(plan) -> dict:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.cfa_plan_describe(plan, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_plan_describe")
    return json.loads(buf.value.decode())


def cfa_plan_layout(B: int, hidden: int, n_heads: int, head_dim: int, max_ctx: int, C: int,
                    exchange: int, stages: int, num_sms: int, smem_per_sm: int, smem_optin: int,
                    smem_reserved: int):
    """(status, layout dict or None): the layout a plan of this shape would use
    with cluster size C on a device with these limits, computed on the host."""
    buf = ctypes.create_string_buffer(1024)
    st = int(_lib.cfa_plan_layout(B, hidden, n_heads, head_dim, max_ctx, C, exchange, stages,
                                  num_sms, smem_per_sm, smem_optin, smem_reserved, buf,
                                  len(buf)))
    return st, (json.loads(buf.value.decode()) if st == CFA_OK else None)


def cfa_plan_status(plan) -> int:
    return int(_lib.cfa_plan_status(plan))


def cfa_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    return int(_lib.cfa_selftest_wait_timeout(int(limit_us), _stream(stream)))


# ---------------------------------------------------------- tensor-level API


class Plan:
    """Owns a cfa_plan; checks tensors and launches decode steps."""

    def __init__(self, B: int, hidden: int, n_heads: int, head_dim: int, max_ctx: int,
                 cluster_size: Optional[int] = None, stages: Optional[int] = None,
                 overlap: Optional[bool] = None, qkv_exchange: Optional[int] = None):
        self.B, self.hidden, self.n_heads, self.head_dim, self.max_ctx = (
            B, hidden, n_heads, head_dim, max_ctx)
        self.handle = cfa_plan_create(B, hidden, n_heads, head_dim, max_ctx)
        try:
            if cluster_size is not None:
                self.set_cluster_size(cluster_size)
            if qkv_exchange is not None:
                self.set_qkv_exchange(qkv_exchange)
            if stages is not None:
                self.set_stages(stages)
            if overlap is not None:
                self.set_overlap(overlap)
        except Exception:
            self.close()
            raise

    def close(self):
        if getattr(self, "handle", None):
            cfa_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def cluster_size(self) -> int:
        return cfa_plan_cluster_size(self.handle)

    def set_cluster_size(self, C: int) -> None:
        st = cfa_plan_set_cluster_size(self.handle, C)
        if st != CFA_OK:
            raise CfaError(st, f"cluster size {C}")

    def set_stages(self, n: int) -> None:
        st = cfa_plan_set_stages(self.handle, n)
        if st != CFA_OK:
            raise CfaError(st, f"stages {n}")

    def set_qkv_exchange(self, mode: int) -> None:
        """-1 automatic, 0 gather, 1 reduce-scatter (cfa_plan_set_qkv_exchange)."""
        st = cfa_plan_set_qkv_exchange(self.handle, mode)
        if st != CFA_OK:
            raise CfaError(st, f"qkv exchange {mode}")

    def set_overlap(self, enable: bool) -> None:
        st = cfa_plan_set_overlap(self.handle, enable)
        if st != CFA_OK:
            raise CfaError(st, "overlap")

    def describe(self) -> dict:
        return cfa_plan_describe(self.handle)

    def status(self) -> int:
        return cfa_plan_status(self.handle)

    def _check(self, x, W_qkv, W_o, k_cache, v_cache, out, host_io: bool):
        B, H, nh, d, mc = self.B, self.hidden, self.n_heads, self.head_dim, self.max_ctx
        want = {"W_qkv": (W_qkv, (H, 3 * H)), "W_o": (W_o, (H, H)),
                "k_cache": (k_cache, (B, nh, mc, d)), "v_cache": (v_cache, (B, nh, mc, d)),
                "x": (x, (B, H)), "out": (out, (B, H))}
        for name, (t, shape) in want.items():
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be bf16")
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            on_host = name in ("x", "out") and host_io
            if on_host == t.is_cuda:
                raise ValueError(f"{name} must be on the {'host' if on_host else 'GPU'}")

    def decode_step(self, x, W_qkv, W_o, k_cache, v_cache, ctx_len: int, out, stream=None):
        """One fused decode step on device tensors; asynchronous on `stream`."""
        self._check(x, W_qkv, W_o, k_cache, v_cache, out, host_io=False)
        st = cfa_decode_step(self.handle, x, W_qkv, W_o, k_cache, v_cache, ctx_len, out, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_decode_step")
        return out

    def decode_step_ex(self, x, W_qkv, W_o, k_cache, v_cache, ctx_lens, out,
                       rope_theta: float = 0.0, stream=None):
        """Decode step with per-sequence lengths and optional rotary embedding."""
        self._check(x, W_qkv, W_o, k_cache, v_cache, out, host_io=False)
        if len(ctx_lens) != self.B:
            raise ValueError("ctx_lens needs one entry per batch row")
        st = cfa_decode_step_ex(self.handle, x, W_qkv, W_o, k_cache, v_cache, ctx_lens,
                                rope_theta, out, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_decode_step_ex")
        return out

    def decode_step_host(self, x_host, W_qkv, W_o, k_cache, v_cache, ctx_len: int, out_host,
                         stream=None):
        """Same step with x and out in (preferably pinned) host memory; synchronous."""
        self._check(x_host, W_qkv, W_o, k_cache, v_cache, out_host, host_io=True)
        st = cfa_decode_step_host(self.handle, x_host, W_qkv, W_o, k_cache, v_cache, ctx_len,
                                  out_host, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_decode_step_host")
        return out_host


# ----------------------------------------------- decoder layers and the loop


def cfa_rmsnorm(B: int, n: int, x, g, eps: float, y, stream=None) -> int:
    return int(_lib.cfa_rmsnorm(int(B), int(n), _ptr(x), _ptr(g), float(eps), _ptr(y),
                                _stream(stream)))


def cfa_mlp_create(B: int, hidden: int, ffn: int) -> int:
    h = _lib.cfa_mlp_create(B, hidden, ffn)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_mlp_create")
    return h


def cfa_mlp_destroy(mlp: int) -> None:
    _lib.cfa_mlp_destroy(mlp)


def cfa_mlp_step(mlp, h, norm_w, eps: float, W_gate, W_up, W_down, y, stream=None) -> int:
    return int(_lib.cfa_mlp_step(mlp, _ptr(h), _ptr(norm_w), float(eps), _ptr(W_gate),
                                 _ptr(W_up), _ptr(W_down), _ptr(y), _stream(stream)))


def cfa_mlp_set_pipeline(mlp, blocks_per_sm: int, stages: int) -> int:
    return int(_lib.cfa_mlp_set_pipeline(mlp, int(blocks_per_sm), int(stages)))


# cfa_mlp_set_path: the MLP GEMVs' kernel
PATH_AUTO, PATH_CUDA_CORES, PATH_TENSOR_CORES = -1, 0, 1


def cfa_mlp_set_path(mlp, path: int) -> int:
    return int(_lib.cfa_mlp_set_path(mlp, int(path)))


def cfa_mlp_status(mlp) -> int:
    return int(_lib.cfa_mlp_status(mlp))


def cfa_mlp_describe(mlp) -> dict:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.cfa_mlp_describe(mlp, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_mlp_describe")
    return json.loads(buf.value.decode())


def cfa_stack_create(n_layers: int, B: int, hidden: int, n_heads: int, head_dim: int, ffn: int,
                     max_ctx: int) -> int:
    h = _lib.cfa_stack_create(n_layers, B, hidden, n_heads, head_dim, ffn, max_ctx)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_stack_create")
    return h


def cfa_stack_destroy(stack: int) -> None:
    _lib.cfa_stack_destroy(stack)


def cfa_stack_set_layer(stack, layer: int, attn_norm, W_qkv, W_o, k_cache, v_cache, mlp_norm,
                        W_gate, W_up, W_down) -> int:
    return int(_lib.cfa_stack_set_layer(stack, int(layer), _ptr(attn_norm), _ptr(W_qkv),
                                        _ptr(W_o), _ptr(k_cache), _ptr(v_cache), _ptr(mlp_norm),
                                        _ptr(W_gate), _ptr(W_up), _ptr(W_down)))


def cfa_stack_step(stack, x, positions, rope_theta: float, eps: float, advance: bool, out,
                   stream=None) -> int:
    return int(_lib.cfa_stack_step(stack, _ptr(x), _ptr(positions), float(rope_theta),
                                   float(eps), 1 if advance else 0, _ptr(out), _stream(stream)))


def cfa_stack_step_graph(stack, x, positions, rope_theta: float, eps: float, advance: bool, out,
                         stream=None) -> int:
    return int(_lib.cfa_stack_step_graph(stack, _ptr(x), _ptr(positions), float(rope_theta),
                                         float(eps), 1 if advance else 0, _ptr(out),
                                         _stream(stream)))


def cfa_stack_status(stack) -> int:
    return int(_lib.cfa_stack_status(stack))


def cfa_stack_describe(stack) -> dict:
    buf = ctypes.create_string_buffer(2048)
    st = _lib.cfa_stack_describe(stack, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_stack_describe")
    return json.loads(buf.value.decode())


def _check_tensor(name, t, shape, dtype=torch.bfloat16):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def rmsnorm(x, g, eps: float, y, stream=None):
    """y = bf16(g * x / sqrt(mean(x^2) + eps)) row by row, on the GPU."""
    B, n = x.shape
    _check_tensor("x", x, (B, n))
    _check_tensor("g", g, (n,))
    _check_tensor("y", y, (B, n))
    st = cfa_rmsnorm(B, n, x, g, eps, y, stream)
    if st != CFA_OK:
        raise CfaError(st, "cfa_rmsnorm")
    return y


class Mlp:
    """Owns a cfa_mlp: y = h + down(silu(gate(hn)) * up(hn)), hn = rmsnorm(h)."""

    def __init__(self, B: int, hidden: int, ffn: int):
        self.B, self.hidden, self.ffn = B, hidden, ffn
        self.handle = cfa_mlp_create(B, hidden, ffn)

    def close(self):
        if getattr(self, "handle", None):
            cfa_mlp_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def describe(self) -> dict:
        return cfa_mlp_describe(self.handle)

    def set_pipeline(self, blocks_per_sm: int = 0, stages: int = 0) -> None:
        st = cfa_mlp_set_pipeline(self.handle, blocks_per_sm, stages)
        if st != CFA_OK:
            raise CfaError(st, f"pipeline {blocks_per_sm} x {stages}")

    def set_path(self, path: int) -> None:
        """PATH_AUTO (tensor cores from B = 2), PATH_CUDA_CORES or PATH_TENSOR_CORES."""
        st = cfa_mlp_set_path(self.handle, path)
        if st != CFA_OK:
            raise CfaError(st, f"path {path}")

    def status(self) -> int:
        return cfa_mlp_status(self.handle)

    def step(self, h, norm_w, W_gate, W_up, W_down, y, eps: float = 1e-5, stream=None):
        B, H, F = self.B, self.hidden, self.ffn
        for name, t, shape in (("h", h, (B, H)), ("norm_w", norm_w, (H,)),
                               ("W_gate", W_gate, (H, F)), ("W_up", W_up, (H, F)),
                               ("W_down", W_down, (F, H)), ("y", y, (B, H))):
            _check_tensor(name, t, shape)
        st = cfa_mlp_step(self.handle, h, norm_w, eps, W_gate, W_up, W_down, y, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_mlp_step")
        return y


class Stack:
    """Owns a cfa_stack: n_layers decoder layers run token by token.

    layers: sequence of mappings with attn_norm, W_qkv, W_o, k_cache, v_cache,
    mlp_norm, W_gate, W_up, W_down (device bf16 tensors, kept referenced here
    so they outlive the stack's use of them)."""

    _KEYS = ("attn_norm", "W_qkv", "W_o", "k_cache", "v_cache", "mlp_norm", "W_gate", "W_up",
             "W_down")

    def __init__(self, n_layers: int, B: int, hidden: int, n_heads: int, head_dim: int,
                 ffn: int, max_ctx: int, layers=None):
        self.n_layers, self.B, self.hidden, self.n_heads, self.head_dim = (
            n_layers, B, hidden, n_heads, head_dim)
        self.ffn, self.max_ctx = ffn, max_ctx
        self.handle = cfa_stack_create(n_layers, B, hidden, n_heads, head_dim, ffn, max_ctx)
        self._layers = [None] * n_layers
        if layers is not None:
            for i, layer in enumerate(layers):
                self.set_layer(i, layer)

    def close(self):
        if getattr(self, "handle", None):
            cfa_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def describe(self) -> dict:
        return cfa_stack_describe(self.handle)

    def status(self) -> int:
        return cfa_stack_status(self.handle)

    def set_layer(self, i: int, layer) -> None:
        B, H, nh, d, F, mc = (self.B, self.hidden, self.n_heads, self.head_dim, self.ffn,
                              self.max_ctx)
        shapes = {"attn_norm": (H,), "W_qkv": (H, 3 * H), "W_o": (H, H),
                  "k_cache": (B, nh, mc, d), "v_cache": (B, nh, mc, d), "mlp_norm": (H,),
                  "W_gate": (H, F), "W_up": (H, F), "W_down": (F, H)}
        for k in self._KEYS:
            _check_tensor(k, layer[k], shapes[k])
        st = cfa_stack_set_layer(self.handle, i, *[layer[k] for k in self._KEYS])
        if st != CFA_OK:
            raise CfaError(st, f"cfa_stack_set_layer({i})")
        self._layers[i] = {k: layer[k] for k in self._KEYS}

    def _check_io(self, x, positions, out):
        _check_tensor("x", x, (self.B, self.hidden))
        _check_tensor("out", out, (self.B, self.hidden))
        _check_tensor("positions", positions, (self.B,), torch.int32)

    def step(self, x, positions, out, rope_theta: float = 10000.0, eps: float = 1e-5,
             advance: bool = False, stream=None):
        """One token through every layer (eager launches)."""
        self._check_io(x, positions, out)
        st = cfa_stack_step(self.handle, x, positions, rope_theta, eps, advance, out, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_stack_step")
        return out

    def step_graph(self, x, positions, out, rope_theta: float = 10000.0, eps: float = 1e-5,
                   advance: bool = False, stream=None):
        """One token through every layer, recorded once into a CUDA graph and
        replayed; `stream` must not be the legacy default stream."""
        self._check_io(x, positions, out)
        st = cfa_stack_step_graph(self.handle, x, positions, rope_theta, eps, advance, out,
                                  stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_stack_step_graph")
        return out


# ------------------------------------------------ multi-head latent attention

MLA_KV, MLA_NOPE, MLA_ROPE, MLA_V = 512, 128, 64, 128
MLA_ROW = MLA_KV + MLA_ROPE
MLA_QK = MLA_NOPE + MLA_ROPE


def cfa_mla_create(B: int, hidden: int, n_heads: int, q_lora: int, max_ctx: int) -> int:
    h = _lib.cfa_mla_create(B, hidden, n_heads, q_lora, max_ctx)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_mla_create")
    return h


def cfa_mla_destroy(mla: int) -> None:
    _lib.cfa_mla_destroy(mla)


def cfa_mla_step(mla, x, W_a, g_q, g_kv, W_uq, W_kvb, W_o, cache, ctx_lens, rope_theta: float,
                 eps: float, out, stream=None) -> int:
    lens = (ctypes.c_int * len(ctx_lens))(*[int(v) for v in ctx_lens])
    return int(_lib.cfa_mla_step(mla, _ptr(x), _ptr(W_a), _ptr(g_q), _ptr(g_kv), _ptr(W_uq),
                                 _ptr(W_kvb), _ptr(W_o), _ptr(cache), lens, float(rope_theta),
                                 float(eps), _ptr(out), _stream(stream)))


def cfa_mla_status(mla) -> int:
    return int(_lib.cfa_mla_status(mla))


def cfa_mla_describe(mla) -> dict:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.cfa_mla_describe(mla, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_mla_describe")
    return json.loads(buf.value.decode())


def cfa_mla_set_row_splits(mla, splits: int) -> int:
    return int(_lib.cfa_mla_set_row_splits(mla, int(splits)))


class Mla:
    """Owns a cfa_mla: DeepSeek-style latent-attention decode steps."""

    _KEYS = ("W_a", "g_q", "g_kv", "W_uq", "W_kvb", "W_o")

    def __init__(self, B: int, hidden: int, n_heads: int, q_lora: int, max_ctx: int):
        self.B, self.hidden, self.n_heads, self.q_lora, self.max_ctx = (
            B, hidden, n_heads, q_lora, max_ctx)
        self.handle = cfa_mla_create(B, hidden, n_heads, q_lora, max_ctx)

    def close(self):
        if getattr(self, "handle", None):
            cfa_mla_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def describe(self) -> dict:
        return cfa_mla_describe(self.handle)

    def set_row_splits(self, splits: int):
        """1, 2 or 4 clusters per (sequence, head group), each over its share of
        the latent rows (0: chosen per step); raises CfaError if that grid does
        not fit at once."""
        st = cfa_mla_set_row_splits(self.handle, splits)
        if st != CFA_OK:
            raise CfaError(st, "cfa_mla_set_row_splits")

    def status(self) -> int:
        return cfa_mla_status(self.handle)

    def step(self, x, weights, cache, ctx_lens, out, rope_theta: float = 10000.0,
             eps: float = 1e-6, stream=None):
        B, H, nh, ql, mc = self.B, self.hidden, self.n_heads, self.q_lora, self.max_ctx
        shapes = {"W_a": (H, ql + MLA_ROW), "g_q": (ql,), "g_kv": (MLA_KV,),
                  "W_uq": (ql, nh * (MLA_NOPE + MLA_ROPE)), "W_kvb": (MLA_KV, nh * (MLA_NOPE + MLA_V)),
                  "W_o": (nh * MLA_V, H)}
        for k in self._KEYS:
            _check_tensor(k, weights[k], shapes[k])
        _check_tensor("x", x, (B, H))
        _check_tensor("out", out, (B, H))
        _check_tensor("cache", cache, (B, mc, MLA_ROW))
        if len(ctx_lens) != B:
            raise ValueError("ctx_lens needs one entry per batch row")
        st = cfa_mla_step(self.handle, x, *[weights[k] for k in self._KEYS], cache, ctx_lens,
                          rope_theta, eps, out, stream)
        if st != CFA_OK:
            raise CfaError(st, "cfa_mla_step")
        return out


# -------------------------------------------- paged caches and shared prefixes

ROPE_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def cfa_paged_create(max_seqs: int, max_tokens: int, n_heads: int, n_kv_heads: int,
                     head_dim: int, page_size: int) -> int:
    h = _lib.cfa_paged_create(max_seqs, max_tokens, n_heads, n_kv_heads, head_dim, page_size)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_paged_create")
    return h


def cfa_paged_destroy(paged: int) -> None:
    _lib.cfa_paged_destroy(paged)


def cfa_paged_status(paged) -> int:
    return int(_lib.cfa_paged_status(paged))


def cfa_paged_describe(paged) -> dict:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.cfa_paged_describe(paged, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_paged_describe")
    return json.loads(buf.value.decode())


class Paged:
    """Owns a cfa_paged: block tables, rotary append and shared-prefix attention.

    k_pages and v_pages are bf16 [n_pages, n_kv_heads, page_size, head_dim];
    q, k, v [tokens, heads, head_dim] may be slices of a fused projection (dense
    within a row); every integer tensor is int32 on the plan's device. Calls go to the
    current stream of that device, or to ``stream``; the tensors of a call on a stream
    other than their own have to be kept (or ``record_stream``-ed) until it has run."""

    def __init__(self, max_seqs: int, max_tokens: int, n_heads: int, n_kv_heads: int,
                 head_dim: int, page_size: int):
        self.max_seqs, self.max_tokens = max_seqs, max_tokens
        self.n_heads, self.n_kv_heads, self.head_dim, self.page_size = (
            n_heads, n_kv_heads, head_dim, page_size)
        self.handle = cfa_paged_create(max_seqs, max_tokens, n_heads, n_kv_heads, head_dim,
                                       page_size)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._page_shape = (n_kv_heads, page_size, head_dim)

    def close(self):
        if getattr(self, "handle", None):
            cfa_paged_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def describe(self) -> dict:
        return cfa_paged_describe(self.handle)

    def status(self) -> int:
        return cfa_paged_status(self.handle)

    def set_rope(self, theta: float = 10000.0, rotary_dim: Optional[int] = None,
                 interleaved: bool = False, scaling: str = "none", factor: float = 1.0,
                 low_turns: float = 1.0, high_turns: float = 32.0, original_ctx: int = 4096,
                 magnitude: float = 1.0) -> None:
        """The rotation of the following append and layer calls (cfa_paged_set_rope);
        rotary_dim None: the whole head, 0: no rotation."""
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        rd = self.head_dim if rotary_dim is None else int(rotary_dim)
        st = _lib.cfa_paged_set_rope(self.handle, float(theta), rd, 1 if interleaved else 0,
                                     ROPE_SCALINGS[scaling], float(factor), float(low_turns),
                                     float(high_turns), int(original_ctx), float(magnitude))
        if st != CFA_OK:
            raise CfaError(st, "cfa_paged_set_rope")

    # Argument checks. The smallest calls take the GPU only microseconds, so each method
    # asks in one expression whether everything is right, and looks for what is wrong
    # (these two) only where it is not.

    def _check(self, name, t, shape, dtype):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")

    def _check_rows(self, name, t, n, heads):
        if t.dtype is not _BF16:
            raise TypeError(f"{name} must be {_BF16}")
        if t.shape != (n, heads, self.head_dim):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                             f"{(n, heads, self.head_dim)}")
        s = t.stride()
        if s[2] != 1 or (heads > 1 and s[1] != self.head_dim):
            raise ValueError(f"{name} must be dense within a row")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")

    def _rows(self, name, t, n, heads):
        """Pointer and row stride of [n, heads, head_dim] with dense rows."""
        d = self.head_dim
        row, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
        if not (t.dtype is _BF16 and t.shape == (n, heads, d) and one == 1
                and (head == d or heads == 1) and t.get_device() == self._index):
            self._check_rows(name, t, n, heads)
        return t.data_ptr(), (row if n > 1 else heads * d)

    def _pages(self, k_pages, v_pages):
        shape = k_pages.shape
        i = self._index
        if not (k_pages.dtype is v_pages.dtype is _BF16 and shape == v_pages.shape
                and shape[1:] == self._page_shape and k_pages.is_contiguous()
                and v_pages.is_contiguous() and k_pages.get_device() == i == v_pages.get_device()):
            shape = (shape[0],) + self._page_shape
            self._check("k_pages", k_pages, shape, _BF16)
            self._check("v_pages", v_pages, shape, _BF16)
        return shape[0], k_pages.data_ptr(), v_pages.data_ptr()

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        return _stream(stream)

    def build_tables(self, lens, fresh, free_pages, pool, tables, lens_out, pool_out, cu, positions,
                     slots, base: int = 0, stream=None):
        """Pages, offsets, positions and slots of one step (cfa_paged_tables):
        lens, fresh, lens_out [B]; free_pages [n]; pool, pool_out [2]; tables
        [B, width]; cu [B + 1]; positions, slots [rows]. base is the prefix's
        length. Returns (cu, positions, slots)."""
        one, n, free, i = lens.shape, slots.shape, free_pages.shape, self._index
        if len(one) != 1 or len(n) != 1 or len(free) != 1 or tables.dim() != 2:
            raise ValueError("lens, slots and free_pages have one dimension, tables two")
        B, width = tables.shape
        if not (lens.dtype is fresh.dtype is free_pages.dtype is pool.dtype is tables.dtype
                is lens_out.dtype is pool_out.dtype is cu.dtype is positions.dtype is slots.dtype
                is _I32 and one[0] == B and fresh.shape == one == lens_out.shape
                and positions.shape == n and pool.shape == (2,) == pool_out.shape
                and cu.shape == (B + 1,)
                and lens.is_contiguous() and fresh.is_contiguous() and free_pages.is_contiguous()
                and pool.is_contiguous() and tables.is_contiguous() and lens_out.is_contiguous()
                and pool_out.is_contiguous() and cu.is_contiguous() and positions.is_contiguous()
                and slots.is_contiguous()
                and lens.get_device() == i == fresh.get_device() == free_pages.get_device()
                == pool.get_device() == tables.get_device() == lens_out.get_device()
                == pool_out.get_device() == cu.get_device() == positions.get_device()
                == slots.get_device()):
            for name, t, shape in (("lens", lens, (B,)), ("fresh", fresh, (B,)),
                                   ("free_pages", free_pages, free), ("pool", pool, (2,)),
                                   ("tables", tables, (B, width)), ("lens_out", lens_out, (B,)),
                                   ("pool_out", pool_out, (2,)), ("cu", cu, (B + 1,)),
                                   ("positions", positions, n), ("slots", slots, n)):
                self._check(name, t, shape, _I32)
        st = _lib.cfa_paged_tables(
            self.handle, B, base, lens.data_ptr(), fresh.data_ptr(), free_pages.data_ptr(), free[0],
            pool.data_ptr(), tables.data_ptr(), width, lens_out.data_ptr(), pool_out.data_ptr(),
            cu.data_ptr(), positions.data_ptr(), slots.data_ptr(), n[0], self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_paged_tables")
        return cu, positions, slots

    def append(self, q, k, v, positions, slots, k_pages, v_pages, q_out, stream=None):
        """Rotate q into q_out and k into its page, put v into its page
        (cfa_paged_append). Returns q_out."""
        T = q.shape[0]
        n, kc, vc = self._pages(k_pages, v_pages)
        st = _lib.cfa_paged_append(
            self.handle, T, *self._rows("q", q, T, self.n_heads), *self._rows("k", k, T, self.n_kv_heads),
            *self._rows("v", v, T, self.n_kv_heads), *self._tokens(T, positions, slots), n, kc, vc,
            self._turned(T, q_out), self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_paged_append")
        return q_out

    def _tokens(self, T, positions, slots):
        i = self._index
        if not (positions.dtype is slots.dtype is _I32 and positions.shape == (T,) == slots.shape
                and positions.is_contiguous() and slots.is_contiguous()
                and positions.get_device() == i == slots.get_device()):
            self._check("positions", positions, (T,), _I32)
            self._check("slots", slots, (T,), _I32)
        return positions.data_ptr(), slots.data_ptr()

    def _turned(self, T, q_out):
        shape = (T, self.n_heads, self.head_dim)
        if not (q_out.dtype is _BF16 and q_out.shape == shape and q_out.is_contiguous()
                and q_out.get_device() == self._index):
            self._check("q_out", q_out, shape, _BF16)
        return q_out.data_ptr()

    def _attn(self, T, cu, lens, tables, prefix_table, prefix_len, scale, out, lse):
        one, i = lens.shape, self._index
        if len(one) != 1 or tables.dim() != 2:
            raise ValueError("lens has one dimension, tables two")
        if prefix_len < 0:
            raise ValueError("prefix_len must not be negative")
        if scale is not None and not ctypes.c_float(scale).value > 0.0:
            raise ValueError("scale must be positive, in 32 bits too")
        B, width = tables.shape
        shape = (T, self.n_heads, self.head_dim)
        if not (lens.dtype is cu.dtype is tables.dtype is _I32 and out.dtype is _BF16
                and one[0] == B and cu.shape == (B + 1,) and out.shape == shape
                and lens.is_contiguous() and cu.is_contiguous() and tables.is_contiguous()
                and out.is_contiguous()
                and lens.get_device() == i == cu.get_device() == tables.get_device() == out.get_device()):
            self._check("lens", lens, one, _I32)
            self._check("cu", cu, one[:0] + (one[0] + 1,), _I32)
            self._check("tables", tables, (one[0], width), _I32)
            self._check("out", out, shape, _BF16)
        pt = None
        if prefix_len:
            if prefix_table is None or prefix_table.numel() * self.page_size < prefix_len:
                raise ValueError("prefix_table does not hold prefix_len positions")
            if not (prefix_table.dtype is _I32 and prefix_table.is_contiguous()
                    and prefix_table.get_device() == i):
                self._check("prefix_table", prefix_table, prefix_table.shape, _I32)
            pt = prefix_table.data_ptr()
        if lse is not None:
            self._check("lse", lse, shape[:2], _F32)
        return (B, cu.data_ptr(), pt, tables.data_ptr(), width, lens.data_ptr(), out.data_ptr(),
                None if lse is None else lse.data_ptr(), scale or 0.0)

    def attend(self, q, cu, lens, tables, k_pages, v_pages, out, prefix_table=None,
               prefix_len: int = 0, scale: Optional[float] = None, lse=None, stream=None):
        """Attention over the shared prefix and each request's own pages
        (cfa_paged_attention). scale None: 1/sqrt(head_dim). Returns out."""
        T = q.shape[0]
        qp, qs = self._rows("q", q, T, self.n_heads)
        n, kc, vc = self._pages(k_pages, v_pages)
        B, cup, pt, tp, width, lp, op, sp, scale = self._attn(T, cu, lens, tables, prefix_table,
                                                              prefix_len, scale, out, lse)
        st = _lib.cfa_paged_attention(self.handle, T, B, qp, qs, cup, pt, prefix_len, tp, width, lp,
                                      n, kc, vc, scale, op, sp, self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_paged_attention")
        return out

    def layer(self, q, k, v, positions, slots, cu, lens, tables, k_pages, v_pages, q_out, out,
              prefix_table=None, prefix_len: int = 0, scale: Optional[float] = None, lse=None,
              stream=None):
        """append, then attend on q_out (cfa_paged_layer). Returns out."""
        T = q.shape[0]
        n, kc, vc = self._pages(k_pages, v_pages)
        B, cup, pt, tp, width, lp, op, sp, scale = self._attn(T, cu, lens, tables, prefix_table,
                                                              prefix_len, scale, out, lse)
        st = _lib.cfa_paged_layer(
            self.handle, T, B, *self._rows("q", q, T, self.n_heads),
            *self._rows("k", k, T, self.n_kv_heads), *self._rows("v", v, T, self.n_kv_heads),
            *self._tokens(T, positions, slots), cup, pt, prefix_len, tp, width, lp, n, kc, vc, scale,
            self._turned(T, q_out), op, sp, self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_paged_layer")
        return out


# --------------------------------------------------------- paged latent caches


def cfa_latent_create(max_seqs: int, max_tokens: int, n_heads: int, page_size: int) -> int:
    h = _lib.cfa_latent_create(max_seqs, max_tokens, n_heads, page_size)
    if not h:
        raise CfaError(cfa_last_error(), "cfa_latent_create")
    return h


def cfa_latent_destroy(latent: int) -> None:
    _lib.cfa_latent_destroy(latent)


def cfa_latent_status(latent) -> int:
    return int(_lib.cfa_latent_status(latent))


def cfa_latent_describe(latent) -> dict:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.cfa_latent_describe(latent, buf, len(buf))
    if st != CFA_OK:
        raise CfaError(st, "cfa_latent_describe")
    return json.loads(buf.value.decode())


class Latent:
    """Owns a cfa_latent: latent attention over paged caches, for ragged batches.

    pages are bf16 [n_pages, page_size, 576] (normed latent 512 | rotated key 64); tables,
    offsets, positions and slots as ``Paged.build_tables`` of the same page_size makes them. W_kvb
    [512, n_heads * 256] is the ``Mla`` step's. Decode: append, fold, attend, unfold (or layer,
    which runs the four); prompts: append, then attend_expanded on keys and values the caller has
    expanded. Integer tensors are int32 on the plan's device; streams as in ``Paged``."""

    def __init__(self, max_seqs: int, max_tokens: int, n_heads: int, page_size: int):
        self.max_seqs, self.max_tokens, self.n_heads, self.page_size = (
            max_seqs, max_tokens, n_heads, page_size)
        self.handle = cfa_latent_create(max_seqs, max_tokens, n_heads, page_size)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        # shapes behind the tokens, keys or pages
        self._q_shape, self._lat_shape, self._o_shape = (n_heads, MLA_QK), (n_heads, MLA_ROW), (n_heads, MLA_KV)
        self._out_shape, self._kv_shape = (n_heads, MLA_V), (n_heads, MLA_NOPE + MLA_V)
        self._page_shape, self._w_shape = (page_size, MLA_ROW), (MLA_KV, n_heads * (MLA_NOPE + MLA_V))
        self._q_width, self._kv_width = n_heads * MLA_QK, n_heads * (MLA_NOPE + MLA_V)

    def close(self):
        if getattr(self, "handle", None):
            cfa_latent_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def describe(self) -> dict:
        return cfa_latent_describe(self.handle)

    def status(self) -> int:
        return cfa_latent_status(self.handle)

    def set_rope(self, theta: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, low_turns: float = 1.0, high_turns: float = 32.0,
                 original_ctx: int = 4096, magnitude: float = 1.0) -> None:
        """The rotation of the following append and layer calls (cfa_latent_set_rope);
        theta 0: no rotation. "by_parts" ramps linearly in a pair's turns, not in its index.
        magnitude is that of the 64 rotated dims; one of the whole score goes, squared, into the
        attention's scale."""
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        st = _lib.cfa_latent_set_rope(self.handle, float(theta), 1 if interleaved else 0,
                                      ROPE_SCALINGS[scaling], float(factor), float(low_turns),
                                      float(high_turns), int(original_ctx), float(magnitude))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_set_rope")

    # Argument checks. The smallest calls take the GPU only microseconds, so each method asks in one
    # expression whether everything is right, and looks for what is wrong (these) only where it is not.

    def _dense(self, name, t, shape, dtype=_BF16):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")

    def _rows(self, name, t, n, *dims):
        """bf16 [n, *dims] with dense rows."""
        if t.dtype is not _BF16:
            raise TypeError(f"{name} must be {_BF16}")
        if t.shape != (n, *dims):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, *dims)}")
        if not self._dense_rows(t.stride(), dims):
            raise ValueError(f"{name} must be dense within a row")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")

    @staticmethod
    def _dense_rows(stride, dims):
        width = 1
        for i in range(len(dims), 0, -1):
            if stride[i] != width and dims[i - 1] != 1:
                return False
            width *= dims[i - 1]
        return True

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        return _stream(stream)

    def _scale(self, scale):
        if scale is None:
            return 0.0
        if not ctypes.c_float(scale).value > 0.0:
            raise ValueError("scale must be positive, in 32 bits too")
        return scale

    def _append(self, a, g_kv, eps, q, positions, slots, pages, q_out):
        shape, one, page, i = q.shape, positions.shape, pages.shape, self._index
        T = shape[0]
        sa, sq = a.stride(), q.stride()
        if not (a.dtype is q.dtype is g_kv.dtype is pages.dtype is q_out.dtype is _BF16
                and positions.dtype is slots.dtype is _I32
                and shape[1:] == self._q_shape and q_out.shape == shape and a.shape == (T, MLA_ROW)
                and one == (T,) == slots.shape and page[1:] == self._page_shape and g_kv.shape == (MLA_KV,)
                and sa[1] == 1 == sq[2] and sq[1] == MLA_QK
                and q_out.is_contiguous() and pages.is_contiguous() and g_kv.is_contiguous()
                and positions.is_contiguous() and slots.is_contiguous()
                and a.get_device() == i == q.get_device() == g_kv.get_device() == pages.get_device()
                == q_out.get_device() == positions.get_device() == slots.get_device()):
            self._rows("q", q, T, *self._q_shape)
            self._rows("a", a, T, MLA_ROW)
            for name, t, shape, dtype in (("g_kv", g_kv, (MLA_KV,), _BF16), ("positions", positions, (T,), _I32),
                                          ("slots", slots, (T,), _I32),
                                          ("pages", pages, (page[0], *self._page_shape), _BF16),
                                          ("q_out", q_out, (T, *self._q_shape), _BF16)):
                self._dense(name, t, shape, dtype)
        return (a.data_ptr(), sa[0] if T > 1 else MLA_ROW, g_kv.data_ptr(), eps, q.data_ptr(),
                sq[0] if T > 1 else self._q_width, positions.data_ptr(), slots.data_ptr(), page[0],
                pages.data_ptr(), q_out.data_ptr())

    def _attn(self, q_lat, cu, lens, tables, pages, o_lat, lse):
        shape, one, page, i = q_lat.shape, lens.shape, pages.shape, self._index
        if len(one) != 1 or tables.dim() != 2:
            raise ValueError("lens has one dimension, tables two")
        T = shape[0]
        B, width = tables.shape
        if not (q_lat.dtype is pages.dtype is o_lat.dtype is _BF16
                and cu.dtype is lens.dtype is tables.dtype is _I32
                and shape[1:] == self._lat_shape and o_lat.shape == (T, *self._o_shape)
                and page[1:] == self._page_shape and one[0] == B and cu.shape == (B + 1,)
                and q_lat.is_contiguous() and pages.is_contiguous() and o_lat.is_contiguous()
                and cu.is_contiguous() and lens.is_contiguous() and tables.is_contiguous()
                and q_lat.get_device() == i == pages.get_device() == o_lat.get_device() == cu.get_device()
                == lens.get_device() == tables.get_device()):
            for name, t, shape, dtype in (("q_lat", q_lat, (T, *self._lat_shape), _BF16),
                                          ("lens", lens, one, _I32), ("cu", cu, (one[0] + 1,), _I32),
                                          ("tables", tables, (one[0], width), _I32),
                                          ("pages", pages, (page[0], *self._page_shape), _BF16),
                                          ("o_lat", o_lat, (T, *self._o_shape), _BF16)):
                self._dense(name, t, shape, dtype)
        if lse is not None:
            self._dense("lse", lse, (T, self.n_heads), _F32)
        return (B, q_lat.data_ptr(), cu.data_ptr(), tables.data_ptr(), width, lens.data_ptr(), page[0],
                pages.data_ptr(), o_lat.data_ptr(), None if lse is None else lse.data_ptr())

    def append(self, a, g_kv, q, positions, slots, pages, q_out, eps: float = 1e-6, stream=None):
        """Cache rows of a [T, 576] (a slice of the down projection) into their slots, q
        [T, heads, 192] rotated into q_out, which may be q (cfa_latent_append). Returns q_out."""
        st = _lib.cfa_latent_append(self.handle, q.shape[0],
                                    *self._append(a, g_kv, eps, q, positions, slots, pages, q_out),
                                    self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_append")
        return q_out

    def fold(self, q, W_kvb, q_lat, stream=None):
        """q [T, heads, 192] into the latent space: q_lat [T, heads, 576] (cfa_latent_fold)."""
        shape, sq, i = q.shape, q.stride(), self._index
        T = shape[0]
        if not (q.dtype is W_kvb.dtype is q_lat.dtype is _BF16 and shape[1:] == self._q_shape and sq[2] == 1
                and sq[1] == MLA_QK and W_kvb.shape == self._w_shape and q_lat.shape == (T, *self._lat_shape)
                and W_kvb.is_contiguous() and q_lat.is_contiguous()
                and q.get_device() == i == W_kvb.get_device() == q_lat.get_device()):
            self._rows("q", q, T, *self._q_shape)
            self._dense("W_kvb", W_kvb, self._w_shape)
            self._dense("q_lat", q_lat, (T, *self._lat_shape))
        st = _lib.cfa_latent_fold(self.handle, T, q.data_ptr(), sq[0] if T > 1 else self._q_width,
                                  W_kvb.data_ptr(), q_lat.data_ptr(), self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_fold")
        return q_lat

    def unfold(self, o_lat, W_kvb, out, stream=None):
        """o_lat [T, heads, 512] out of the latent space: out [T, heads, 128] (cfa_latent_unfold)."""
        shape, i = o_lat.shape, self._index
        T = shape[0]
        if not (o_lat.dtype is W_kvb.dtype is out.dtype is _BF16 and shape[1:] == self._o_shape
                and W_kvb.shape == self._w_shape and out.shape == (T, *self._out_shape)
                and o_lat.is_contiguous() and W_kvb.is_contiguous() and out.is_contiguous()
                and o_lat.get_device() == i == W_kvb.get_device() == out.get_device()):
            self._dense("o_lat", o_lat, (T, *self._o_shape))
            self._dense("W_kvb", W_kvb, self._w_shape)
            self._dense("out", out, (T, *self._out_shape))
        st = _lib.cfa_latent_unfold(self.handle, T, o_lat.data_ptr(), W_kvb.data_ptr(), out.data_ptr(),
                                    self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_unfold")
        return out

    def attend(self, q_lat, cu, lens, tables, pages, o_lat, scale: Optional[float] = None, lse=None,
               stream=None):
        """Attention of folded queries over the cached rows (cfa_latent_attention). scale None:
        1/sqrt(192). Returns o_lat [T, heads, 512]."""
        B, qp, cup, tp, width, lp, n, pp, op, sp = self._attn(q_lat, cu, lens, tables, pages, o_lat, lse)
        st = _lib.cfa_latent_attention(self.handle, q_lat.shape[0], B, qp, cup, tp, width, lp, n, pp,
                                       self._scale(scale), op, sp, self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_attention")
        return o_lat

    def attend_expanded(self, q, kv, k_rope, cu, cu_k, out, scale: Optional[float] = None, lse=None,
                        stream=None):
        """Attention of prompts: q [T, heads, 192] over kv [S, heads, 256] (key 128 | value 128)
        and k_rope [S, 64], requests' rows by cu and cu_k (cfa_latent_expanded). Returns out
        [T, heads, 128]."""
        shape, many, one, i = q.shape, kv.shape, cu.shape, self._index
        if len(one) != 1:
            raise ValueError("cu has one dimension")
        T, S, B = shape[0], many[0], one[0] - 1
        sq, sk, sr = q.stride(), kv.stride(), k_rope.stride()
        if not (q.dtype is kv.dtype is k_rope.dtype is out.dtype is _BF16 and cu.dtype is cu_k.dtype is _I32
                and shape[1:] == self._q_shape and many[1:] == self._kv_shape and k_rope.shape == (S, MLA_ROPE)
                and out.shape == (T, *self._out_shape) and cu_k.shape == one
                and sq[2] == 1 == sk[2] == sr[1] and sq[1] == MLA_QK and sk[1] == MLA_NOPE + MLA_V
                and out.is_contiguous() and cu.is_contiguous() and cu_k.is_contiguous()
                and q.get_device() == i == kv.get_device() == k_rope.get_device() == out.get_device()
                == cu.get_device() == cu_k.get_device()):
            self._rows("q", q, T, *self._q_shape)
            self._rows("kv", kv, S, *self._kv_shape)
            self._rows("k_rope", k_rope, S, MLA_ROPE)
            self._dense("cu", cu, (B + 1,), _I32)
            self._dense("cu_k", cu_k, (B + 1,), _I32)
            self._dense("out", out, (T, *self._out_shape))
        if lse is not None:
            self._dense("lse", lse, (T, self.n_heads), _F32)
        st = _lib.cfa_latent_expanded(
            self.handle, T, S, B, q.data_ptr(), sq[0] if T > 1 else self._q_width, kv.data_ptr(),
            sk[0] if S > 1 else self._kv_width, k_rope.data_ptr(), sr[0] if S > 1 else MLA_ROPE, cu.data_ptr(),
            cu_k.data_ptr(), self._scale(scale), out.data_ptr(), None if lse is None else lse.data_ptr(),
            self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_expanded")
        return out

    def layer(self, a, g_kv, q, positions, slots, cu, lens, tables, pages, W_kvb, q_out, q_lat, o_lat, out,
              eps: float = 1e-6, scale: Optional[float] = None, lse=None, stream=None):
        """append, fold, attend, unfold in one call (cfa_latent_layer). Returns out."""
        T = q.shape[0]
        ap, ast, gp, eps, qp, qs, pos, sl, n, pp, qo = self._append(a, g_kv, eps, q, positions, slots, pages, q_out)
        if q_lat.shape[0] != T:
            raise ValueError(f"q_lat has {q_lat.shape[0]} tokens, expected {T}")
        B, qlp, cup, tp, width, lp, _, _, op, sp = self._attn(q_lat, cu, lens, tables, pages, o_lat, lse)
        self._dense("W_kvb", W_kvb, self._w_shape)
        self._dense("out", out, (T, *self._out_shape))
        st = _lib.cfa_latent_layer(
            self.handle, T, B, ap, ast, gp, eps, qp, qs, pos, sl, cup, tp, width, lp, n, pp, W_kvb.data_ptr(),
            self._scale(scale), qo, qlp, op, sp, out.data_ptr(), self._stream(stream))
        if st != CFA_OK:
            raise CfaError(st, "cfa_latent_layer")
        return out
