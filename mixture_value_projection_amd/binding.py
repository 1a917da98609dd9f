"""ctypes binding of ``libmova.so`` (the C ABI in include/mova.h).

Argument marshalling only: torch tensors are checked (device, dtype, shape,
contiguity), their device pointers and the current HIP stream are handed to
the library, and a negative status becomes ``MovaError``.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, NamedTuple, Optional, Tuple

import torch

from .build import LIBPATH

_LIB = None

MOVA_OK = 0
STAGES = ("router", "dispatch", "experts", "combine", "dense")


class MovaError(RuntimeError):
    def __init__(self, rc: int, what: str):
        super().__init__(f"{what}: {status_str(rc)} ({rc})")
        self.rc = rc


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmova.so once; raise if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    p = path or os.environ.get("MOVA_LIB", LIBPATH)
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m mixture_value_projection_amd.build`")
    lib = ctypes.CDLL(p)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.mova_version.restype = i
    lib.mova_version.argtypes = []
    lib.mova_status_str.restype = ctypes.c_char_p
    lib.mova_status_str.argtypes = [i]
    lib.mova_workspace_bytes.restype = sz
    lib.mova_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.mova_route.restype = i
    lib.mova_route.argtypes = [vp, vp, vp, i, i, i, i, f, vp, vp, vp]
    lib.mova_value_forward.restype = i
    lib.mova_value_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, f, i, i, vp, vp, vp, vp, sz, vp]
    lib.mova_value_forward_paged.restype = i
    lib.mova_value_forward_paged.argtypes = [vp, vp, vp, vp, i, i, i, i, f, i, i, vp, i, i, vp, vp,
                                             vp, vp, vp, sz, vp]
    lib.mova_value_forward_noalloc.restype = i
    lib.mova_value_forward_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, f, i, i, vp, vp, vp, vp]
    lib.mova_value_forward_record.restype = i
    lib.mova_value_forward_record.argtypes = [vp, vp, vp, vp, i, i, i, i, f, i, i, vp, vp, vp, vp,
                                              sz, vp]
    lib.mova_value_from_record.restype = i
    lib.mova_value_from_record.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, sz, vp]
    lib.mova_value_from_routing.restype = i
    lib.mova_value_from_routing.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, sz, vp]
    lib.mova_ffn_workspace_bytes.restype = sz
    lib.mova_ffn_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.mova_ffn_pack_gate_up.restype = i
    lib.mova_ffn_pack_gate_up.argtypes = [vp, vp, i, i, i, vp, vp]
    lib.mova_ffn_moe_forward.restype = i
    lib.mova_ffn_moe_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, vp, i, i, i, f, vp, vp,
                                         vp, vp, sz, vp]
    lib.mova_dense_workspace_bytes.restype = sz
    lib.mova_dense_workspace_bytes.argtypes = [i, i, i, i]
    lib.mova_dense_value_proj.restype = i
    lib.mova_dense_value_proj.argtypes = [vp, vp, i, i, i, i, vp, vp, sz, vp]
    lib.mova_paged_plan.restype = i
    lib.mova_paged_plan.argtypes = [vp, vp, i, i, i, i, vp, vp, i, vp, vp, vp, vp, vp, vp, vp]
    lib.mova_kv_store_paged.restype = i
    lib.mova_kv_store_paged.argtypes = [vp, vp, i, i, i, vp, vp, i, vp, vp, i, i, vp, vp, vp]
    lib.mova_block_select_workspace_bytes.restype = sz
    lib.mova_block_select_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.mova_block_select.restype = i
    lib.mova_block_select.argtypes = [vp, vp, i, i, vp, i, vp, i, i, i, i, i, i, i, vp, vp, sz, vp]
    lib.mova_attention_workspace_bytes.restype = sz
    lib.mova_attention_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.mova_attention_paged.restype = i
    lib.mova_attention_paged.argtypes = [vp, vp, vp, i, vp, vp, i, i, vp, i, vp, vp, i, i, i, i, i,
                                         f, i, vp, vp, vp, sz, vp]
    lib.mova_attention_chunk_workspace_bytes.restype = sz
    lib.mova_attention_chunk_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.mova_attention_chunk_paged.restype = i
    lib.mova_attention_chunk_paged.argtypes = [vp, vp, vp, i, vp, vp, i, i, vp, i, vp, vp, vp, i, i,
                                               i, i, i, f, i, vp, vp, vp, sz, vp]
    lib.mova_paged_copy.restype = i
    lib.mova_paged_copy.argtypes = [vp, vp, i, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.mova_paged_fork.restype = i
    lib.mova_paged_fork.argtypes = [vp, vp, vp, i, vp, i, i, i, vp, vp, i, vp, vp, vp, i, vp, vp,
                                    vp, vp]
    lib.mova_paged_free.restype = i
    lib.mova_paged_free.argtypes = [vp, vp, i, i, i, vp, vp, i, vp, vp, vp, i, vp, vp, sz, vp]
    lib.mova_paged_free_workspace_bytes.restype = sz
    lib.mova_paged_free_workspace_bytes.argtypes = [i]
    lib.mova_paged_compact_workspace_bytes.restype = sz
    lib.mova_paged_compact_workspace_bytes.argtypes = [i]
    lib.mova_paged_compact.restype = i
    lib.mova_paged_compact.argtypes = [vp, i, i, i, vp, vp, vp, vp, i, vp, vp, vp, vp, i, i, vp, vp,
                                       vp, vp, vp, sz, vp]
    lib.mova_debug_override.restype = i
    lib.mova_debug_override.argtypes = [i, i]
    lib.mova_debug_override_get.restype = i
    lib.mova_debug_override_get.argtypes = [i]
    lib.mova_timing_enable.restype = i
    lib.mova_timing_enable.argtypes = [i, ctypes.c_uint]
    lib.mova_timing_read.restype = i
    lib.mova_timing_read.argtypes = [i, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]
    _LIB = lib
    return lib


def status_str(rc: int) -> str:
    return load_library().mova_status_str(int(rc)).decode()


def version() -> int:
    return load_library().mova_version()


def workspace_bytes(T: int, d: int, E: int, k: int, n_kv_heads: int, head_dim: int) -> int:
    n = load_library().mova_workspace_bytes(T, d, E, k, n_kv_heads, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise MovaError(-2, "mova_workspace_bytes")
    return n


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape: Tuple[int, ...], device) -> None:
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def route(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor], k: int,
          scale: float = 2.5, topk_idx: Optional[torch.Tensor] = None,
          topk_w: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """mova_route: returns (idx int32 [T, k], w float32 [T, k])."""
    lib = load_library()
    T, d = x.shape
    E = router_w.shape[0]
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    if topk_idx is None:
        topk_idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=torch.float32, device=dev)
    _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    rc = lib.mova_route(_ptr(x), _ptr(router_w), _ptr(router_b), T, d, E, k, float(scale),
                        _ptr(topk_idx), _ptr(topk_w), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_route")
    return topk_idx, topk_w


def value_forward(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
                  expert_w: torch.Tensor, k: int, scale: float = 2.5,
                  n_kv_heads: Optional[int] = None, head_dim: int = 128,
                  out: Optional[torch.Tensor] = None,
                  topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_value_forward: returns out bf16 [T, n_kv_heads, head_dim].

    ``topk_idx`` / ``topk_w`` (optional, int32 / float32 [T, k]) receive the
    routing; ``workspace`` (optional uint8 tensor) is reused when large enough.
    """
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if n_kv_heads is None:
        n_kv_heads = N // head_dim
    if n_kv_heads * head_dim != N:
        raise ValueError("n_kv_heads * head_dim must equal the expert width")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    if out is None:
        out = torch.empty(T, n_kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, n_kv_heads, head_dim), dev)
    if topk_idx is not None:
        _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    if topk_w is not None:
        _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    nbytes = workspace_bytes(T, d, E, k, n_kv_heads, head_dim)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_value_forward(_ptr(x), _ptr(router_w), _ptr(router_b), _ptr(expert_w),
                                T, d, E, k, float(scale), n_kv_heads, head_dim, _ptr(out),
                                _ptr(topk_idx), _ptr(topk_w), _ptr(workspace),
                                workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_forward")
    return out


# Size of the static scratch of mova_value_forward_noalloc (MOVA_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 48 << 20


def value_forward_noalloc(x: torch.Tensor, router_w: torch.Tensor,
                          router_b: Optional[torch.Tensor], expert_w: torch.Tensor, k: int,
                          scale: float, out: torch.Tensor,
                          topk_idx: Optional[torch.Tensor] = None,
                          topk_w: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_value_forward_noalloc: mova_value_forward with the library's static
    scratch instead of a workspace.  ``out`` (bf16 [T, n_kv_heads, head_dim])
    is required, so this wrapper allocates nothing either."""
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if out.dim() != 3 or out.shape[1] * out.shape[2] != N:
        raise ValueError("out must be [T, n_kv_heads, head_dim] with n_kv_heads * head_dim = N")
    H, D = out.shape[1], out.shape[2]
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    _check(out, "out", torch.bfloat16, (T, H, D), dev)
    if topk_idx is not None:
        _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    if topk_w is not None:
        _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    rc = lib.mova_value_forward_noalloc(_ptr(x), _ptr(router_w), _ptr(router_b), _ptr(expert_w),
                                        T, d, E, k, float(scale), H, D, _ptr(out), _ptr(topk_idx),
                                        _ptr(topk_w), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_forward_noalloc")
    return out


def value_forward_paged(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
                        expert_w: torch.Tensor, k: int, scale: float, v_cache: torch.Tensor,
                        slot_mapping: torch.Tensor, out: Optional[torch.Tensor] = None,
                        topk_idx: Optional[torch.Tensor] = None,
                        topk_w: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """mova_value_forward_paged: stores each token's value vector in
    ``v_cache`` (bf16 [num_blocks, block_size, n_kv_heads, head_dim]) at
    ``slot_mapping[t]`` (int64 [T]; slots outside the pool store nothing) and,
    if ``out`` is given, in ``out`` too.  Returns ``out``."""
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if v_cache.dim() != 4:
        raise ValueError("v_cache must be [num_blocks, block_size, n_kv_heads, head_dim]")
    nb, bs, H, D = v_cache.shape
    if H * D != N:
        raise ValueError("v_cache's n_kv_heads * head_dim must equal the expert width")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    _check(v_cache, "v_cache", torch.bfloat16, (nb, bs, H, D), dev)
    _check(slot_mapping, "slot_mapping", torch.int64, (T,), dev)
    if out is not None:
        _check(out, "out", torch.bfloat16, (T, H, D), dev)
    if topk_idx is not None:
        _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    if topk_w is not None:
        _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    nbytes = workspace_bytes(T, d, E, k, H, D)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_value_forward_paged(_ptr(x), _ptr(router_w), _ptr(router_b), _ptr(expert_w),
                                      T, d, E, k, float(scale), H, D, _ptr(v_cache), nb, bs,
                                      _ptr(slot_mapping), _ptr(out), _ptr(topk_idx), _ptr(topk_w),
                                      _ptr(workspace), workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_forward_paged")
    return out


def value_from_routing(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                       expert_w: torch.Tensor, n_kv_heads: Optional[int] = None,
                       head_dim: int = 128, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_value_from_routing: value vectors rebuilt from stored inputs and
    stored routing (int32 ids, float32 weights [T, k]); ids outside [0, E)
    mark unused slots.  Returns bf16 [T, n_kv_heads, head_dim]."""
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    k = topk_idx.shape[1] if topk_idx.dim() == 2 else -1
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if n_kv_heads is None:
        n_kv_heads = N // head_dim
    if n_kv_heads * head_dim != N:
        raise ValueError("n_kv_heads * head_dim must equal the expert width")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    if out is None:
        out = torch.empty(T, n_kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, n_kv_heads, head_dim), dev)
    nbytes = workspace_bytes(T, d, E, k, n_kv_heads, head_dim)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_value_from_routing(_ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(expert_w), T, d,
                                     E, k, n_kv_heads, head_dim, _ptr(out), _ptr(workspace),
                                     workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_from_routing")
    return out


def value_forward_record(x: torch.Tensor, router_w: torch.Tensor,
                         router_b: Optional[torch.Tensor], expert_w: torch.Tensor, k: int,
                         scale: float = 2.5, n_kv_heads: Optional[int] = None, head_dim: int = 128,
                         out: Optional[torch.Tensor] = None,
                         record_ids: Optional[torch.Tensor] = None,
                         record_w: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """mova_value_forward_record: returns (out bf16 [T, H, D], record_ids int32
    [T] holding the uint32 words, record_w float16 [T, k])."""
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if n_kv_heads is None:
        n_kv_heads = N // head_dim
    if n_kv_heads * head_dim != N:
        raise ValueError("n_kv_heads * head_dim must equal the expert width")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    if out is None:
        out = torch.empty(T, n_kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
    if record_ids is None:
        record_ids = torch.empty(T, dtype=torch.int32, device=dev)
    if record_w is None:
        record_w = torch.empty(T, k, dtype=torch.float16, device=dev)
    _check(out, "out", torch.bfloat16, (T, n_kv_heads, head_dim), dev)
    _check(record_ids, "record_ids", torch.int32, (T,), dev)
    _check(record_w, "record_w", torch.float16, (T, k), dev)
    nbytes = workspace_bytes(T, d, E, k, n_kv_heads, head_dim)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_value_forward_record(_ptr(x), _ptr(router_w), _ptr(router_b), _ptr(expert_w),
                                       T, d, E, k, float(scale), n_kv_heads, head_dim, _ptr(out),
                                       _ptr(record_ids), _ptr(record_w), _ptr(workspace),
                                       workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_forward_record")
    return out, record_ids, record_w


def value_from_record(x: torch.Tensor, record_ids: torch.Tensor, record_w: torch.Tensor,
                      expert_w: torch.Tensor, n_kv_heads: Optional[int] = None,
                      head_dim: int = 128, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_value_from_record: value vectors rebuilt from stored inputs and
    compact records (record_ids int32 [T] as uint32 words, record_w float16
    [T, k])."""
    lib = load_library()
    T, d = x.shape
    E, N, d2 = expert_w.shape
    k = record_w.shape[1] if record_w.dim() == 2 else -1
    if d2 != d:
        raise ValueError("expert_w's last dim must equal x's width")
    if n_kv_heads is None:
        n_kv_heads = N // head_dim
    if n_kv_heads * head_dim != N:
        raise ValueError("n_kv_heads * head_dim must equal the expert width")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(record_ids, "record_ids", torch.int32, (T,), dev)
    _check(record_w, "record_w", torch.float16, (T, k), dev)
    _check(expert_w, "expert_w", torch.bfloat16, (E, N, d), dev)
    if out is None:
        out = torch.empty(T, n_kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, n_kv_heads, head_dim), dev)
    nbytes = workspace_bytes(T, d, E, k, n_kv_heads, head_dim)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_value_from_record(_ptr(x), _ptr(record_ids), _ptr(record_w), _ptr(expert_w), T, d,
                                    E, k, n_kv_heads, head_dim, _ptr(out), _ptr(workspace),
                                    workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_value_from_record")
    return out


def ffn_workspace_bytes(T: int, d: int, E: int, k: int, inter: int, inter_shared: int) -> int:
    n = load_library().mova_ffn_workspace_bytes(T, d, E, k, inter, inter_shared)
    if n == ctypes.c_size_t(-1).value:
        raise MovaError(-2, "mova_ffn_workspace_bytes")
    return n


def ffn_pack_gate_up(gate_w: torch.Tensor, up_w: torch.Tensor) -> torch.Tensor:
    """mova_ffn_pack_gate_up: bf16 [E, inter, d] gate and up weights (or
    [inter, d] for the shared expert) -> the interleaved [E, 2 inter, d]
    (or [2 inter, d]) layout the FFN forward reads."""
    lib = load_library()
    squeeze = gate_w.dim() == 2
    g = gate_w.unsqueeze(0) if squeeze else gate_w
    u = up_w.unsqueeze(0) if squeeze else up_w
    E, inter, d = g.shape
    _check(g, "gate_w", torch.bfloat16, (E, inter, d), g.device)
    _check(u, "up_w", torch.bfloat16, (E, inter, d), g.device)
    dst = torch.empty(E, 2 * inter, d, dtype=torch.bfloat16, device=g.device)
    rc = lib.mova_ffn_pack_gate_up(_ptr(g), _ptr(u), E, inter, d, _ptr(dst), _stream(g.device))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_ffn_pack_gate_up")
    return dst[0] if squeeze else dst


def ffn_moe_forward(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
                    gate_up_w: torch.Tensor, down_w: torch.Tensor, k: int, scale: float,
                    shared_gate_up_w: Optional[torch.Tensor] = None,
                    shared_down_w: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                    topk_w: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_ffn_moe_forward: returns bf16 [T, d].  gate_up_w comes from
    ``ffn_pack_gate_up``; the shared expert is optional."""
    lib = load_library()
    T, d = x.shape
    E, two_inter, d2 = gate_up_w.shape
    inter = two_inter // 2
    if d2 != d:
        raise ValueError("gate_up_w's last dim must equal x's width")
    inter_s = 0 if shared_gate_up_w is None else shared_gate_up_w.shape[0] // 2
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(router_w, "router_w", torch.bfloat16, (E, d), dev)
    if router_b is not None:
        _check(router_b, "router_b", torch.float32, (E,), dev)
    _check(gate_up_w, "gate_up_w", torch.bfloat16, (E, 2 * inter, d), dev)
    _check(down_w, "down_w", torch.bfloat16, (E, d, inter), dev)
    if inter_s:
        _check(shared_gate_up_w, "shared_gate_up_w", torch.bfloat16, (2 * inter_s, d), dev)
        _check(shared_down_w, "shared_down_w", torch.bfloat16, (d, inter_s), dev)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, d), dev)
    if topk_idx is not None:
        _check(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    if topk_w is not None:
        _check(topk_w, "topk_w", torch.float32, (T, k), dev)
    nbytes = ffn_workspace_bytes(T, d, E, k, inter, inter_s)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_ffn_moe_forward(_ptr(x), _ptr(router_w), _ptr(router_b), _ptr(gate_up_w),
                                  _ptr(down_w), E, k, inter, _ptr(shared_gate_up_w),
                                  _ptr(shared_down_w), inter_s, T, d, float(scale), _ptr(out),
                                  _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                                  _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_ffn_moe_forward")
    return out


def dense_workspace_bytes(T: int, d: int, n_kv_heads: int, head_dim: int) -> int:
    n = load_library().mova_dense_workspace_bytes(T, d, n_kv_heads, head_dim)
    if n == ctypes.c_size_t(-1).value:
        raise MovaError(-2, "mova_dense_workspace_bytes")
    return n


def dense_value_proj(x: torch.Tensor, w_v: torch.Tensor, n_kv_heads: Optional[int] = None,
                     head_dim: int = 128, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_dense_value_proj: the plain value projection x w_v^T as bf16
    [T, n_kv_heads, head_dim] (w_v is bf16 [n_kv_heads * head_dim, d])."""
    lib = load_library()
    T, d = x.shape
    N, d2 = w_v.shape
    if d2 != d:
        raise ValueError("w_v's last dim must equal x's width")
    if n_kv_heads is None:
        n_kv_heads = N // head_dim
    if n_kv_heads * head_dim != N:
        raise ValueError("n_kv_heads * head_dim must equal w_v's row count")
    dev = x.device
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(w_v, "w_v", torch.bfloat16, (N, d), dev)
    if out is None:
        out = torch.empty(T, n_kv_heads, head_dim, dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, n_kv_heads, head_dim), dev)
    nbytes = dense_workspace_bytes(T, d, n_kv_heads, head_dim)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    rc = lib.mova_dense_value_proj(_ptr(x), _ptr(w_v), T, d, n_kv_heads, head_dim, _ptr(out),
                                   _ptr(workspace), workspace.numel(), _stream(dev))
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_dense_value_proj")
    return out


# ---- the paged key-value cache ------------------------------------------------

# Element types of a cache pool (mova_cache_dtype).
CACHE_DTYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


class PagedPlan(NamedTuple):
    """Outputs of ``paged_plan``."""
    seq_lens: torch.Tensor      # int32 [B]
    cu_new: torch.Tensor        # int32 [B + 1]
    slot_mapping: torch.Tensor  # int64 [T]
    positions: torch.Tensor     # int32 [T]
    free_count: torch.Tensor    # int32 [1]


_NO_SIZE = ctypes.c_size_t(-1).value


def _scratch(workspace: Optional[torch.Tensor], nbytes: int, what: str, device) -> torch.Tensor:
    if nbytes == _NO_SIZE:
        raise MovaError(-2, what)
    if workspace is not None:
        if workspace.device != device or workspace.dtype is not torch.uint8:
            raise ValueError(f"workspace must be uint8 on {device}")
        if workspace.numel() >= nbytes and workspace.is_contiguous():
            return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


# The current stream's handle without the Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, name: str, device, *args) -> None:
    """Call an entry point on the device's current stream, with that device
    current."""
    if device.type != "cuda":
        raise ValueError(f"{name} needs GPU tensors, got {device}")
    index = device.index
    stream = _raw_stream(index) if _raw_stream is not None else _stream(device)
    if torch.cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != MOVA_OK:
        raise MovaError(rc, name)


_INT_MAX = 0x7fffffff


def _fits(*sizes: int) -> None:
    """The C ABI takes sizes as int, and ctypes would cut longer ones."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX:
        raise ValueError(f"sizes must fit 32 bits, got {sizes}")


def _dims(t: torch.Tensor, name: str, n: int, layout: str) -> Tuple[int, ...]:
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must be {layout}")
    if max(shape) > _INT_MAX:
        raise ValueError(f"{name}'s sizes must fit 32 bits, got {tuple(shape)}")
    return shape


# Workspace sizes depend on the sizes alone, and a served model asks for the
# same few again and again.
@functools.lru_cache(maxsize=1024)
def _attention_bytes(*sizes: int) -> int:
    return load_library().mova_attention_workspace_bytes(*sizes)


@functools.lru_cache(maxsize=1024)
def _select_bytes(*sizes: int) -> int:
    return load_library().mova_block_select_workspace_bytes(*sizes)


def paged_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, T: int, block_size: int,
               block_table: torch.Tensor, free_blocks: torch.Tensor, free_count: torch.Tensor,
               seq_lens: Optional[torch.Tensor] = None, cu_new: Optional[torch.Tensor] = None,
               slot_mapping: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None,
               free_count_out: Optional[torch.Tensor] = None) -> PagedPlan:
    """mova_paged_plan: blocks and slots of one step's T token rows.

    ``block_table`` (int32 [B, max_blocks]) and ``free_blocks`` (int32, a stack
    with ``free_count`` (int32 [1]) entries in use) are updated in place; the
    lengths are int32 [B], a negative ``new_lens`` entry ends its request.
    The new lengths and count are new tensors (pass two sets in turn to
    allocate nothing)."""
    lib = load_library()
    B, mb = _dims(block_table, "block_table", 2, "[B, max_blocks]")
    (cap,) = _dims(free_blocks, "free_blocks", 1, "[capacity]")
    dev = block_table.device
    i32 = torch.int32
    _check(block_table, "block_table", i32, (B, mb), dev)
    _check(free_blocks, "free_blocks", i32, (cap,), dev)
    _check(free_count, "free_count", i32, (1,), dev)
    _check(cached_lens, "cached_lens", i32, (B,), dev)
    _check(new_lens, "new_lens", i32, (B,), dev)
    _fits(T, block_size)
    if T < 0:
        raise ValueError("T must not be negative")
    if seq_lens is None:
        seq_lens = torch.empty_like(cached_lens)
    else:
        _check(seq_lens, "seq_lens", i32, (B,), dev)
    if cu_new is None:
        cu_new = cached_lens.new_empty(B + 1)
    else:
        _check(cu_new, "cu_new", i32, (B + 1,), dev)
    if slot_mapping is None:
        slot_mapping = torch.empty(T, dtype=torch.int64, device=dev)
    else:
        _check(slot_mapping, "slot_mapping", torch.int64, (T,), dev)
    if positions is None:
        positions = cached_lens.new_empty(T)
    else:
        _check(positions, "positions", i32, (T,), dev)
    if free_count_out is None:
        free_count_out = torch.empty_like(free_count)
    else:
        _check(free_count_out, "free_count_out", i32, (1,), dev)
    _launch(lib.mova_paged_plan, "mova_paged_plan", dev, _ptr(cached_lens), _ptr(new_lens), B, T,
            block_size, mb, _ptr(block_table), _ptr(free_blocks), cap, _ptr(free_count),
            _ptr(free_count_out), _ptr(seq_lens), _ptr(cu_new), _ptr(slot_mapping),
            _ptr(positions))
    return PagedPlan(seq_lens, cu_new, slot_mapping, positions, free_count_out)


def _check_pool(pool: torch.Tensor, name: str, shape, device) -> int:
    dtype = pool.dtype
    if dtype not in CACHE_DTYPES:
        raise ValueError(f"{name} has dtype {dtype}, expected bfloat16 or float8_e4m3fn")
    _check(pool, name, dtype, shape, device)
    return CACHE_DTYPES[dtype]


def _check_scales(k_scale, v_scale, heads: int, device) -> None:
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None:
            _check(t, name, torch.float32, (heads,), device)


def kv_store_paged(k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                   k_cache: Optional[torch.Tensor], v_cache: Optional[torch.Tensor],
                   slot_mapping: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None,
                   k_bounds: Optional[torch.Tensor] = None) -> None:
    """mova_kv_store_paged: stores key and value rows (bf16 [T, n_kv_heads,
    head_dim], either may be None with its pool) at their slots of the pools
    ([num_blocks, block_size, n_kv_heads, head_dim], bfloat16 or
    float8_e4m3fn with float32 [n_kv_heads] scales) and, if given, refreshes
    ``k_bounds`` (bf16 [num_blocks, n_kv_heads, 2, head_dim]) of the blocks
    touched."""
    lib = load_library()
    if (k is None) != (k_cache is None) or (v is None) != (v_cache is None):
        raise ValueError("k and k_cache, and v and v_cache, go together")
    if k is None and v is None:
        raise ValueError("neither keys nor values are given")
    rows, pool = (k, k_cache) if k is not None else (v, v_cache)
    T, H, D = _dims(rows, "k and v", 3, "[T, n_kv_heads, head_dim]")
    nb, bs = _dims(pool, "the pools", 4, "[num_blocks, block_size, n_kv_heads, head_dim]")[:2]
    dev = rows.device
    dtype = CACHE_DTYPES.get(pool.dtype)
    for t, p, name in ((k, k_cache, "k"), (v, v_cache, "v")):
        if t is not None:
            _check(t, name, torch.bfloat16, (T, H, D), dev)
            if _check_pool(p, name + "_cache", (nb, bs, H, D), dev) != dtype:
                raise ValueError("the pools must have the same dtype")
    _check(slot_mapping, "slot_mapping", torch.int64, (T,), dev)
    _check_scales(k_scale, v_scale, H, dev)
    if k_bounds is not None:
        _check(k_bounds, "k_bounds", torch.bfloat16, (nb, H, 2, D), dev)
    _launch(lib.mova_kv_store_paged, "mova_kv_store_paged", dev, _ptr(k), _ptr(v), T, H, D,
            _ptr(k_cache), _ptr(v_cache), dtype, _ptr(k_scale), _ptr(v_scale), nb, bs,
            _ptr(slot_mapping), _ptr(k_bounds))


def block_select(q: torch.Tensor, k_bounds: torch.Tensor, block_size: int,
                 block_table: torch.Tensor, seq_lens: torch.Tensor, keep: int,
                 keep_first: int = 1, keep_last: int = 1,
                 sel_blocks: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_block_select: int32 [B, n_kv_heads, keep] positions in each
    request's block table of the blocks whose keys can reach the highest
    logits, ascending, -1 behind the last.  ``workspace`` (optional uint8 tensor)
    is reused when large enough; else one is allocated."""
    lib = load_library()
    B, Hq, D = _dims(q, "q", 3, "[B, n_heads, head_dim]")
    nb, H = _dims(k_bounds, "k_bounds", 4, "[num_blocks, n_kv_heads, 2, head_dim]")[:2]
    mb = _dims(block_table, "block_table", 2, "[B, max_blocks]")[1]
    dev = q.device
    _check(q, "q", torch.bfloat16, (B, Hq, D), dev)
    _check(k_bounds, "k_bounds", torch.bfloat16, (nb, H, 2, D), dev)
    _check(block_table, "block_table", torch.int32, (B, mb), dev)
    _check(seq_lens, "seq_lens", torch.int32, (B,), dev)
    _fits(block_size, keep, keep_first, keep_last)
    nbytes = _select_bytes(B, Hq, H, D, mb, block_size, keep)
    workspace = _scratch(workspace, nbytes, "mova_block_select", dev)
    if sel_blocks is None:
        sel_blocks = block_table.new_empty((B, H, keep))
    else:
        _check(sel_blocks, "sel_blocks", torch.int32, (B, H, keep), dev)
    _launch(lib.mova_block_select, "mova_block_select", dev, _ptr(q), _ptr(k_bounds), nb,
            block_size, _ptr(block_table), mb, _ptr(seq_lens), B, Hq, H, D, keep, keep_first,
            keep_last, _ptr(sel_blocks), _ptr(workspace),
            workspace.numel())
    return sel_blocks


def attention_workspace_bytes(B: int, n_heads: int, n_kv_heads: int, head_dim: int,
                              max_blocks: int, block_size: int, keep: int = 0) -> int:
    _fits(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep)
    n = _attention_bytes(B, n_heads, n_kv_heads, head_dim, max_blocks, block_size, keep)
    if n == ctypes.c_size_t(-1).value:
        raise MovaError(-2, "mova_attention_workspace_bytes")
    return n


def attention_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_table: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                    k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, window: int = 0,
                    sel_blocks: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_attention_paged: one new token per request attending over the
    paged cache; returns bf16 [B, n_heads, head_dim].

    ``window`` > 0 keeps the last ``window`` positions, ``sel_blocks`` (int32
    [B, n_kv_heads, keep], as from ``block_select``) the listed blocks;
    ``lse`` (float32 [B, n_heads]) receives the log-sum-exp of the logits.
    ``workspace`` (optional uint8 tensor) is reused when large enough
    (``attention_workspace_bytes``); else one is allocated."""
    lib = load_library()
    B, Hq, D = _dims(q, "q", 3, "[B, n_heads, head_dim]")
    nb, bs, H, _ = _dims(k_cache, "k_cache", 4, "[num_blocks, block_size, n_kv_heads, head_dim]")
    mb = _dims(block_table, "block_table", 2, "[B, max_blocks]")[1]
    dev = q.device
    _check(q, "q", torch.bfloat16, (B, Hq, D), dev)
    dtype = _check_pool(k_cache, "k_cache", (nb, bs, H, D), dev)
    if _check_pool(v_cache, "v_cache", (nb, bs, H, D), dev) != dtype:
        raise ValueError("the pools must have the same dtype")
    _check(block_table, "block_table", torch.int32, (B, mb), dev)
    _check(seq_lens, "seq_lens", torch.int32, (B,), dev)
    _check_scales(k_scale, v_scale, H, dev)
    keep = 0
    if sel_blocks is not None:
        keep = _dims(sel_blocks, "sel_blocks", 3, "[B, n_kv_heads, keep]")[2]
        _check(sel_blocks, "sel_blocks", torch.int32, (B, H, keep), dev)
        if keep == 0:
            raise ValueError("sel_blocks lists no blocks")
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, Hq), dev)
    nbytes = _attention_bytes(B, Hq, H, D, mb, bs, keep)
    workspace = _scratch(workspace, nbytes, "mova_attention_paged", dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out", torch.bfloat16, (B, Hq, D), dev)
    _launch(lib.mova_attention_paged, "mova_attention_paged", dev, _ptr(q), _ptr(k_cache),
            _ptr(v_cache), dtype, _ptr(k_scale), _ptr(v_scale), nb, bs, _ptr(block_table), mb,
            _ptr(seq_lens), _ptr(sel_blocks), keep, B, Hq, H, D, float(scale),
            max(-1, min(int(window), _INT_MAX)), _ptr(out), _ptr(lse), _ptr(workspace),
            workspace.numel())
    return out


@functools.lru_cache(maxsize=1024)
def _chunk_bytes(*sizes: int) -> int:
    return load_library().mova_attention_chunk_workspace_bytes(*sizes)


def attention_chunk_workspace_bytes(T: int, B: int, n_heads: int, n_kv_heads: int, head_dim: int,
                                    max_blocks: int, block_size: int) -> int:
    _fits(T, B, n_heads, n_kv_heads, head_dim, max_blocks, block_size)
    n = _chunk_bytes(T, B, n_heads, n_kv_heads, head_dim, max_blocks, block_size)
    if n == _NO_SIZE:
        raise MovaError(-2, "mova_attention_chunk_workspace_bytes")
    return n


def attention_chunk_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_table: torch.Tensor, cached_lens: torch.Tensor,
                          seq_lens: torch.Tensor, cu_new: torch.Tensor, scale: float,
                          k_scale: Optional[torch.Tensor] = None,
                          v_scale: Optional[torch.Tensor] = None, window: int = 0,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mova_attention_chunk_paged: the new tokens of each request attending
    over the paged cache that already holds them; returns bf16 [T, n_heads,
    head_dim].

    Rows ``cu_new[b]`` up to ``cu_new[b + 1]`` of ``q`` are request b's, at
    positions from ``cached_lens[b]`` on; each sees the positions up to its
    own (``window`` > 0: the last ``window`` of them).  Rows at or past
    ``seq_lens[b]`` give zeros; rows that belong to no request are not
    written.  With ``paged_plan``: its ``cached_lens`` argument and the
    ``seq_lens`` and ``cu_new`` that it returns.  ``lse`` (float32 [T,
    n_heads]) receives the log-sum-exp of the logits; ``workspace`` (optional
    uint8 tensor) is reused when large enough
    (``attention_chunk_workspace_bytes``); else one is allocated."""
    lib = load_library()
    T, Hq, D = _dims(q, "q", 3, "[T, n_heads, head_dim]")
    nb, bs, H, _ = _dims(k_cache, "k_cache", 4, "[num_blocks, block_size, n_kv_heads, head_dim]")
    B, mb = _dims(block_table, "block_table", 2, "[B, max_blocks]")
    dev = q.device
    _check(q, "q", torch.bfloat16, (T, Hq, D), dev)
    dtype = _check_pool(k_cache, "k_cache", (nb, bs, H, D), dev)
    if _check_pool(v_cache, "v_cache", (nb, bs, H, D), dev) != dtype:
        raise ValueError("the pools must have the same dtype")
    _check(block_table, "block_table", torch.int32, (B, mb), dev)
    _check(cached_lens, "cached_lens", torch.int32, (B,), dev)
    _check(seq_lens, "seq_lens", torch.int32, (B,), dev)
    _check(cu_new, "cu_new", torch.int32, (B + 1,), dev)
    _check_scales(k_scale, v_scale, H, dev)
    if lse is not None:
        _check(lse, "lse", torch.float32, (T, Hq), dev)
    workspace = _scratch(workspace, _chunk_bytes(T, B, Hq, H, D, mb, bs),
                         "mova_attention_chunk_paged", dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out", torch.bfloat16, (T, Hq, D), dev)
    _launch(lib.mova_attention_chunk_paged, "mova_attention_chunk_paged", dev, _ptr(q),
            _ptr(k_cache), _ptr(v_cache), dtype, _ptr(k_scale), _ptr(v_scale), nb, bs,
            _ptr(block_table), mb, _ptr(cached_lens), _ptr(seq_lens), _ptr(cu_new), T, B, Hq, H, D,
            float(scale), max(-1, min(int(window), _INT_MAX)), _ptr(out), _ptr(lse),
            _ptr(workspace), workspace.numel())
    return out


class PagedFork(NamedTuple):
    """Outputs of ``paged_fork``."""
    seq_lens: torch.Tensor    # int32 [B]
    copy_src: torch.Tensor    # int32 [n]
    copy_dst: torch.Tensor    # int32 [n]
    free_count: torch.Tensor  # int32 [1]


class PagedFree(NamedTuple):
    """Outputs of ``paged_free``."""
    seq_lens: torch.Tensor    # int32 [B]
    free_count: torch.Tensor  # int32 [1]


class PagedCompact(NamedTuple):
    """Outputs of ``paged_compact``."""
    block_table: torch.Tensor  # int32 [B, max_blocks]
    free_blocks: torch.Tensor  # int32 [capacity]
    free_count: torch.Tensor   # int32 [1]
    shares: torch.Tensor       # int32 [num_blocks]
    remap: torch.Tensor        # int32 [num_blocks]
    move_src: torch.Tensor     # int32 [num_blocks // 2]
    move_dst: torch.Tensor     # int32 [num_blocks // 2]
    move_count: torch.Tensor   # int32 [1]


def _given(t: Optional[torch.Tensor], name: str, shape, like: torch.Tensor) -> torch.Tensor:
    """An int32 output: the caller's, or a new one."""
    if t is None:
        return like.new_empty(shape)
    _check(t, name, torch.int32, shape, like.device)
    return t


def _upkeep(block_table, free_blocks, free_count, shares, cached_lens, block_size):
    """The checks that the upkeep of the blocks shares."""
    B, mb = _dims(block_table, "block_table", 2, "[B, max_blocks]")
    (cap,) = _dims(free_blocks, "free_blocks", 1, "[capacity]")
    (nb,) = _dims(shares, "shares", 1, "[num_blocks]")
    dev, i32 = block_table.device, torch.int32
    _check(block_table, "block_table", i32, (B, mb), dev)
    _check(free_blocks, "free_blocks", i32, (cap,), dev)
    _check(free_count, "free_count", i32, (1,), dev)
    _check(shares, "shares", i32, (nb,), dev)
    _check(cached_lens, "cached_lens", i32, (B,), dev)
    _fits(block_size)
    return B, mb, cap, nb, dev


def paged_fork(parents: torch.Tensor, children: torch.Tensor, block_size: int,
               block_table: torch.Tensor, cached_lens: torch.Tensor, free_blocks: torch.Tensor,
               free_count: torch.Tensor, shares: torch.Tensor,
               fork_lens: Optional[torch.Tensor] = None, seq_lens: Optional[torch.Tensor] = None,
               copy_src: Optional[torch.Tensor] = None, copy_dst: Optional[torch.Tensor] = None,
               free_count_out: Optional[torch.Tensor] = None) -> PagedFork:
    """mova_paged_fork: rows ``children`` of the block table begin with the
    first ``fork_lens`` tokens (None: all) of rows ``parents`` (int32 [n]).

    Full blocks are shared and counted in ``shares`` (int32 [num_blocks],
    updated in place like ``block_table``); for a last block filled in part a
    free one is taken, and ``copy_src`` and ``copy_dst`` name the two for
    ``paged_copy`` (-1: nothing to copy).  The new lengths and count are new
    tensors."""
    lib = load_library()
    (n,) = _dims(parents, "parents", 1, "[n]")
    B, mb, cap, nb, dev = _upkeep(block_table, free_blocks, free_count, shares, cached_lens,
                                  block_size)
    _check(parents, "parents", torch.int32, (n,), dev)
    _check(children, "children", torch.int32, (n,), dev)
    if fork_lens is not None:
        _check(fork_lens, "fork_lens", torch.int32, (n,), dev)
    seq_lens = _given(seq_lens, "seq_lens", (B,), cached_lens)
    copy_src = _given(copy_src, "copy_src", (n,), cached_lens)
    copy_dst = _given(copy_dst, "copy_dst", (n,), cached_lens)
    free_count_out = _given(free_count_out, "free_count_out", (1,), free_count)
    _launch(lib.mova_paged_fork, "mova_paged_fork", dev, _ptr(parents), _ptr(children),
            _ptr(fork_lens), n, _ptr(cached_lens), B, block_size, mb, _ptr(block_table),
            _ptr(free_blocks), cap, _ptr(free_count), _ptr(free_count_out), _ptr(shares), nb,
            _ptr(seq_lens), _ptr(copy_src), _ptr(copy_dst))
    return PagedFork(seq_lens, copy_src, copy_dst, free_count_out)


@functools.lru_cache(maxsize=64)
def _free_bytes(num_blocks: int) -> int:
    return load_library().mova_paged_free_workspace_bytes(num_blocks)


def paged_free(cached_lens: torch.Tensor, keep_lens: torch.Tensor, block_size: int,
               block_table: torch.Tensor, free_blocks: torch.Tensor, free_count: torch.Tensor,
               shares: torch.Tensor, seq_lens: Optional[torch.Tensor] = None,
               free_count_out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> PagedFree:
    """mova_paged_free: each row keeps its first ``keep_lens`` tokens (0 ends
    the request) and lets go of the blocks behind them; a block's last holder
    puts it on the free stack.  ``free_blocks`` and ``shares`` are updated in
    place; the new lengths and count are new tensors.  A row that would be cut
    inside a block that others hold too keeps its length."""
    lib = load_library()
    B, mb, cap, nb, dev = _upkeep(block_table, free_blocks, free_count, shares, cached_lens,
                                  block_size)
    _check(keep_lens, "keep_lens", torch.int32, (B,), dev)
    seq_lens = _given(seq_lens, "seq_lens", (B,), cached_lens)
    free_count_out = _given(free_count_out, "free_count_out", (1,), free_count)
    workspace = _scratch(workspace, _free_bytes(nb), "mova_paged_free", dev)
    _launch(lib.mova_paged_free, "mova_paged_free", dev, _ptr(cached_lens), _ptr(keep_lens), B,
            block_size, mb, _ptr(block_table), _ptr(free_blocks), cap, _ptr(free_count),
            _ptr(free_count_out), _ptr(shares), nb, _ptr(seq_lens), _ptr(workspace),
            workspace.numel())
    return PagedFree(seq_lens, free_count_out)


@functools.lru_cache(maxsize=64)
def _compact_bytes(num_blocks: int) -> int:
    return load_library().mova_paged_compact_workspace_bytes(num_blocks)


def paged_compact(cached_lens: torch.Tensor, block_size: int, block_table: torch.Tensor,
                  free_blocks: torch.Tensor, free_count: torch.Tensor, shares: torch.Tensor,
                  limit: int = 0, block_table_out: Optional[torch.Tensor] = None,
                  free_blocks_out: Optional[torch.Tensor] = None,
                  shares_out: Optional[torch.Tensor] = None,
                  remap: Optional[torch.Tensor] = None, move_src: Optional[torch.Tensor] = None,
                  move_dst: Optional[torch.Tensor] = None,
                  move_count: Optional[torch.Tensor] = None,
                  free_count_out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> PagedCompact:
    """mova_paged_compact: blocks in use at or above max(``limit``, their
    number) go to the lowest free ones.  ``block_table``, ``free_blocks`` and
    ``shares`` are updated in place unless other tensors are given for the new
    ones; ``move_src``, ``move_dst`` and ``move_count`` are the list for
    ``paged_copy``, ``remap`` gives every block's new place (-1: free)."""
    lib = load_library()
    B, mb, cap, nb, dev = _upkeep(block_table, free_blocks, free_count, shares, cached_lens,
                                  block_size)
    _fits(limit)
    if block_table_out is None:
        block_table_out = block_table
    else:
        _check(block_table_out, "block_table_out", torch.int32, (B, mb), dev)
    if free_blocks_out is None:
        free_blocks_out = free_blocks
    else:
        _check(free_blocks_out, "free_blocks_out", torch.int32, (cap,), dev)
    if shares_out is None:
        shares_out = shares
    else:
        _check(shares_out, "shares_out", torch.int32, (nb,), dev)
    remap = _given(remap, "remap", (nb,), shares)
    move_src = _given(move_src, "move_src", (nb // 2,), shares)
    move_dst = _given(move_dst, "move_dst", (nb // 2,), shares)
    move_count = _given(move_count, "move_count", (1,), free_count)
    free_count_out = _given(free_count_out, "free_count_out", (1,), free_count)
    workspace = _scratch(workspace, _compact_bytes(nb), "mova_paged_compact", dev)
    _launch(lib.mova_paged_compact, "mova_paged_compact", dev, _ptr(cached_lens), B, block_size,
            mb, _ptr(block_table), _ptr(block_table_out), _ptr(free_blocks), _ptr(free_blocks_out),
            cap, _ptr(free_count), _ptr(free_count_out), _ptr(shares), _ptr(shares_out), nb, limit,
            _ptr(remap), _ptr(move_src), _ptr(move_dst), _ptr(move_count), _ptr(workspace),
            workspace.numel())
    return PagedCompact(block_table_out, free_blocks_out, free_count_out, shares_out, remap,
                        move_src, move_dst, move_count)


def paged_copy(copy_src: torch.Tensor, copy_dst: torch.Tensor, k_cache: Optional[torch.Tensor],
               v_cache: Optional[torch.Tensor] = None, k_bounds: Optional[torch.Tensor] = None,
               count: Optional[torch.Tensor] = None) -> None:
    """mova_paged_copy: block ``copy_dst[i]`` of each pool given becomes as
    block ``copy_src[i]`` (int32 [n], as from ``paged_fork`` or
    ``paged_compact``); pairs outside the pool, and those behind ``count``
    (int32 [1], None: n), are passed over.  Any of the keys, values and bounds
    may be left out, as long as one is there."""
    lib = load_library()
    (n,) = _dims(copy_src, "copy_src", 1, "[n]")
    dev = copy_src.device
    pool = k_cache if k_cache is not None else v_cache
    if pool is not None:
        nb, bs, H, D = _dims(pool, "the pools", 4, "[num_blocks, block_size, n_kv_heads, head_dim]")
    elif k_bounds is not None:
        nb, H, _, D = _dims(k_bounds, "k_bounds", 4, "[num_blocks, n_kv_heads, 2, head_dim]")
        bs = 1  # (of no account without keys or values)
    else:
        raise ValueError("neither keys, values nor bounds are given")
    dtype = CACHE_DTYPES.get(torch.bfloat16 if pool is None else pool.dtype)
    for p, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if p is not None and _check_pool(p, name, (nb, bs, H, D), dev) != dtype:
            raise ValueError("the pools must have the same dtype")
    _check(copy_src, "copy_src", torch.int32, (n,), dev)
    _check(copy_dst, "copy_dst", torch.int32, (n,), dev)
    if k_bounds is not None:
        _check(k_bounds, "k_bounds", torch.bfloat16, (nb, H, 2, D), dev)
    if count is not None:
        _check(count, "count", torch.int32, (1,), dev)
    _launch(lib.mova_paged_copy, "mova_paged_copy", dev, _ptr(copy_src), _ptr(copy_dst), n,
            _ptr(count), _ptr(k_cache), _ptr(v_cache), _ptr(k_bounds), dtype, nb, bs, H, D)


# Kernel-choice overrides (mova_debug_override): name -> (key, {value name: value}).
OVERRIDES = {
    "path": (0, {"decode": 1, "grouped": 2}),
    "router": (1, {"16": 1, "32s4": 2, "32s3": 3, "64": 4}),
    "gemm_tile": (2, {"256x256": 1, "128x256": 2, "128x128": 3, "128x128s3": 4,
                      "128x128s4": 5, "128x128w4": 6, "352x256": 7}),
    "dense_path": (3, {"skinny": 1, "tiled": 2}),
    "decode_chain": (4, {"on": 1, "off": 2, "token": 3}),
    "decode_groups": (5, {"1": 1, "2": 2}),
    "serial": (6, {"on": 1}),
}


def set_override(name: str, value: Optional[str]) -> None:
    """Force one kernel choice for later calls (tests, measurements); value
    None restores the automatic choice."""
    key, values = OVERRIDES[name]
    v = 0 if value is None else values[str(value)]
    rc = load_library().mova_debug_override(key, v)
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_debug_override")


def get_override(name: str) -> Optional[str]:
    key, values = OVERRIDES[name]
    v = load_library().mova_debug_override_get(key)
    return None if v == 0 else {i: n for n, i in values.items()}[v]


def clear_overrides() -> None:
    for name in OVERRIDES:
        set_override(name, None)


class overrides:
    """Context manager: ``with overrides(path="grouped"): ...`` forces the
    named choices inside the block and restores the previous ones after."""

    def __init__(self, **kw):
        self.kw = kw
        self.saved = {}

    def __enter__(self):
        for name, value in self.kw.items():
            self.saved[name] = get_override(name)
            set_override(name, value)
        return self

    def __exit__(self, *exc):
        for name, value in self.saved.items():
            set_override(name, value)
        return False


def timing_enable(capacity: int, stages=STAGES) -> None:
    """Record HIP events around the named stages for up to ``capacity`` calls."""
    mask = 0
    for s in stages:
        mask |= 1 << STAGES.index(s)
    rc = load_library().mova_timing_enable(int(capacity), mask)
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_timing_enable")


def timing_read() -> List[Tuple[float, int]]:
    """[(total_ms, launches)] per stage, in the order of ``STAGES``."""
    n = len(STAGES)
    tot = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    rc = load_library().mova_timing_read(n, tot, cnt)
    if rc != MOVA_OK:
        raise MovaError(rc, "mova_timing_read")
    return [(tot[i], cnt[i]) for i in range(n)]
