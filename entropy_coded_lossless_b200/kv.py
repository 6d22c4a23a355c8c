"""Binding of the paged INT8 KV cache (include/shn_kv.h) — tensor checks and argument marshalling only, the calls' in
csrc/kv_binding.cpp (a small batch's kernels take microseconds, and so must what comes before them).

Plan (block tables and slots from request lengths), store (norm, rotation, quantisation into the pages),
load (rows as bf16) and attention over the pages, for packed prompts and for single tokens that share a prefix:

    cache = kv.Cache.empty(n_pages, kv_heads, page_tokens, head_dim, device="cuda")
    work = kv.workspace(kv.WORKSPACE_BYTES, "cuda")
    kv.shn_kv_plan(ctx_len, new_len, page_tokens, table, free, head, head, cu, kv_len, positions, slots, work)
    kv.shn_kv_store(q, k, v, positions, slots, cache, q, work, q_weight=wq, k_weight=wk, cos_sin=angles)
    kv.shn_kv_attn_prompt(q, cache, table, cu, kv_len, scale, out, work)

Calls run on the tensors' device, by default on its current stream, and do not synchronise; errors the device
finds are in the workspace's status word (shn.shn_get_device_status). A page's bytes are a codec segment
(Cache.segments), so pages are compressed, offloaded and reloaded by the calls of ``shn``.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import shn
from .shn import ShnError, _check  # noqa: F401  (ShnError: what the calls raise)

try:
    from . import _kv
except ImportError as e:  # pragma: no cover - not built
    raise ImportError(f"_kv.so not built beside this file ({e}); run python -m entropy_coded_lossless_b200.build") from e

WORKSPACE_BYTES = 256


class _CacheStruct(ctypes.Structure):
    _fields_ = [("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p), ("d_k_scale", ctypes.c_void_p),
                ("d_v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_uint32), ("kv_heads", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32), ("head_dim", ctypes.c_uint32)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = shn.lib()
        u32, u64, i32, vp, sz, f32 = (ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_float)
        C = ctypes.POINTER(_CacheStruct)
        sigs = {
            "shn_kv_check_cache": (i32, [C]),
            "shn_kv_plan": (i32, [vp, vp, u32, u32, vp, u32, vp, u32, vp, vp, vp, vp, vp, vp, u32, vp, sz, vp]),
            "shn_kv_store": (i32, [vp, u64, u32, vp, u64, vp, u64, u32, vp, vp, vp, vp, f32, vp, u32, u32, u32, C, vp,
                                   u64, vp, sz, vp]),
            "shn_kv_load": (i32, [C, vp, u32, vp, u64, vp, u64, vp, sz, vp]),
            "shn_kv_attn_prompt": (i32, [vp, u64, u32, u32, C, vp, u32, vp, vp, u32, f32, vp, u64, vp, sz, vp]),
            "shn_kv_attn_shared_workspace_bytes": (sz, [C, u32, u32]),
            "shn_kv_attn_shared": (i32, [vp, u64, u32, u32, C, vp, u32, vp, vp, u32, vp, f32, vp, u64, vp, sz, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _bound = L
    return _bound


def _dev(t, name, dtype, device, shape=None):
    """Device address of a contiguous tensor of this type on this device (shape: what it must be, where given)."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace for the calls here (its status word zero until the first call)."""
    t = shn.empty_aligned(int(nbytes), device)
    t[:8].zero_()
    return t


class Cache:
    """One layer's paged cache: k, v int8 [n_pages, kv_heads, page_tokens, head_dim] and their float32 scales
    [n_pages, kv_heads, page_tokens], contiguous, on one device. The tensors are the caller's."""

    def __init__(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be int8 [n_pages, kv_heads, page_tokens, head_dim]")
        self.device = _device(k, "k")
        shape = k.shape
        pages, heads, page_tokens, head_dim = shape
        if page_tokens & (page_tokens - 1) or not 16 <= page_tokens <= 1024:
            raise ValueError("page_tokens must be a power of two, 16 .. 1024")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.kv_heads, self.page_tokens, self.head_dim = pages, heads, page_tokens, head_dim
        self.c = _CacheStruct(_dev(k, "k", torch.int8, self.device), _dev(v, "v", torch.int8, self.device, shape),
                              _dev(k_scale, "k_scale", torch.float32, self.device, shape[:3]),
                              _dev(v_scale, "v_scale", torch.float32, self.device, shape[:3]), pages, heads, page_tokens,
                              head_dim)
        _check(_lib().shn_kv_check_cache(ctypes.byref(self.c)), "shn_kv_check_cache")
        self.handle = ctypes.addressof(self.c), self.device.index  # what the calls take (self.c lives as long as this)

    @classmethod
    def empty(cls, n_pages, kv_heads, page_tokens, head_dim, device="cuda"):
        """A cache of zeros (values and scales)."""
        k, v = (torch.zeros(n_pages, kv_heads, page_tokens, head_dim, dtype=torch.int8, device=device) for _ in range(2))
        ks, vs = (torch.zeros(n_pages, kv_heads, page_tokens, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def segments(self, pages):
        """Codec segments of these pages within k (or v) as a flat INT8 tensor."""
        n = self.kv_heads * self.page_tokens * self.head_dim
        return [(int(p) * n, n) for p in pages]

    @property
    def log2_group(self):
        """log2 of the values per scale, as shn.shn_decode_bf16 takes it."""
        return int(math.log2(self.head_dim))


# --------------------------------------------------------------------------------------------
# the calls, one-to-one with the C ABI


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def shn_kv_plan(ctx_len, new_len, page_tokens, block_table, free_pages, free_head, free_next, cu_new, kv_len, positions,
                slots, work, stream=None):
    code = _kv.plan(ctx_len, new_len, page_tokens, block_table, free_pages, free_head, free_next, cu_new, kv_len,
                    positions, slots, work, _raw(stream))
    if code:
        raise ShnError(code, "shn_kv_plan")


def shn_kv_store(q, k, v, positions, slots, cache, q_out, work, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None,
                 pairs=False, stream=None):
    """q and q_out may be None (keys and values only); positions may be None without cos_sin."""
    code = _kv.store(*cache.handle, q, k, v, positions, slots, q_out, work, q_weight, k_weight, eps, cos_sin, pairs,
                     _raw(stream))
    if code:
        raise ShnError(code, "shn_kv_store")


def shn_kv_load(cache, slots, k_out, v_out, work, stream=None):
    """k_out or v_out may be None."""
    code = _kv.load(*cache.handle, slots, k_out, v_out, work, _raw(stream))
    if code:
        raise ShnError(code, "shn_kv_load")


def shn_kv_attn_prompt(q, cache, block_table, cu_q, kv_len, scale, out, work, stream=None):
    code = _kv.attn_prompt(*cache.handle, q, block_table, cu_q, kv_len, scale, out, work, _raw(stream))
    if code:
        raise ShnError(code, "shn_kv_attn_prompt")


def attn_shared_workspace_bytes(cache, n_reqs: int, q_heads: int) -> int:
    return int(_lib().shn_kv_attn_shared_workspace_bytes(ctypes.byref(cache.c), n_reqs, q_heads))


def shn_kv_attn_shared(q, cache, prefix_pages, prefix_len, block_table, kv_len, scale, out, work, stream=None):
    """q, out: [requests, heads, head_dim]. prefix_pages may be None (then prefix_len holds 0)."""
    code = _kv.attn_shared(*cache.handle, q, prefix_pages, prefix_len, block_table, kv_len, scale, out, work, _raw(stream))
    if code:
        raise ShnError(code, "shn_kv_attn_shared")
