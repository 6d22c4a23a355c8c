"""ctypes binding of the paged INT8 KV cache (include/shn_kv.h) — argument marshalling only.

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

WORKSPACE_BYTES = 256
_I32, _BF16 = torch.int32, torch.bfloat16


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


class _on:
    """The device of a call made current around it, where it is not, and the stream the call runs on."""

    __slots__ = ("device", "guard", "stream")

    def __init__(self, device, stream):
        self.device = device
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        self.stream = (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.stream

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


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


def _rows(t, name, device, head_dim, heads=None, tokens=None):
    """Address and token stride of bf16 rows [tokens, heads, head_dim] whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != _BF16 or t.dim() != 3:
        raise ValueError(f"{name} must be bfloat16 [tokens, heads, head_dim]")
    n, h, d = t.shape
    if d != head_dim or (heads is not None and h != heads) or (tokens is not None and n != tokens):
        raise ValueError(f"{name} has the shape {tuple(t.shape)}; expected [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {head_dim}]")
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if n <= 1:
        st = h * d  # the stride of a single token means nothing
    if st < 0 or (n > 1 and st < h * d):
        raise ValueError(f"{name}: tokens overlap")
    return t.data_ptr(), st


def _work(t, device):
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError(f"work must be a contiguous uint8 tensor on {device}")
    return t.data_ptr(), t.numel()


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


def shn_kv_plan(ctx_len, new_len, page_tokens, block_table, free_pages, free_head, free_next, cu_new, kv_len, positions,
                slots, work, stream=None):
    dev = _device(ctx_len, "ctx_len")
    n = ctx_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"block_table must be [{n}, max_blocks]")
    if positions.shape != slots.shape:
        raise ValueError("positions and slots must have the same length")
    w, nw = _work(work, dev)
    with _on(dev, stream) as s:
        _check(_lib().shn_kv_plan(
            _dev(ctx_len, "ctx_len", _I32, dev, (n,)), _dev(new_len, "new_len", _I32, dev, (n,)), n, page_tokens,
            _dev(block_table, "block_table", _I32, dev), block_table.shape[1], _dev(free_pages, "free_pages", _I32, dev),
            free_pages.numel(), _dev(free_head, "free_head", _I32, dev, (1,)), _dev(free_next, "free_next", _I32, dev, (1,)),
            _dev(cu_new, "cu_new", _I32, dev, (n + 1,)), _dev(kv_len, "kv_len", _I32, dev, (n,)),
            _dev(positions, "positions", _I32, dev), _dev(slots, "slots", _I32, dev), slots.numel(), w, nw, s), "shn_kv_plan")


def shn_kv_store(q, k, v, positions, slots, cache, q_out, work, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None,
                 pairs=False, stream=None):
    """q and q_out may be None (keys and values only); positions may be None without cos_sin."""
    dev, d, hk, c = cache.device, cache.head_dim, cache.kv_heads, cache.c
    kp, ks = _rows(k, "k", dev, d, hk)
    n = k.shape[0]
    vp, vs = _rows(v, "v", dev, d, hk, n)
    qp, qs, op, os_, h = None, 0, None, 0, 0
    if q is not None:
        qp, qs = _rows(q, "q", dev, d, tokens=n)
        h = q.shape[1]
        op, os_ = _rows(q_out, "q_out", dev, d, h, n)
    if cos_sin is not None and cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rot_dim]")
    w, nw = _work(work, dev)
    with _on(dev, stream) as s:
        _check(_lib().shn_kv_store(
            qp, qs, h, kp, ks, vp, vs, n, None if positions is None else _dev(positions, "positions", _I32, dev, (n,)),
            _dev(slots, "slots", _I32, dev, (n,)), None if q_weight is None else _dev(q_weight, "q_weight", _BF16, dev, (d,)),
            None if k_weight is None else _dev(k_weight, "k_weight", _BF16, dev, (d,)), eps,
            None if cos_sin is None else _dev(cos_sin, "cos_sin", torch.float32, dev),
            0 if cos_sin is None else cos_sin.shape[0], 0 if cos_sin is None else cos_sin.shape[1], int(bool(pairs)),
            ctypes.byref(c), op, os_, w, nw, s), "shn_kv_store")


def shn_kv_load(cache, slots, k_out, v_out, work, stream=None):
    """k_out or v_out may be None."""
    dev, d, hk = cache.device, cache.head_dim, cache.kv_heads
    n = slots.numel()
    kp, ks = (None, 0) if k_out is None else _rows(k_out, "k_out", dev, d, hk, n)
    vp, vs = (None, 0) if v_out is None else _rows(v_out, "v_out", dev, d, hk, n)
    w, nw = _work(work, dev)
    with _on(dev, stream) as s:
        _check(_lib().shn_kv_load(ctypes.byref(cache.c), _dev(slots, "slots", _I32, dev), n, kp, ks, vp, vs, w, nw, s),
               "shn_kv_load")


def _attn(q, cache, block_table, kv_len, out):
    dev, d = cache.device, cache.head_dim
    qp, qs = _rows(q, "q", dev, d)
    n, h = q.shape[:2]
    op, os_ = _rows(out, "out", dev, d, h, n)
    b = kv_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, max_blocks]")
    return dev, qp, qs, n, h, op, os_, b, _dev(block_table, "block_table", _I32, dev), _dev(kv_len, "kv_len", _I32, dev)


def shn_kv_attn_prompt(q, cache, block_table, cu_q, kv_len, scale, out, work, stream=None):
    dev, qp, qs, n, h, op, os_, b, tp, lp = _attn(q, cache, block_table, kv_len, out)
    w, nw = _work(work, dev)
    with _on(dev, stream) as s:
        _check(_lib().shn_kv_attn_prompt(qp, qs, n, h, ctypes.byref(cache.c), tp, block_table.shape[1],
                                         _dev(cu_q, "cu_q", _I32, dev, (b + 1,)), lp, b, scale, op, os_, w, nw, s),
               "shn_kv_attn_prompt")


def attn_shared_workspace_bytes(cache, n_reqs: int, q_heads: int) -> int:
    return int(_lib().shn_kv_attn_shared_workspace_bytes(ctypes.byref(cache.c), n_reqs, q_heads))


def shn_kv_attn_shared(q, cache, prefix_pages, prefix_len, block_table, kv_len, scale, out, work, stream=None):
    """q, out: [requests, heads, head_dim]. prefix_pages may be None (then prefix_len holds 0)."""
    dev, qp, qs, n, h, op, os_, b, tp, lp = _attn(q, cache, block_table, kv_len, out)
    if n != b:
        raise ValueError(f"q has {n} queries for {b} requests")
    w, nw = _work(work, dev)
    with _on(dev, stream) as s:
        _check(_lib().shn_kv_attn_shared(qp, qs, n, h, ctypes.byref(cache.c),
                                         None if prefix_pages is None else _dev(prefix_pages, "prefix_pages", _I32, dev),
                                         0 if prefix_pages is None else prefix_pages.numel(),
                                         _dev(prefix_len, "prefix_len", _I32, dev, (1,)), tp, block_table.shape[1], lp,
                                         scale, op, os_, w, nw, s), "shn_kv_attn_shared")
