"""Thin ctypes binding of ``libmla.so`` (declared in ``include/mla.h``).

Argument marshalling only: torch provides device memory and the current CUDA
stream, every computation runs in the library's kernels.  There is no fallback:
if the library is missing or a call fails, an exception says so.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from . import build as _build

_lib = None


class MLAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (status {code})")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("s_q", ctypes.c_int), ("d_c", ctypes.c_int),
                ("d_rope", ctypes.c_int), ("d_nope", ctypes.c_int), ("d_v", ctypes.c_int),
                ("scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("seq_stride", ctypes.c_longlong), ("capacity", ctypes.c_int),
                ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int),
                ("kv_dtype", ctypes.c_int), ("kv_scale", ctypes.c_float)]


KV_BF16, KV_E4M3, KV_E4M3_BLOCKS = 0, 1, 3
ABI_VERSION = 2
SPLITS_BALANCED = -1  # num_splits asking for the balanced plan (MLA_SPLITS_BALANCED)


EXPORTS = ("mla_status_string", "mla_abi_version", "mla_absorb_q", "mla_decode_workspace_size",
           "mla_decode_num_splits", "mla_decode_attn", "mla_out_proj", "mla_naive_workspace_size",
           "mla_naive_decode", "mla_read_status", "mla_decode_attn_noalloc", "mla_cache_append_workspace_size",
           "mla_cache_append", "mla_decode_sparse_workspace_size", "mla_decode_attn_sparse", "mla_prefill_crossover",
           "mla_prefill_expand_workspace_size", "mla_prefill_expand", "mla_prefill_workspace_size", "mla_prefill",
           "mla_decode_step", "mla_set_wait_limit_ns", "mla_rope_init", "mla_rope", "mla_pages_update",
           "mla_latent_store", "mla_linear_workspace_size", "mla_linear", "mla_linear_status",
           "mla_linear_query_cut", "mla_latent_row_bytes", "mla_latent_load", "mla_quantize", "mla_linear_fp8",
           "mla_linear_fp8_query_cut")
PATH_ABSORB, PATH_EXPAND = 0, 1
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4


class RopeConfig(ctypes.Structure):
    _fields_ = [("d_rope", ctypes.c_int), ("layout", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_len", ctypes.c_int), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("mscale", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class RopePlan(ctypes.Structure):
    _fields_ = [("d_rope", ctypes.c_int), ("layout", ctypes.c_int), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int), ("turn", ctypes.c_ulonglong * 32)]


class PagePool(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("block_table", ctypes.c_void_p), ("free_ring", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("state_out", ctypes.c_void_p)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int), ("act", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong),
                ("residual_stride", ctypes.c_longlong)]


class QuantizeDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("K", ctypes.c_int), ("block_rows", ctypes.c_int), ("x_stride", ctypes.c_longlong),
                ("code_stride", ctypes.c_longlong), ("scale_stride", ctypes.c_longlong)]


class LinearFp8Desc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int), ("act", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("x_scale_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong),
                ("residual_stride", ctypes.c_longlong)]


class LinearCut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tile_rows", "tile_columns", "k_parts", "runs", "ctas")]


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Open libmla.so (it must have been built: ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"MLA CUDA library not built ({p}); run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    pd, pc = ctypes.POINTER(Dims), ctypes.POINTER(Cache)
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [I]
    lib.mla_abi_version.restype = I
    lib.mla_absorb_q.argtypes = [pd, P, P, P, P, P]
    lib.mla_absorb_q.restype = I
    lib.mla_decode_workspace_size.argtypes = [pd, pc, I]
    lib.mla_decode_workspace_size.restype = SZ
    lib.mla_decode_num_splits.argtypes = [pd, pc]
    lib.mla_decode_num_splits.restype = I
    lib.mla_decode_attn.argtypes = [pd, P, pc, P, P, P, SZ, I, P]
    lib.mla_decode_attn.restype = I
    lib.mla_out_proj.argtypes = [pd, P, P, P, P]
    lib.mla_out_proj.restype = I
    lib.mla_naive_workspace_size.argtypes = [pd, pc]
    lib.mla_naive_workspace_size.restype = SZ
    lib.mla_naive_decode.argtypes = [pd, P, P, pc, P, P, P, P, P, SZ, P]
    lib.mla_naive_decode.restype = I
    lib.mla_decode_sparse_workspace_size.argtypes = [pd, pc, I, I]
    lib.mla_decode_sparse_workspace_size.restype = SZ
    lib.mla_decode_attn_sparse.argtypes = [pd, P, pc, P, I, P, P, P, SZ, I, P]
    lib.mla_decode_attn_sparse.restype = I
    lib.mla_cache_append_workspace_size.argtypes = [pd, I]
    lib.mla_cache_append_workspace_size.restype = SZ
    lib.mla_cache_append.argtypes = [pd, I, P, P, P, pc, P, SZ, P]
    lib.mla_cache_append.restype = I
    lib.mla_read_status.argtypes = [P, ctypes.POINTER(I), P]
    lib.mla_read_status.restype = I
    lib.mla_decode_step.argtypes = [pd, P, P, pc, P, P, P, P, P, P, P, SZ, I, P]
    lib.mla_decode_step.restype = I
    lib.mla_prefill_crossover.argtypes = [pd, ctypes.c_longlong]
    lib.mla_prefill_crossover.restype = ctypes.c_double
    lib.mla_prefill_expand_workspace_size.argtypes = [pd, pc]
    lib.mla_prefill_expand_workspace_size.restype = SZ
    lib.mla_prefill_expand.argtypes = [pd, P, P, pc, P, P, P, P, P, SZ, P]
    lib.mla_prefill_expand.restype = I
    lib.mla_prefill_workspace_size.argtypes = [pd, pc]
    lib.mla_prefill_workspace_size.restype = SZ
    lib.mla_prefill.argtypes = [pd, P, P, pc, P, P, P, P, P, SZ, ctypes.POINTER(I), P]
    lib.mla_prefill.restype = I
    lib.mla_decode_attn_noalloc.argtypes = [pd, P, pc, P, P, I, P, P]
    lib.mla_decode_attn_noalloc.restype = I
    lib.mla_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.mla_set_wait_limit_ns.restype = I
    LL, pr, pp, pl = ctypes.c_longlong, ctypes.POINTER(RopePlan), ctypes.POINTER(PagePool), ctypes.POINTER(LinearDesc)
    lib.mla_rope_init.argtypes = [ctypes.POINTER(RopeConfig), pr]
    lib.mla_rope_init.restype = I
    lib.mla_rope.argtypes = [pd, pr, P, LL, LL, P, P, P, P, I, P]
    lib.mla_rope.restype = I
    lib.mla_pages_update.argtypes = [pp, P, P, I, P, P, P, P, P, P]
    lib.mla_pages_update.restype = I
    lib.mla_latent_store.argtypes = [pd, pr, P, LL, P, ctypes.c_float, P, P, pc, P, P]
    lib.mla_latent_store.restype = I
    lib.mla_linear_workspace_size.argtypes = [pl]
    lib.mla_linear_workspace_size.restype = SZ
    lib.mla_linear.argtypes = [pl, P, P, P, P, P, P, SZ, P]
    lib.mla_linear.restype = I
    lib.mla_linear_status.argtypes = [pl, P, P, P, P, P, P, SZ, P, P]
    lib.mla_linear_status.restype = I
    lib.mla_linear_query_cut.argtypes = [pl, ctypes.POINTER(LinearCut)]
    lib.mla_linear_query_cut.restype = I
    pq, pf = ctypes.POINTER(QuantizeDesc), ctypes.POINTER(LinearFp8Desc)
    lib.mla_latent_row_bytes.argtypes = [pd]
    lib.mla_latent_row_bytes.restype = LL
    lib.mla_latent_load.argtypes = [pd, pc, I, P, P, LL, P, P]
    lib.mla_latent_load.restype = I
    lib.mla_quantize.argtypes = [pq, P, P, ctypes.c_float, P, P, P]
    lib.mla_quantize.restype = I
    lib.mla_linear_fp8.argtypes = [pf, P, P, P, P, P, P, P, P, P]
    lib.mla_linear_fp8.restype = I
    lib.mla_linear_fp8_query_cut.argtypes = [pf, ctypes.POINTER(LinearCut)]
    lib.mla_linear_fp8_query_cut.restype = I
    if path is None:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().mla_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != 0:
        raise MLAError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class Problem:
    """Sizes of one decode step (mirrors ``mla_dims``)."""
    __slots__ = ("__dict__", "__weakref__", "_kept")  # _kept: what dims_ref() made, beside the fields
    B: int
    H: int
    s_q: int
    d_c: int
    d_rope: int
    d_nope: int
    d_v: int
    scale: float

    def __getstate__(self):  # copies and pickles take the fields alone
        return dict(self.__dict__)

    def dims_ref(self):
        """A reference to ``dims()`` for ctypes, made once until a field changes."""
        kept = getattr(self, "_kept", None)
        if kept is None or kept[0] != self.__dict__:
            # made from one snapshot and kept with it: a field set meanwhile shows at the next call
            seen = dict(self.__dict__)
            kept = self._kept = seen, ctypes.byref(Dims(*[float(seen[n]) if n == "scale" else seen[n] for n, _ in Dims._fields_]))
        return kept[1]

    def dims(self) -> Dims:
        return Dims(self.B, self.H, self.s_q, self.d_c, self.d_rope, self.d_nope, self.d_v, float(self.scale))

    @classmethod
    def of(cls, cfg) -> "Problem":
        return cls(cfg.B, cfg.H, cfg.s_q, cfg.d_c, cfg.d_rope, cfg.d_nope, cfg.d_v, cfg.scale)


def make_cache(prob: Problem, kv: torch.Tensor, seq_lens: torch.Tensor, block_table=None,
               page_size: int = 64, max_seq_len: int = 0, kv_scale: float | None = None) -> Cache:
    """Cache descriptor for a contiguous [B, T_max, W] (any sequence stride) or paged
    [P, page, W] latent cache already on the device: bf16 values, or FP8 E4M3 codes
    (uint8 or float8_e4m3fn) with their ``kv_scale`` (value = kv_scale * code), or uint8 rows
    of ``latent_row_bytes`` (codes, a scale a block of 128, keys in bf16: no ``kv_scale``)."""
    W = prob.d_c + prob.d_rope
    blocks = kv.dtype == torch.uint8 and kv.shape[-1] == prob.d_c + 16 + 2 * prob.d_rope
    if blocks:
        W = kv.shape[-1]
    fp8 = kv.dtype in (torch.uint8, torch.float8_e4m3fn)
    if (kv.dtype != torch.bfloat16 and not fp8) or kv.shape[-1] != W or kv.stride(-1) != 1:
        raise ValueError("kv must be bf16 or FP8 codes with rows of d_c + d_rope contiguous values")
    if fp8 and not blocks and kv_scale is None:
        raise ValueError("an FP8 cache needs its kv_scale")
    if blocks and kv_scale is not None:
        raise ValueError(f"uint8 rows of {W} bytes are blocks with scales of their own: they have no kv_scale")
    dt, sc = (KV_E4M3_BLOCKS, 1.0) if blocks else (KV_E4M3, float(kv_scale)) if fp8 else (KV_BF16, 1.0)
    if block_table is None:
        if kv.dim() != 3 or kv.stride(1) != W:
            raise ValueError("contiguous kv must be [B, T_max, W] with dense token rows")
        return Cache(kv.data_ptr(), kv.stride(0), kv.shape[1], None, 0, page_size, 0,
                     seq_lens.data_ptr(), int(max_seq_len), dt, sc)
    if not kv.is_contiguous() or kv.dim() != 3:
        raise ValueError("paged kv must be a dense [P, page, W] pool")
    if block_table.dtype != torch.int32 or not block_table.is_contiguous():
        raise ValueError("block_table must be a dense int32 [B, max_pages] tensor")
    return Cache(kv.data_ptr(), 0, 0, block_table.data_ptr(), block_table.shape[1], kv.shape[1],
                 kv.shape[0], seq_lens.data_ptr(), int(max_seq_len), dt, sc)


# ---------------------------------------------------------------------------- entry points
def absorb_q(prob: Problem, q_nope, q_rope, w_uk, q_cat=None, stream=None):
    lib = load()
    if q_cat is None:
        q_cat = torch.empty(prob.B, prob.s_q, prob.H, prob.d_c + prob.d_rope, dtype=torch.bfloat16,
                            device=q_nope.device)
    d = prob.dims()
    _check(lib.mla_absorb_q(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), _ptr(w_uk), _ptr(q_cat),
                            _stream(stream)), "mla_absorb_q")
    return q_cat


def decode_workspace_size(prob: Problem, cache: Cache, num_splits: int = 0) -> int:
    d = prob.dims()
    n = load().mla_decode_workspace_size(ctypes.byref(d), ctypes.byref(cache), int(num_splits))
    if n == 0:
        raise ValueError("mla_decode_workspace_size rejected the arguments")
    return int(n)


def decode_num_splits(prob: Problem, cache: Cache) -> int:
    d = prob.dims()
    return int(load().mla_decode_num_splits(ctypes.byref(d), ctypes.byref(cache)))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def decode_attn(prob: Problem, q_cat, cache: Cache, o_lat=None, lse=None, workspace=None, num_splits: int = 0,
                stream=None):
    lib = load()
    dev = q_cat.device
    if o_lat is None:
        o_lat = torch.empty(prob.B, prob.s_q, prob.H, prob.d_c, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(prob.B, prob.s_q, prob.H, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_workspace_size(prob, cache, num_splits), dev)
    d = prob.dims()
    _check(lib.mla_decode_attn(ctypes.byref(d), _ptr(q_cat), ctypes.byref(cache), _ptr(o_lat), _ptr(lse),
                               _ptr(workspace), workspace.numel(), int(num_splits), _stream(stream)),
           "mla_decode_attn")
    return o_lat, lse, workspace


def out_proj(prob: Problem, o_lat, w_uv, out=None, stream=None):
    lib = load()
    if out is None:
        out = torch.empty(prob.B, prob.s_q, prob.H, prob.d_v, dtype=torch.bfloat16, device=o_lat.device)
    d = prob.dims()
    _check(lib.mla_out_proj(ctypes.byref(d), _ptr(o_lat), _ptr(w_uv), _ptr(out), _stream(stream)),
           "mla_out_proj")
    return out


def decode_sparse_workspace_size(prob: Problem, cache: Cache, topk: int, num_splits: int = 0) -> int:
    d = prob.dims()
    n = load().mla_decode_sparse_workspace_size(ctypes.byref(d), ctypes.byref(cache), int(topk), int(num_splits))
    if n == 0:
        raise ValueError("mla_decode_sparse_workspace_size rejected the arguments")
    return int(n)


def decode_attn_sparse(prob: Problem, q_cat, cache: Cache, indices, num_splits: int = 0, o_lat=None, lse=None,
                       workspace=None, stream=None):
    """mla_decode_attn_sparse: attention over the listed tokens (indices int32 [B, s_q, topk])."""
    lib = load()
    dev = q_cat.device
    topk = int(indices.shape[-1])
    if o_lat is None:
        o_lat = torch.empty(prob.B, prob.s_q, prob.H, prob.d_c, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(prob.B, prob.s_q, prob.H, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_sparse_workspace_size(prob, cache, topk, num_splits), dev)
    d = prob.dims()
    _check(lib.mla_decode_attn_sparse(ctypes.byref(d), _ptr(q_cat), ctypes.byref(cache), _ptr(indices), topk,
                                      _ptr(o_lat), _ptr(lse), _ptr(workspace), workspace.numel(), int(num_splits),
                                      _stream(stream)), "mla_decode_attn_sparse")
    return o_lat, lse, workspace


def cache_append_workspace_size(prob: Problem, d_model: int) -> int:
    d = prob.dims()
    n = load().mla_cache_append_workspace_size(ctypes.byref(d), int(d_model))
    if n == 0:
        raise ValueError("mla_cache_append_workspace_size rejected the arguments")
    return int(n)


def cache_append(prob: Problem, x, w_dkv, k_rope, cache: Cache, workspace=None, stream=None):
    """mla_cache_append: c = x . W_DKV of the new tokens, written with k_rope into
    rows seq_lens[b] - s_q + i of the cache (whose kv buffer is modified)."""
    lib = load()
    if workspace is None:
        workspace = alloc_workspace(cache_append_workspace_size(prob, int(x.shape[-1])), x.device)
    d = prob.dims()
    _check(lib.mla_cache_append(ctypes.byref(d), int(x.shape[-1]), _ptr(x), _ptr(w_dkv), _ptr(k_rope),
                                ctypes.byref(cache), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mla_cache_append")
    return workspace


def naive_workspace_size(prob: Problem, cache: Cache) -> int:
    d = prob.dims()
    n = load().mla_naive_workspace_size(ctypes.byref(d), ctypes.byref(cache))
    if n == 0:
        raise ValueError("mla_naive_workspace_size rejected the arguments")
    return int(n)


def naive_decode(prob: Problem, q_nope, q_rope, cache: Cache, w_uk, w_uv, out=None, lse=None, workspace=None,
                 stream=None):
    lib = load()
    dev = q_nope.device
    if out is None:
        out = torch.empty(prob.B, prob.s_q, prob.H, prob.d_v, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(prob.B, prob.s_q, prob.H, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(naive_workspace_size(prob, cache), dev)
    d = prob.dims()
    _check(lib.mla_naive_decode(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), ctypes.byref(cache), _ptr(w_uk),
                                _ptr(w_uv), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                _stream(stream)), "mla_naive_decode")
    return out, lse, workspace


def prefill_crossover(prob: Problem, L: int) -> float:
    """mla_prefill_crossover: the query count S* where both bracketings tie (host only)."""
    d = prob.dims()
    return float(load().mla_prefill_crossover(ctypes.byref(d), int(L)))


def _prefill_outputs(prob, dev, out, lse):
    if out is None:
        out = torch.empty(prob.B, prob.s_q, prob.H, prob.d_v, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(prob.B, prob.s_q, prob.H, dtype=torch.float32, device=dev)
    return out, lse


def prefill_expand(prob: Problem, q_nope, q_rope, cache: Cache, w_uk, w_uv, out=None, lse=None, workspace=None,
                   stream=None):
    """mla_prefill_expand: K, V re-expanded per head, then per-head attention."""
    lib = load()
    out, lse = _prefill_outputs(prob, q_nope.device, out, lse)
    d = prob.dims()
    if workspace is None:
        n = lib.mla_prefill_expand_workspace_size(ctypes.byref(d), ctypes.byref(cache))
        if n == 0:
            raise ValueError("mla_prefill_expand_workspace_size rejected the arguments")
        workspace = alloc_workspace(n, q_nope.device)
    _check(lib.mla_prefill_expand(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), ctypes.byref(cache), _ptr(w_uk),
                                  _ptr(w_uv), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                  _stream(stream)), "mla_prefill_expand")
    return out, lse, workspace


def prefill(prob: Problem, q_nope, q_rope, cache: Cache, w_uk, w_uv, out=None, lse=None, workspace=None,
            stream=None):
    """mla_prefill: absorbed below the crossover S*, expanded at or above it.
    Returns (out, lse, workspace, path)."""
    lib = load()
    out, lse = _prefill_outputs(prob, q_nope.device, out, lse)
    d = prob.dims()
    if workspace is None:
        n = lib.mla_prefill_workspace_size(ctypes.byref(d), ctypes.byref(cache))
        if n == 0:
            raise ValueError("mla_prefill_workspace_size rejected the arguments")
        workspace = alloc_workspace(n, q_nope.device)
    path = ctypes.c_int(-1)
    _check(lib.mla_prefill(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), ctypes.byref(cache), _ptr(w_uk), _ptr(w_uv),
                           _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), ctypes.byref(path),
                           _stream(stream)), "mla_prefill")
    return out, lse, workspace, int(path.value)


def decode_attn_noalloc(prob: Problem, q_cat, cache: Cache, o_lat, lse, num_splits: int = 0,
                        device_status=None, stream=None):
    """mla_decode_attn_noalloc: the same attention with the library's built-in
    scratch array instead of a workspace (for callers that cannot allocate)."""
    d = prob.dims()
    _check(load().mla_decode_attn_noalloc(ctypes.byref(d), _ptr(q_cat), ctypes.byref(cache), _ptr(o_lat),
                                          _ptr(lse), int(num_splits), _ptr(device_status), _stream(stream)),
           "mla_decode_attn_noalloc")
    return o_lat, lse


def set_wait_limit_ns(ns: int) -> None:
    """mla_set_wait_limit_ns: the bound of the attention kernels' and of linear's waits for
    work (0: the default 2 s).  For tests of the timeout path."""
    _check(load().mla_set_wait_limit_ns(int(ns)), "mla_set_wait_limit_ns")


def read_status(workspace, stream=None) -> int:
    v = ctypes.c_int(0)
    _check(load().mla_read_status(_ptr(workspace), ctypes.byref(v), _stream(stream)), "mla_read_status")
    return int(v.value)


# ------------------------------------------------------------- the layer around the attention
# These calls take a few microseconds on the GPU, so what a call costs on the host counts: every
# property of a tensor is read once, without further calls, and pointers and streams go to ctypes
# as plain integers.
# Tensors that a call with ``stream=`` makes belong to that stream, as if the call stood under
# ``torch.cuda.stream(stream)``; inputs from another stream are the caller's to order.
_BF16, _I32 = torch.bfloat16, torch.int32
_ERR_WORKSPACE = 5  # MLA_ERR_WORKSPACE
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

try:  # an allocation on the current device without the dispatcher: 1.3 us against torch.empty's 2.8 (Grace host)
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    def _empty_strided_cuda(shape, stride, dtype):
        return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")


def _device(t, what: str) -> int:
    """Index of t's device, which must be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"{what} must be on the current CUDA device")
    return dev


def _refuse(t, what: str, need: str):
    raise ValueError(f"{what} must be {need}, not {t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")


def _dense(t, what: str, dtype, dev: int, shape) -> int:
    """Address of t, a dense tensor of this type and shape on device ``dev``."""
    if t.dtype != dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        _refuse(t, what, f"a dense {dtype} tensor {list(shape)} on device {dev}")
    return t.data_ptr()


def _per_token(t, what: str, dev: int, tokens: int) -> int:
    """Address of t, int32 with one entry a token."""
    if t.dtype != _I32 or t.get_device() != dev or not t.is_contiguous() or t.numel() != tokens:
        _refuse(t, what, f"a dense int32 tensor with one entry a token ({tokens}) on device {dev}")
    return t.data_ptr()


def _word(t, dev: int) -> int:
    """Address of a status word."""
    if t.dtype != _I32 or t.get_device() != dev or t.numel() < 1:
        _refuse(t, "status", f"an int32 tensor on device {dev}")
    return t.data_ptr()


def _rows(t, what: str, dev: int, M: int, N: int) -> int:
    """Address of t, a bf16 matrix with contiguous rows (any stride between them)."""
    if t.dtype != _BF16 or t.get_device() != dev or t.shape != (M, N) or (N > 1 and t.stride(1) != 1):
        _refuse(t, what, f"a torch.bfloat16 tensor [{M}, {N}] with contiguous rows on device {dev}")
    return t.data_ptr()


def _raw_stream(dev: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream must be one of device {dev}, not of {stream.device}")
    return stream.cuda_stream


def _allocator(stream):
    """What makes tensors (shape, stride, dtype) for kernels on ``stream`` (None: the current one), from that stream's
    memory: what was freed there is handed out again in the order of that stream's work alone."""
    if stream is None:
        return _empty_strided_cuda

    def new(shape, stride, dtype):
        with torch.cuda.stream(stream):
            return _empty_strided_cuda(shape, stride, dtype)
    return new


def rope_plan(d_rope: int, layout: int = ROPE_INTERLEAVED, base: float = 10000.0, scaling: int = ROPE_PLAIN,
              factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
              mscale: float = 1.0, inv_freq=None) -> RopePlan:
    """mla_rope_init: the rotation of one model (host only).  ``inv_freq``, d_rope / 2
    frequencies in radians a position, replaces base and scaling."""
    freq = None
    if inv_freq is not None:
        freq = [float(f) for f in inv_freq]
        if len(freq) != d_rope // 2:
            raise ValueError(f"inv_freq must have d_rope / 2 = {d_rope // 2} entries, not {len(freq)}")
        freq = (ctypes.c_double * len(freq))(*freq)
    cfg = RopeConfig(d_rope, layout, scaling, base, factor, original_len, beta_fast, beta_slow, mscale, freq)
    plan = RopePlan()
    _check(load().mla_rope_init(ctypes.byref(cfg), ctypes.byref(plan)), "mla_rope_init")
    return plan


def rope(prob: Problem, plan: RopePlan, x, positions=None, seq_lens=None, q_nope=None, q_rope=None,
         transpose: bool = False, stream=None):
    """mla_rope: x [B, s_q, H, d_nope + d_rope] (rows of heads may lie inside wider ones) split
    and rotated, returns (q_nope, q_rope); x [B, s_q, H, d_rope] rotated, returns q_rope (which
    may be x itself).  Tokens are at ``positions`` [B, s_q], or the last of ``seq_lens`` [B]."""
    lib = _lib or load()
    B, s_q, H, d_nope, d_rope = prob.B, prob.s_q, prob.H, prob.d_nope, prob.d_rope
    dev, shape = _device(x, "x"), x.shape
    split = shape == (B, s_q, H, d_nope + d_rope)
    if x.dtype != _BF16 or not (split or shape == (B, s_q, H, d_rope)):
        _refuse(x, "x", "torch.bfloat16 [B, s_q, H, d_nope + d_rope or d_rope]")
    s0, s1, head_stride, s3 = x.stride()
    if s3 != 1 or (B > 1 and s_q > 1 and s0 != s_q * s1):
        _refuse(x, "x", "of contiguous values and evenly spaced tokens")
    if H == 1:
        head_stride = shape[3]
    token_stride = s1 if s_q > 1 else s0 if B > 1 else (H - 1) * head_stride + shape[3]
    pos = None if positions is None else _per_token(positions, "positions", dev, B * s_q)
    lens = None if seq_lens is None else _dense(seq_lens, "seq_lens", _I32, dev, (B,))
    nope, new = None, _allocator(stream)
    if split:
        if q_nope is None:
            q_nope = new((B, s_q, H, d_nope), (s_q * H * d_nope, H * d_nope, d_nope, 1), _BF16)
            nope = q_nope.data_ptr()
        else:
            nope = _dense(q_nope, "q_nope", _BF16, dev, (B, s_q, H, d_nope))
    elif q_nope is not None:
        raise ValueError("rows of d_rope values have no part for q_nope")
    if q_rope is None:
        q_rope = new((B, s_q, H, d_rope), (s_q * H * d_rope, H * d_rope, d_rope, 1), _BF16)
        turned = q_rope.data_ptr()
    else:
        turned = _dense(q_rope, "q_rope", _BF16, dev, (B, s_q, H, d_rope))
    code = lib.mla_rope(prob.dims_ref(), ctypes.byref(plan), x.data_ptr(), token_stride, head_stride, pos, lens, nope,
                        turned, int(transpose), _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_rope")
    return (q_nope, q_rope) if split else q_rope


@dataclass
class Pages:
    """A batch's pages: the block table (int32 [B, max_pages]) and the ring of free page ids
    (int32 [num_pages]), both updated by ``pages_update``."""
    block_table: torch.Tensor
    free_ring: torch.Tensor
    page_size: int = 64

    def __post_init__(self):
        dev = _device(self.block_table, "block_table")
        if self.block_table.dim() != 2 or self.free_ring.dim() != 1:
            raise ValueError("block_table must be [B, max_pages], free_ring [num_pages]")
        _dense(self.block_table, "block_table", _I32, dev, self.block_table.shape)
        _dense(self.free_ring, "free_ring", _I32, dev, self.free_ring.shape)

    @classmethod
    def empty(cls, B: int, max_pages: int, num_pages: int, page_size: int = 64, device="cuda"):
        """A pool with every page free, and the ring's state for the first update."""
        table = torch.full((B, max_pages), -1, dtype=torch.int32, device=device)
        ring = torch.arange(num_pages, dtype=torch.int32, device=device)
        return cls(table, ring, page_size), torch.tensor([0, num_pages], dtype=torch.int32, device=device)


@dataclass(slots=True)
class PagesStep:
    """What one ``pages_update`` gives: the batch's lengths, the ring's state, and for the new
    tokens where each request's begin, their positions and their slots."""
    seq_lens: torch.Tensor
    ring_state: torch.Tensor
    token_start: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor


def pages_update(pages: Pages, ring_state, old_lens, new_lens, max_tokens: int, out: PagesStep | None = None,
                 status=None, stream=None) -> PagesStep:
    """mla_pages_update: every request from old_lens[b] to new_lens[b] tokens.  ``out`` (the
    result of an earlier call) is written over; its tensors must not be this call's inputs."""
    lib = _lib or load()
    table, ring = pages.block_table, pages.free_ring
    dev = _device(table, "block_table")
    # the fields may have been assigned since the batch was made
    if table.dim() != 2 or ring.dim() != 1:
        raise ValueError("block_table must be [B, max_pages], free_ring [num_pages]")
    if table.dtype != _I32 or not table.is_contiguous():
        _refuse(table, "block_table", f"a dense int32 tensor on device {dev}")
    if ring.dtype != _I32 or ring.get_device() != dev or not ring.is_contiguous():
        _refuse(ring, "free_ring", f"a dense int32 tensor on device {dev}")
    B, max_pages = table.shape
    state = _dense(ring_state, "ring_state", _I32, dev, (2,))
    old = _dense(old_lens, "old_lens", _I32, dev, (B,))
    new = _dense(new_lens, "new_lens", _I32, dev, (B,))
    word = None if status is None else _word(status, dev)
    if out is None:
        one, make = (1,), _allocator(stream)
        lens = make((B,), one, _I32)
        state_out = make((2,), one, _I32)
        start = make((B + 1,), one, _I32)
        pos = make((max_tokens,), one, _I32)
        slot = make((max_tokens,), one, _I32)
        out = PagesStep(lens, state_out, start, pos, slot)
        lens, state_out, start = lens.data_ptr(), state_out.data_ptr(), start.data_ptr()
        pos, slot = pos.data_ptr(), slot.data_ptr()
    else:
        lens = _dense(out.seq_lens, "seq_lens", _I32, dev, (B,))
        state_out = _dense(out.ring_state, "ring_state", _I32, dev, (2,))
        start = _dense(out.token_start, "token_start", _I32, dev, (B + 1,))
        pos = _dense(out.positions, "positions", _I32, dev, (max_tokens,))
        slot = _dense(out.slots, "slots", _I32, dev, (max_tokens,))
    pool = PagePool(B, pages.page_size, max_pages, ring.shape[0], table.data_ptr(), ring.data_ptr(), state, state_out)
    code = lib.mla_pages_update(ctypes.byref(pool), old, new, max_tokens, lens, start, pos, slot, word,
                                _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_pages_update")
    return out


def latent_store(prob: Problem, x, cache: Cache, plan: RopePlan | None = None, norm_weight=None, eps: float = 1e-6,
                 positions=None, slots=None, status=None, stream=None) -> None:
    """mla_latent_store: rows [c | k] of the new tokens (x [B * s_q, d_c + d_rope], inside wider
    rows or not) normalised, rotated and written to the cache, whose kv buffer is modified."""
    lib = _lib or load()
    dev = _device(x, "x")
    tokens, width = prob.B * prob.s_q, prob.d_c + prob.d_rope
    rows = _rows(x, "x", dev, tokens, width)
    weight = None if norm_weight is None else _dense(norm_weight, "norm_weight", _BF16, dev, (prob.d_c,))
    pos = None if positions is None else _per_token(positions, "positions", dev, tokens)
    slot = None if slots is None else _per_token(slots, "slots", dev, tokens)
    word = None if status is None else _word(status, dev)
    code = lib.mla_latent_store(prob.dims_ref(), None if plan is None else ctypes.byref(plan), rows,
                                x.stride(0) if tokens > 1 else width, weight, eps, pos, slot, ctypes.byref(cache), word,
                                _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_latent_store")


def linear_workspace_size(M: int, K: int, N: int) -> int:
    desc = LinearDesc(M, K, N, ACT_NONE, K, N, N)
    n = load().mla_linear_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise ValueError("mla_linear_workspace_size rejected the arguments")
    return int(n)


def linear_cut(M: int, K: int, N: int) -> LinearCut:
    """mla_linear_query_cut: how a product of these sizes is cut on the current device (host only)."""
    desc, cut = LinearDesc(M, K, N, ACT_NONE, K, N, N), LinearCut()
    _check(load().mla_linear_query_cut(ctypes.byref(desc), ctypes.byref(cut)), "mla_linear_query_cut")
    return cut


def linear(x, w, bias=None, residual=None, act: int = ACT_NONE, out=None, workspace=None, stream=None, status=None):
    """mla_linear: residual + act(x . w + bias), x [M, K] and residual [M, N] with any row stride
    (multiples of 8), w [K, N] dense.  ``out`` may be ``residual``; ``status`` (an int32 word)
    takes MLA_ERR_TIMEOUT where a wait on the device ran out."""
    lib = _lib or load()
    dev = _device(x, "x")
    if w.dim() != 2 or x.dim() != 2:
        raise ValueError("x must be [M, K], w [K, N]")
    K, N = w.shape
    M = x.shape[0]
    rows = _rows(x, "x", dev, M, K)
    if w.dtype != _BF16 or w.get_device() != dev or not w.is_contiguous():
        _refuse(w, "w", f"a dense torch.bfloat16 tensor on device {dev}")
    b = None if bias is None else _dense(bias, "bias", _BF16, dev, (N,))
    res = None if residual is None else _rows(residual, "residual", dev, M, N)
    word = None if status is None else _word(status, dev)
    if out is None:
        out = _allocator(stream)((M, N), (N, 1), _BF16)
        to, out_stride = out.data_ptr(), N
    else:
        to, out_stride = _rows(out, "out", dev, M, N), out.stride(0)
    if M > 1:
        desc = LinearDesc(M, K, N, act, x.stride(0), out_stride, N if res is None else residual.stride(0))
    else:  # a single row has no stride
        desc = LinearDesc(M, K, N, act, K, N, N)
    at, weight, st = ctypes.byref(desc), w.data_ptr(), _raw_stream(dev, stream)
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(workspace, "workspace", f"dense memory on device {dev}")
        code = lib.mla_linear_status(at, rows, weight, b, res, to, workspace.data_ptr(), workspace.nbytes, word, st)
    else:  # most shapes need none
        code = lib.mla_linear_status(at, rows, weight, b, res, to, None, 256, word, st)
        if code == _ERR_WORKSPACE:
            nbytes = lib.mla_linear_workspace_size(at)
            workspace = _allocator(stream)((nbytes,), (1,), torch.uint8)
            code = lib.mla_linear_status(at, rows, weight, b, res, to, workspace.data_ptr(), nbytes, word, st)
    if code:
        raise MLAError(code, "mla_linear")
    return out


# --------------------------------------------------------------- 8 bits with scales by blocks of 128
_E4M3, _F32 = torch.float8_e4m3fn, torch.float32


def latent_row_bytes(prob: Problem) -> int:
    """mla_latent_row_bytes: the width of a cache row in blocks (a uint8 cache of it is one for ``make_cache``)."""
    n = load().mla_latent_row_bytes(prob.dims_ref())
    if n == 0:
        raise ValueError("mla_latent_row_bytes rejected the widths")
    return int(n)


def _matrix(t, what: str, dtype, dev: int, M: int, N: int):
    """Address of t, a matrix of this type with contiguous rows, and the elements between them (any; a single
    row has none of its own)."""
    if t.dtype != dtype or t.get_device() != dev or t.shape != (M, N):
        _refuse(t, what, f"a {dtype} tensor [{M}, {N}] with contiguous rows on device {dev}")
    if t.is_contiguous():
        return t.data_ptr(), N
    if N > 1 and t.stride(1) != 1:
        _refuse(t, what, f"a {dtype} tensor [{M}, {N}] with contiguous rows on device {dev}")
    return t.data_ptr(), t.stride(0)


def quantize(x, norm_weight=None, eps: float = 1e-6, block_rows: int = 1, codes=None, scales=None, stream=None):
    """mla_quantize: x [M, K] (any row stride), after its RMS norm if ``norm_weight`` [K] is given, as E4M3 codes
    [M, K] with fp32 scales: [ceil(K / 128), M] for ``block_rows`` 1 (activations), [ceil(M / 128), ceil(K / 128)]
    for 128 (weights, [N, K] as ``linear_fp8`` takes them).  Returns (codes, scales)."""
    lib = _lib or load()
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    rows, x_stride = _matrix(x, "x", _BF16, dev, M, K)
    weight = None if norm_weight is None else _dense(norm_weight, "norm_weight", _BF16, dev, (K,))
    wide = (K + 127) // 128
    shape = (wide, M) if block_rows == 1 else ((M + 127) // 128, wide)
    new = _allocator(stream)
    if codes is None:
        codes = new((M, K), (K, 1), _E4M3)
        to, code_stride = codes.data_ptr(), K
    else:
        to, code_stride = _matrix(codes, "codes", _E4M3, dev, M, K)
    if scales is None:
        scales = new(shape, (shape[1], 1), _F32)
        at = scales.data_ptr()
    else:
        at = _dense(scales, "scales", _F32, dev, shape)
    desc = QuantizeDesc(M, K, block_rows, x_stride, code_stride, shape[1])
    code = lib.mla_quantize(ctypes.byref(desc), rows, weight, eps, to, at, _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_quantize")
    return codes, scales


def linear_fp8(x, x_scale, w, w_scale, bias=None, residual=None, act: int = ACT_NONE, out=None, stream=None, status=None):
    """mla_linear_fp8: residual + act(x . w^T + bias) of E4M3 codes x [M, K] (rows any multiple of 16 bytes apart) and
    w [N, K] dense, with the scales that ``quantize`` gives: x_scale [ceil(K / 128), M] (rows any distance apart: those of a
    slice of x are a slice of the whole's), w_scale [ceil(N / 128), ceil(K / 128)].  bias, residual, out and ``status`` as for ``linear``."""
    lib = _lib or load()
    dev = _device(x, "x")
    if w.dim() != 2 or x.dim() != 2:
        raise ValueError("x must be [M, K], w [N, K]")
    N, K = w.shape
    M = x.shape[0]
    rows, x_stride = _matrix(x, "x", _E4M3, dev, M, K)
    if w.dtype != _E4M3 or w.get_device() != dev or not w.is_contiguous():
        _refuse(w, "w", f"a dense torch.float8_e4m3fn tensor on device {dev}")
    wide = (K + 127) // 128
    xs, xs_stride = _matrix(x_scale, "x_scale", _F32, dev, wide, M)
    ws = _dense(w_scale, "w_scale", _F32, dev, ((N + 127) // 128, wide))
    b = None if bias is None else _dense(bias, "bias", _BF16, dev, (N,))
    res, res_stride = (None, N) if residual is None else _matrix(residual, "residual", _BF16, dev, M, N)
    word = None if status is None else _word(status, dev)
    if out is None:
        out = _allocator(stream)((M, N), (N, 1), _BF16)
        to, out_stride = out.data_ptr(), N
    else:
        to, out_stride = _matrix(out, "out", _BF16, dev, M, N)
    desc = LinearFp8Desc(M, K, N, act, x_stride, xs_stride, out_stride, res_stride)
    code = lib.mla_linear_fp8(ctypes.byref(desc), rows, xs, w.data_ptr(), ws, b, res, to, word, _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_linear_fp8")
    return out


def linear_fp8_cut(M: int, K: int, N: int) -> LinearCut:
    """mla_linear_fp8_query_cut: how a product of these sizes is cut on the current device (host only)."""
    desc, cut = LinearFp8Desc(M, K, N, ACT_NONE, K, M, N, N), LinearCut()
    _check(load().mla_linear_fp8_query_cut(ctypes.byref(desc), ctypes.byref(cut)), "mla_linear_fp8_query_cut")
    return cut


def latent_load(prob: Problem, cache: Cache, rows: int, positions=None, out=None, status=None, stream=None):
    """mla_latent_load: ``rows`` tokens of each sequence back as bf16 [B, rows, d_c + d_rope] (``out``: any stride
    between sequences), the first ones or those of ``positions`` [B, rows].  Rows of no token stay as they were in ``out``;
    without it they are 0, which costs a fill of the whole result before the call."""
    lib = _lib or load()
    B, width = prob.B, prob.d_c + prob.d_rope
    dev = _current_device()
    if out is None:
        with torch.cuda.stream(stream):
            out = _empty_strided_cuda((B, rows, width), (rows * width, width, 1), _BF16).zero_()
        stride = rows * width
    else:
        if (out.dtype != _BF16 or out.get_device() != dev or out.shape != (B, rows, width) or out.stride(2) != 1 or
                (rows > 1 and out.stride(1) != width)):
            _refuse(out, "out", f"torch.bfloat16 [{B}, {rows}, {width}] with dense rows on device {dev}")
        stride = out.stride(0) if B > 1 else rows * width
    at = None if positions is None else _dense(positions, "positions", _I32, dev, (B, rows))
    word = None if status is None else _word(status, dev)
    code = lib.mla_latent_load(prob.dims_ref(), ctypes.byref(cache), rows, at, out.data_ptr(), stride, word,
                               _raw_stream(dev, stream))
    if code:
        raise MLAError(code, "mla_latent_load")
    return out


class Decoder:
    """One layer's absorbed decode step with its buffers allocated once:
    absorb_q -> decode_attn -> out_proj on the current stream."""

    def __init__(self, prob: Problem, kv, seq_lens, w_uk, w_uv, block_table=None, page_size=64,
                 max_seq_len=0, num_splits=0, kv_scale=None):
        self.prob = prob
        self.kv, self.seq_lens, self.block_table = kv, seq_lens, block_table
        self.w_uk, self.w_uv = w_uk, w_uv
        self.cache = make_cache(prob, kv, seq_lens, block_table, page_size, max_seq_len, kv_scale)
        self.num_splits = num_splits
        dev = kv.device
        B, s_q, H = prob.B, prob.s_q, prob.H
        self.q_cat = torch.empty(B, s_q, H, prob.d_c + prob.d_rope, dtype=torch.bfloat16, device=dev)
        self.o_lat = torch.empty(B, s_q, H, prob.d_c, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(B, s_q, H, dtype=torch.float32, device=dev)
        self.out = torch.empty(B, s_q, H, prob.d_v, dtype=torch.bfloat16, device=dev)
        self.workspace = alloc_workspace(decode_workspace_size(prob, self.cache, num_splits), dev)

    def absorb(self, q_nope, q_rope, stream=None):
        return absorb_q(self.prob, q_nope, q_rope, self.w_uk, self.q_cat, stream)

    def attend(self, stream=None):
        return decode_attn(self.prob, self.q_cat, self.cache, self.o_lat, self.lse, self.workspace,
                           self.num_splits, stream)

    def project(self, stream=None):
        return out_proj(self.prob, self.o_lat, self.w_uv, self.out, stream)

    def step(self, q_nope, q_rope, stream=None):
        """mla_decode_step: the three launches as one call, overlapping."""
        d = self.prob.dims()
        _check(load().mla_decode_step(ctypes.byref(d), _ptr(q_nope), _ptr(q_rope), ctypes.byref(self.cache),
                                      _ptr(self.w_uk), _ptr(self.w_uv), _ptr(self.q_cat), _ptr(self.o_lat),
                                      _ptr(self.out), _ptr(self.lse), _ptr(self.workspace), self.workspace.numel(),
                                      int(self.num_splits), _stream(stream)), "mla_decode_step")
        return self.out

    def __call__(self, q_nope, q_rope, stream=None):
        self.absorb(q_nope, q_rope, stream)
        self.attend(stream)
        self.project(stream)
        return self.out
