"""Python binding of the GB300 attention library ``libna.so`` (C ABI in ``include/na.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libna.so``.  PyTorch supplies device memory and streams.  There is
no CPU fallback: importing works without a GPU (so the symbols can be checked),
but every compute call needs the built library and CUDA tensors, and raises
otherwise.

Entry points (same names as the C ABI):
  na_rope_append_kv      fused qk-norm + RoPE + KV-cache append
  na_attn_prefill_chunk  causal GQA attention of a chunk against the cache
  na_attn_decode         single-token decode with per-key probabilities
  na_decode_importance   the step's Born-rule importance (sum over heads of the probabilities)
  na_attn_decode_static_ws  na_attn_decode with library-owned scratch
  na_rope_append_kv_paged, na_attn_prefill_chunk_paged, na_attn_decode_paged
                         the same over a paged cache of bf16 or 8-bit (E4M3) pages
  na_latent_append_paged, na_attn_latent_paged, na_attn_latent_expanded
                         latent attention: fused append of latent rows, the absorbed form over
                         pages, the expanded form
  na_pages_fork          page tables of a step: sequences forked, ended, begun, given room
  na_pages_copy          whole pages copied
  na_pages_compact       kept tokens to the front of new pages, keys turned to their new positions
  na_prefill_workspace_size / na_decode_workspace_size, the same with _paged,
  na_latent_paged_workspace_size, na_status_string
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libna.so")

NA_OK = 0
NA_ERR_INVALID_ARG = -1
NA_ERR_UNSUPPORTED = -2
NA_ERR_CAPACITY = -3
NA_ERR_WORKSPACE = -4
NA_ERR_CUDA = -5
NA_ERR_DEVICE_TIMEOUT = -6
NA_ERR_PAGE = -7

NA_QK_NORM = 1
NA_QK_NORM_ZERO_CENTERED = 2
NA_V_NORM = 4
NA_OUT_GATE = 8
NA_RING_CACHE = 16

NA_LATENT_NORM = 1
NA_ROPE_INTERLEAVED = 2

NA_KV_BF16 = 0
NA_KV_E4M3 = 1

# Every symbol include/na.h declares.
EXPORTED = ("na_rope_append_kv", "na_attn_prefill_chunk", "na_attn_decode",
            "na_attn_decode_static_ws", "na_decode_importance",
            "na_prefill_workspace_size", "na_decode_workspace_size", "na_status_string",
            "na_selftest_wait_timeout", "na_rope_append_kv_paged", "na_attn_prefill_chunk_paged",
            "na_attn_decode_paged", "na_prefill_paged_workspace_size",
            "na_decode_paged_workspace_size", "na_pages_fork", "na_pages_copy",
            "na_pages_compact", "na_latent_append_paged", "na_attn_latent_paged",
            "na_latent_paged_workspace_size", "na_attn_latent_expanded")


class na_attn_cfg(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("flags", ctypes.c_uint32), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int32)]


class na_rope_params(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("yarn", ctypes.c_int32), ("factor", ctypes.c_double),
                ("orig_max_pos", ctypes.c_int32), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("attn_factor", ctypes.c_double)]


class na_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]


class na_paged_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class na_latent_cfg(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("kv_rank", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("nope_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class na_paged_latent_cache(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32)]


class NAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {status_string(code)} ({code})")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libna.so (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libna.so is not built ({path}); run __graft_entry__.build() or "
                           f"python -m causal_gqa_attention_rope_gb300._build")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    cfgp = ctypes.POINTER(na_attn_cfg)
    ropep = ctypes.POINTER(na_rope_params)
    cachep = ctypes.POINTER(na_kv_cache)
    lib.na_rope_append_kv.argtypes = [cfgp, ropep, I32, P, P, I32, P, P, P, P, P, P, cachep, P, P]
    lib.na_attn_prefill_chunk.argtypes = [cfgp, I32, P, P, I32, I32, I32, P, cachep, P, P, P, SZ,
                                          P, P]
    lib.na_attn_decode.argtypes = [cfgp, I32, P, cachep, P, I32, P, P, P, I32, I32, P, SZ, P, P]
    lib.na_attn_decode_static_ws.argtypes = [cfgp, I32, P, cachep, P, I32, P, P, P, I32, I32, P,
                                             P]
    lib.na_decode_importance.argtypes = [cfgp, I32, P, I32, P, I32, P, I32, I32, P, P]
    lib.na_prefill_workspace_size.argtypes = [cfgp, I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.na_decode_workspace_size.argtypes = [cfgp, I32, I32, I32, ctypes.POINTER(SZ)]
    pagedp = ctypes.POINTER(na_paged_kv_cache)
    lib.na_rope_append_kv_paged.argtypes = [cfgp, ropep, I32, P, P, I32, P, P, P, P, P, P, pagedp,
                                            P, P]
    lib.na_attn_prefill_chunk_paged.argtypes = [cfgp, I32, P, P, I32, I32, I32, P, pagedp, P, P, P,
                                                SZ, P, P]
    lib.na_attn_decode_paged.argtypes = [cfgp, I32, P, pagedp, P, I32, P, P, P, I32, I32, P, SZ, P,
                                         P]
    lib.na_prefill_paged_workspace_size.argtypes = [cfgp, I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.na_decode_paged_workspace_size.argtypes = [cfgp, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.na_pages_fork.argtypes = [I32, I32, P, P, P, P, I32, I32, P, I32, P, P, P, P, P, P, P]
    lib.na_pages_copy.argtypes = [I32, I32, pagedp, I32, P, P, P, P]
    lib.na_pages_compact.argtypes = [I32, I32, I32, pagedp, pagedp, P, P, I32, ropep, I32, I32,
                                     ctypes.c_uint32, P, P]
    latp, lcachep, I64 = ctypes.POINTER(na_latent_cfg), ctypes.POINTER(na_paged_latent_cache), ctypes.c_int64
    lib.na_latent_append_paged.argtypes = [latp, ropep, I32, P, P, I32, P, I64, P, I64, P, I64, P,
                                           lcachep, P, P]
    lib.na_attn_latent_paged.argtypes = [latp, I32, P, P, I32, I32, I32, P, lcachep, P, P, SZ, P, P]
    lib.na_latent_paged_workspace_size.argtypes = [latp, I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.na_attn_latent_expanded.argtypes = [latp, I32, P, P, P, I32, I32, I32, I32, P, P, P, I64, P, P,
                                            P]
    lib.na_selftest_wait_timeout.argtypes = [P, P]
    lib.na_status_string.argtypes = [ctypes.c_int]
    lib.na_status_string.restype = ctypes.c_char_p
    for name in ("na_rope_append_kv", "na_attn_prefill_chunk", "na_attn_decode",
                 "na_attn_decode_static_ws", "na_decode_importance",
                 "na_prefill_workspace_size", "na_decode_workspace_size",
                 "na_selftest_wait_timeout", "na_rope_append_kv_paged",
                 "na_attn_prefill_chunk_paged", "na_attn_decode_paged",
                 "na_prefill_paged_workspace_size", "na_decode_paged_workspace_size",
                 "na_pages_fork", "na_pages_copy", "na_pages_compact", "na_latent_append_paged",
                 "na_attn_latent_paged", "na_latent_paged_workspace_size", "na_attn_latent_expanded"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().na_status_string(int(code)).decode()


# ------------------------------------------------------------ configuration --

@dataclass
class AttnConfig:
    num_heads: int
    num_kv_heads: int
    head_dim: int
    rotary_dim: Optional[int] = None
    sm_scale: float = 0.0
    rms_eps: float = 1e-6
    qk_norm: bool = False
    qk_norm_zero_centered: bool = False
    v_norm: bool = False
    out_gate: bool = False
    softcap: float = 0.0
    window: int = 0
    ring_cache: bool = False

    @property
    def flags(self) -> int:
        return ((NA_QK_NORM if self.qk_norm else 0)
                | (NA_QK_NORM_ZERO_CENTERED if self.qk_norm_zero_centered else 0)
                | (NA_V_NORM if self.v_norm else 0) | (NA_OUT_GATE if self.out_gate else 0)
                | (NA_RING_CACHE if self.ring_cache else 0))

    def c(self) -> na_attn_cfg:
        rd = self.head_dim if self.rotary_dim is None else self.rotary_dim
        return na_attn_cfg(self.num_heads, self.num_kv_heads, self.head_dim, rd, self.sm_scale,
                           self.rms_eps, self.flags, self.softcap, self.window)


@dataclass
class RopeConfig:
    base: float = 10000.0
    yarn: bool = False
    factor: float = 1.0
    orig_max_pos: int = 0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    attn_factor: float = 0.0

    def c(self) -> na_rope_params:
        return na_rope_params(self.base, int(self.yarn), self.factor, self.orig_max_pos,
                              self.beta_fast, self.beta_slow, self.attn_factor)


@dataclass
class LatentConfig:
    """Latent attention: num_heads heads over rows of kv_rank + rope_dim numbers a token."""
    num_heads: int
    kv_rank: int = 512
    rope_dim: int = 64
    nope_dim: int = 128
    v_dim: int = 128
    sm_scale: float = 0.0
    rms_eps: float = 1e-6
    kv_norm: bool = True
    rope_interleaved: bool = False

    def c(self) -> na_latent_cfg:
        flags = ((NA_LATENT_NORM if self.kv_norm else 0)
                 | (NA_ROPE_INTERLEAVED if self.rope_interleaved else 0))
        return na_latent_cfg(self.num_heads, self.kv_rank, self.rope_dim, self.nope_dim, self.v_dim,
                             self.sm_scale, self.rms_eps, flags)


@dataclass
class KVCache:
    """Caller-owned bf16 cache tensors [batch, num_kv_heads, capacity, head_dim]."""
    k: "object"
    v: "object"

    def c(self) -> na_kv_cache:
        return na_kv_cache(_ptr(self.k), _ptr(self.v), int(self.k.shape[0]), int(self.k.shape[2]))


@dataclass
class PagedKVCache:
    """Caller-owned pages and page table.

    k, v        [num_pages, num_kv_heads, page_size, head_dim], bfloat16 or float8_e4m3fn
    page_table  int32 [batch, pages_per_seq]: the page of positions
                [i * page_size, (i + 1) * page_size) of each sequence
    k_scale, v_scale  with float8 pages: uint8 [num_pages, num_kv_heads], E8M0 (2^(s - 127))
    """
    k: "object"
    v: "object"
    page_table: "object"
    k_scale: "object" = None
    v_scale: "object" = None

    def c(self) -> na_paged_kv_cache:
        num_pages, _, page_size, _ = self.k.shape
        batch, pages_per_seq = self.page_table.shape
        return na_paged_kv_cache(
            _ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale),
            _ptr(self.page_table), num_pages, page_size, batch, pages_per_seq,
            NA_KV_BF16 if self.k_scale is None else NA_KV_E4M3)


@dataclass
class PagedLatentCache:
    """Caller-owned pages of latent rows and page table.

    kv          bfloat16 [num_pages, page_size, kv_rank + rope_dim]: one row a token for all heads
    page_table  int32 [batch, pages_per_seq], as PagedKVCache's
    """
    kv: "object"
    page_table: "object"

    def c(self) -> na_paged_latent_cache:
        num_pages, page_size, _ = self.kv.shape
        batch, pages_per_seq = self.page_table.shape
        return na_paged_latent_cache(_ptr(self.kv), _ptr(self.page_table), num_pages, page_size, batch,
                                     pages_per_seq)


# ---------------------------------------------------------------- helpers --

def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libna operates on CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libna needs contiguous tensors")
    return t.data_ptr()


_current_stream = None
_current_device = None


def _find_current():
    """Set the lookups of the current device and of its current stream."""
    global _current_stream, _current_device
    import torch
    torch.cuda.current_device()  # initialises CUDA
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:  # the handle alone, without building a Stream object
        _current_stream = lambda: raw(_current_device())
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream


def _stream(stream) -> Optional[int]:
    """Raw handle of `stream`, or of the current device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    if _current_stream is None:
        _find_current()
    return _current_stream()


def _on_current(*tensors):
    """Refuse tensors of another device than the current one."""
    if _current_device is None:
        _find_current()
    for t in tensors:
        if t is not None and t.get_device() != _current_device():
            raise ValueError(f"a tensor is on cuda:{t.get_device()}, but the current device is "
                             f"cuda:{_current_device()}")


_dtypes = {}  # torch's dtype objects by name


def _dtype(name: str):
    import torch
    _dtypes[name] = getattr(torch, name)
    return _dtypes[name]


def _want(t, name: str, dtype: str, shape=None, min_rows: int = 0):
    """A tensor's dtype and shape, checked before its pointer crosses the C ABI
    (the library sees only pointers: a wrong dtype would be read as another
    type, a short tensor past its end).  `shape` entries of None match any
    size; the first dimension must also hold at least `min_rows`."""
    if t is None:
        return
    if t.dtype is not (_dtypes.get(dtype) or _dtype(dtype)):
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None:
        got = t.shape
        if got != shape:  # not the very sizes: None matches any
            ok = len(got) == len(shape)
            if ok:
                for w, g in zip(shape, got):
                    if w != g and w is not None:
                        ok = False
            if not ok:
                want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
                raise ValueError(f"{name}: expected shape {want}, got {list(got)}")
        if got[0] < min_rows:
            raise ValueError(f"{name}: {int(got[0])} rows, at least {min_rows} needed")


def _want_cache(cache: "KVCache", cfg: "AttnConfig", batch: int):
    _want(cache.k, "cache.k", "bfloat16", (None, cfg.num_kv_heads, None, cfg.head_dim), batch)
    _want(cache.v, "cache.v", "bfloat16", tuple(cache.k.shape))


def _paged(cache: "PagedKVCache", cfg: "AttnConfig", batch: int) -> na_paged_kv_cache:
    """The C struct of a paged cache, its tensors checked."""
    bf16 = cache.k_scale is None and cache.v_scale is None
    kind = "bfloat16" if bf16 else "float8_e4m3fn"
    _want(cache.k, "cache.k", kind, (None, cfg.num_kv_heads, None, cfg.head_dim))
    _want(cache.v, "cache.v", kind, cache.k.shape)
    _want(cache.page_table, "cache.page_table", "int32", (None, None), batch)
    if not bf16:
        scales = (cache.k.shape[0], cfg.num_kv_heads)
        for t, name in ((cache.k_scale, "cache.k_scale"), (cache.v_scale, "cache.v_scale")):
            if t is None:
                raise ValueError(f"{name}: missing")
            _want(t, name, "uint8", scales)
    return cache.c()


_native = None


def _calls():
    """The compiled paged calls (csrc/paged_calls.cpp): they answer a call's status, or None,
    without having called, for what is not plainly right; the checks here then say what."""
    global _native
    if _native is None:
        lib = load_library()
        import torch  # its libraries have to be there first
        how = "run __graft_entry__.build() or python -m causal_gqa_attention_rope_gb300._build"
        try:
            from . import _paged_calls as calls
        except ImportError as e:
            raise RuntimeError(f"the paged calls are not built; {how}") from e
        here = f"{torch.__version__} {torch.version.git_version}"
        if getattr(calls, "torch", "") != here:  # it reads tensors through that torch's layout
            raise RuntimeError(f"the paged calls were built for another torch than {here}; {how}")
        calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                     for f in (lib.na_rope_append_kv_paged, lib.na_attn_prefill_chunk_paged,
                               lib.na_attn_decode_paged)), AttnConfig, RopeConfig, PagedKVCache)
        calls.bind_latent(*(ctypes.cast(f, ctypes.c_void_p).value
                            for f in (lib.na_latent_append_paged, lib.na_attn_latent_paged,
                                      lib.na_attn_latent_expanded, lib.na_pages_fork, lib.na_pages_copy,
                                      lib.na_pages_compact)), LatentConfig, PagedLatentCache)
        _native = calls
    return _native


def _check(fn: str, rc: int):
    if rc != NA_OK:
        raise NAError(fn, rc)


# ------------------------------------------------------------ entry points --

def _append_args(cfg, cu_seqlens, cache_lens, q, k, v, q_out, q_norm_w, k_norm_w, status,
                 total_tokens):
    """Checks of the arguments that the contiguous and the paged append share; (batch, tokens)."""
    T = int(q.shape[0]) if total_tokens is None else int(total_tokens)
    batch = int(cu_seqlens.numel()) - 1
    H, KV, d = cfg.num_heads, cfg.num_kv_heads, cfg.head_dim
    _want(cu_seqlens, "cu_seqlens", "int32", (None,))
    _want(cache_lens, "cache_lens", "int32", (None,), batch)
    bf16, kv = q.dtype, (T, KV, d)
    # the usual sizes, checked at once; anything else one by one
    if not (bf16 is _dtypes.get("bfloat16") and q_out.dtype is bf16 and k.dtype is bf16
            and v.dtype is bf16 and q.shape == (T, H, d) and q_out.shape == (T, H, d)
            and k.shape == kv and v.shape == kv):
        _want(q, "q", "bfloat16", (None, H, d), T)
        _want(q_out, "q_out", "bfloat16", (None, H, d), T)
        _want(k, "k", "bfloat16", (None, KV, d), T)
        _want(v, "v", "bfloat16", (None, KV, d), T)
    _want(q_norm_w, "q_norm_w", "bfloat16", (d,))
    _want(k_norm_w, "k_norm_w", "bfloat16", (d,))
    _want(status, "status", "int32", (None,), 1)
    return batch, T


def na_rope_append_kv(cfg: AttnConfig, rope: RopeConfig, cu_seqlens, cache_lens, q, k, v,
                      q_out, cache: KVCache, q_norm_w=None, k_norm_w=None, status=None,
                      total_tokens: Optional[int] = None, stream=None):
    lib = load_library()
    batch, T = _append_args(cfg, cu_seqlens, cache_lens, q, k, v, q_out, q_norm_w, k_norm_w,
                            status, total_tokens)
    _want_cache(cache, cfg, batch)
    c, r, kc = cfg.c(), rope.c(), cache.c()
    rc = lib.na_rope_append_kv(ctypes.byref(c), ctypes.byref(r), batch, _ptr(cu_seqlens),
                               _ptr(cache_lens), T, _ptr(q), _ptr(k), _ptr(v), _ptr(q_norm_w),
                               _ptr(k_norm_w), _ptr(q_out), ctypes.byref(kc), _ptr(status),
                               _stream(stream))
    _check("na_rope_append_kv", rc)


def na_rope_append_kv_paged(cfg: AttnConfig, rope: RopeConfig, cu_seqlens, cache_lens, q, k, v,
                            q_out, cache: PagedKVCache, q_norm_w=None, k_norm_w=None, status=None,
                            total_tokens: Optional[int] = None, stream=None):
    """na_rope_append_kv into bf16 or E4M3 pages."""
    rc = (_native or _calls()).append(cfg, rope, cu_seqlens, cache_lens, q, k, v, q_out,
                                           cache, q_norm_w, k_norm_w, status, total_tokens, stream)
    if rc is None:
        batch, T = _append_args(cfg, cu_seqlens, cache_lens, q, k, v, q_out, q_norm_w, k_norm_w,
                                status, total_tokens)
        kc = _paged(cache, cfg, batch)
        c, r = cfg.c(), rope.c()
        args = [_ptr(t) for t in (q, k, v, q_norm_w, k_norm_w, q_out)]
        cu, lens, st = _ptr(cu_seqlens), _ptr(cache_lens), _ptr(status)
        _on_current(cu_seqlens, cache_lens, q, k, v, q_norm_w, k_norm_w, q_out, status, cache.k,
                    cache.v, cache.k_scale, cache.v_scale, cache.page_table)
        rc = load_library().na_rope_append_kv_paged(
            ctypes.byref(c), ctypes.byref(r), batch, cu, lens, T, *args, ctypes.byref(kc), st,
            _stream(stream))
    if rc != NA_OK:
        raise NAError("na_rope_append_kv_paged", rc)


def na_prefill_workspace_size(cfg: AttnConfig, batch: int, total_tokens: int, max_new_len: int,
                              max_total_len: int) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    c = cfg.c()
    _check("na_prefill_workspace_size",
           lib.na_prefill_workspace_size(ctypes.byref(c), batch, total_tokens, max_new_len,
                                         max_total_len, ctypes.byref(out)))
    return int(out.value)


def na_decode_workspace_size(cfg: AttnConfig, batch: int, max_kv_len: int,
                             num_splits: int = 0) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    c = cfg.c()
    _check("na_decode_workspace_size",
           lib.na_decode_workspace_size(ctypes.byref(c), batch, max_kv_len, num_splits,
                                        ctypes.byref(out)))
    return int(out.value)


def na_prefill_paged_workspace_size(cfg: AttnConfig, batch: int, total_tokens: int,
                                    max_new_len: int, max_total_len: int) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    c = cfg.c()
    _check("na_prefill_paged_workspace_size",
           lib.na_prefill_paged_workspace_size(ctypes.byref(c), batch, total_tokens, max_new_len,
                                               max_total_len, ctypes.byref(out)))
    return int(out.value)


def na_decode_paged_workspace_size(cfg: AttnConfig, batch: int, max_kv_len: int,
                                   num_splits: int = 0) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    c = cfg.c()
    _check("na_decode_paged_workspace_size",
           lib.na_decode_paged_workspace_size(ctypes.byref(c), batch, max_kv_len, num_splits,
                                              ctypes.byref(out)))
    return int(out.value)


def _prefill_args(cfg, cu_seqlens, cache_lens, q_rot, out, gate, status, total_tokens):
    """Checks of the arguments that both prefill calls share; (batch, tokens)."""
    T = int(q_rot.shape[0]) if total_tokens is None else int(total_tokens)
    batch = int(cu_seqlens.numel()) - 1
    H, d = cfg.num_heads, cfg.head_dim
    _want(cu_seqlens, "cu_seqlens", "int32", (None,))
    _want(cache_lens, "cache_lens", "int32", (None,), batch)
    if not (q_rot.dtype is _dtypes.get("bfloat16") and out.dtype is q_rot.dtype
            and q_rot.shape == (T, H, d) and out.shape == (T, H, d)):
        _want(q_rot, "q_rot", "bfloat16", (None, H, d), T)
        _want(out, "out", "bfloat16", (None, H, d), T)
    _want(gate, "gate", "bfloat16", (None, H, d), T)
    _want(status, "status", "int32", (None,), 1)
    return batch, T


def na_attn_prefill_chunk(cfg: AttnConfig, cu_seqlens, cache_lens, max_new_len: int,
                          max_total_len: int, q_rot, cache: KVCache, out, gate=None,
                          workspace=None, status=None, total_tokens: Optional[int] = None,
                          stream=None):
    lib = load_library()
    batch, T = _prefill_args(cfg, cu_seqlens, cache_lens, q_rot, out, gate, status, total_tokens)
    _want_cache(cache, cfg, batch)
    c, kc = cfg.c(), cache.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.na_attn_prefill_chunk(ctypes.byref(c), batch, _ptr(cu_seqlens), _ptr(cache_lens), T,
                                   int(max_new_len), int(max_total_len), _ptr(q_rot),
                                   ctypes.byref(kc), _ptr(gate), _ptr(out), _ptr(workspace),
                                   ws_bytes, _ptr(status), _stream(stream))
    _check("na_attn_prefill_chunk", rc)


def na_attn_prefill_chunk_paged(cfg: AttnConfig, cu_seqlens, cache_lens, max_new_len: int,
                                max_total_len: int, q_rot, cache: PagedKVCache, out, gate=None,
                                workspace=None, status=None, total_tokens: Optional[int] = None,
                                stream=None):
    """na_attn_prefill_chunk against bf16 or E4M3 pages (workspace:
    na_prefill_paged_workspace_size)."""
    rc = (_native or _calls()).prefill(cfg, cu_seqlens, cache_lens, max_new_len,
                                            max_total_len, q_rot, cache, out, gate, workspace,
                                            status, total_tokens, stream)
    if rc is None:
        batch, T = _prefill_args(cfg, cu_seqlens, cache_lens, q_rot, out, gate, status,
                                 total_tokens)
        kc = _paged(cache, cfg, batch)
        c = cfg.c()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        cu, lens, pq, pgate, po, ws, st = [
            _ptr(t) for t in (cu_seqlens, cache_lens, q_rot, gate, out, workspace, status)]
        _on_current(cu_seqlens, cache_lens, q_rot, gate, out, workspace, status, cache.k, cache.v,
                    cache.k_scale, cache.v_scale, cache.page_table)
        rc = load_library().na_attn_prefill_chunk_paged(
            ctypes.byref(c), batch, cu, lens, T, int(max_new_len), int(max_total_len), pq,
            ctypes.byref(kc), pgate, po, ws, ws_bytes, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_attn_prefill_chunk_paged", rc)


def _want_decode(cfg, q_rot, kv_lens, out, probs, gate, status):
    H, d = cfg.num_heads, cfg.head_dim
    shape, dtype = q_rot.shape, q_rot.dtype
    B = int(shape[0])
    if not (dtype is _dtypes.get("bfloat16") and shape[1:] == (H, d) and out.dtype is dtype
            and out.shape == shape):
        _want(q_rot, "q_rot", "bfloat16", (None, H, d))
        _want(out, "out", "bfloat16", (B, H, d))
    _want(gate, "gate", "bfloat16", (B, H, d))
    _want(kv_lens, "kv_lens", "int32", (None,), B)
    _want(probs, "probs", "float32", (B, H, None))
    _want(status, "status", "int32", (None,), 1)
    return B


def na_attn_decode(cfg: AttnConfig, q_rot, cache: KVCache, kv_lens, max_kv_len: int, out,
                   probs=None, gate=None, workspace=None, num_splits: int = 0, status=None,
                   stream=None):
    lib = load_library()
    batch = _want_decode(cfg, q_rot, kv_lens, out, probs, gate, status)
    _want_cache(cache, cfg, batch)
    c, kc = cfg.c(), cache.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    stride = int(probs.shape[-1]) if probs is not None else 0
    rc = lib.na_attn_decode(ctypes.byref(c), batch, _ptr(q_rot), ctypes.byref(kc), _ptr(kv_lens),
                            int(max_kv_len), _ptr(gate), _ptr(out), _ptr(probs), stride,
                            int(num_splits), _ptr(workspace), ws_bytes, _ptr(status),
                            _stream(stream))
    _check("na_attn_decode", rc)


def na_attn_decode_paged(cfg: AttnConfig, q_rot, cache: PagedKVCache, kv_lens, max_kv_len: int,
                         out, probs=None, gate=None, workspace=None, num_splits: int = 0,
                         status=None, stream=None):
    """na_attn_decode over bf16 or E4M3 pages (workspace: na_decode_paged_workspace_size)."""
    rc = (_native or _calls()).decode(cfg, q_rot, cache, kv_lens, max_kv_len, out, probs,
                                           gate, workspace, num_splits, status, stream)
    if rc is None:
        batch = _want_decode(cfg, q_rot, kv_lens, out, probs, gate, status)
        kc = _paged(cache, cfg, batch)
        c = cfg.c()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        stride = int(probs.shape[-1]) if probs is not None else 0
        pq, lens, pgate, po, pp, ws, st = [
            _ptr(t) for t in (q_rot, kv_lens, gate, out, probs, workspace, status)]
        _on_current(q_rot, kv_lens, gate, out, probs, workspace, status, cache.k, cache.v,
                    cache.k_scale, cache.v_scale, cache.page_table)
        rc = load_library().na_attn_decode_paged(
            ctypes.byref(c), batch, pq, ctypes.byref(kc), lens, int(max_kv_len), pgate, po, pp,
            stride, int(num_splits), ws, ws_bytes, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_attn_decode_paged", rc)


def na_attn_decode_static_ws(cfg: AttnConfig, q_rot, cache: KVCache, kv_lens, max_kv_len: int,
                             out, probs=None, gate=None, num_splits: int = 0, status=None,
                             stream=None):
    """na_attn_decode without a workspace argument: the split partials live in
    a fixed 20 MiB device array inside the library, for callers that cannot
    allocate device memory.  Calls that overlap on the GPU race on that array."""
    lib = load_library()
    batch = _want_decode(cfg, q_rot, kv_lens, out, probs, gate, status)
    _want_cache(cache, cfg, batch)
    c, kc = cfg.c(), cache.c()
    stride = int(probs.shape[-1]) if probs is not None else 0
    rc = lib.na_attn_decode_static_ws(ctypes.byref(c), batch, _ptr(q_rot), ctypes.byref(kc),
                                      _ptr(kv_lens), int(max_kv_len), _ptr(gate), _ptr(out),
                                      _ptr(probs), stride, int(num_splits), _ptr(status),
                                      _stream(stream))
    _check("na_attn_decode_static_ws", rc)


def na_decode_importance(cfg: AttnConfig, probs, kv_lens, max_kv_len: int, imp,
                         accumulate: bool = False, status=None, stream=None):
    """Born-rule importance of a decode step: imp[b][j] (+)= sum over heads of
    probs[b][h][j] for j < kv_lens[b].  probs [B,H,stride] fp32, imp [B,stride2]."""
    lib = load_library()
    _want(probs, "probs", "float32", (None, cfg.num_heads, None))
    B = int(probs.shape[0])
    _want(imp, "imp", "float32", (B, None))
    _want(kv_lens, "kv_lens", "int32", (None,), B)
    _want(status, "status", "int32", (None,), 1)
    c = cfg.c()
    rc = lib.na_decode_importance(ctypes.byref(c), int(probs.shape[0]), _ptr(probs),
                                  int(probs.shape[-1]), _ptr(kv_lens), int(max_kv_len), _ptr(imp),
                                  int(imp.shape[-1]), 1 if accumulate else 0, _ptr(status),
                                  _stream(stream))
    _check("na_decode_importance", rc)


def na_pages_fork(parents, lens, table, ref, page_size: int, new_table, new_ref, new_lens, copy_src,
                  copy_dst, grow=None, status=None, stream=None):
    """One step of a batch's page tables: sequence b continues parents[b] (< 0: starts empty) and
    gets room for grow[b] more tokens; the page copies that this needs are copy_src -> copy_dst
    (na_pages_copy)."""
    rc = (_native or _calls()).fork(parents, lens, table, ref, page_size, new_table, new_ref,
                                    new_lens, copy_src, copy_dst, grow, status, stream)
    if rc is None:
        _want(parents, "parents", "int32", (None,))
        _want(table, "table", "int32", (None, None))
        batch, (old, P) = int(parents.shape[0]), table.shape
        _want(lens, "lens", "int32", (old,))
        _want(ref, "ref", "int32", (None,))
        _want(new_table, "new_table", "int32", (batch, P))
        _want(new_ref, "new_ref", "int32", ref.shape)
        for t, name in ((new_lens, "new_lens"), (copy_src, "copy_src"), (copy_dst, "copy_dst"),
                        (grow, "grow")):
            _want(t, name, "int32", (batch,))
        _want(status, "status", "int32", (None,), 1)
        args = [_ptr(t) for t in (parents, grow, lens, table)]
        outs = [_ptr(t) for t in (new_table, new_ref, new_lens, copy_src, copy_dst, status)]
        pref = _ptr(ref)
        _on_current(parents, grow, lens, table, ref, new_table, new_ref, new_lens, copy_src, copy_dst,
                    status)
        rc = load_library().na_pages_fork(
            batch, old, *args, P, int(page_size), pref, int(ref.shape[0]), *outs, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_pages_fork", rc)


def _pages(cache, name: str):
    """The C struct of a cache's pages (with its table where it has one), its tensors checked, and
    (kv heads, row width)."""
    if isinstance(cache, PagedLatentCache):
        _want(cache.kv, f"{name}.kv", "bfloat16", (None, None, None))
        pages, page, d = cache.kv.shape
        heads, tensors = 1, (cache.kv, None, None, None)
    else:
        kind = "bfloat16" if cache.k_scale is None and cache.v_scale is None else "float8_e4m3fn"
        _want(cache.k, f"{name}.k", kind, (None, None, None, None))
        _want(cache.v, f"{name}.v", kind, cache.k.shape)
        pages, heads, page, d = cache.k.shape
        tensors = (cache.k, cache.v, cache.k_scale, cache.v_scale)
        if kind != "bfloat16":
            for t, which in ((cache.k_scale, "k_scale"), (cache.v_scale, "v_scale")):
                if t is None:
                    raise ValueError(f"{name}.{which}: missing")
                _want(t, f"{name}.{which}", "uint8", (pages, heads))
    _want(cache.page_table, f"{name}.page_table", "int32", (None, None))
    batch, per = (0, 0) if cache.page_table is None else cache.page_table.shape
    c = na_paged_kv_cache(*(_ptr(t) for t in tensors), _ptr(cache.page_table), pages, page, batch,
                          per, NA_KV_BF16 if tensors[2] is None else NA_KV_E4M3)
    _on_current(*tensors, cache.page_table)
    return c, int(heads), int(d)


def na_pages_copy(cache, src, dst, status=None, stream=None):
    """Copy whole pages src[i] -> dst[i] of a PagedKVCache or PagedLatentCache (a negative entry:
    nothing)."""
    rc = (_native or _calls()).copy(cache, src, dst, status, stream)
    if rc is None:
        c, heads, d = _pages(cache, "cache")
        _want(src, "src", "int32", (None,))
        _want(dst, "dst", "int32", src.shape)
        _want(status, "status", "int32", (None,), 1)
        ps, pd, st = _ptr(src), _ptr(dst), _ptr(status)
        _on_current(src, dst, status)
        rc = load_library().na_pages_copy(
            heads, d, ctypes.byref(c), int(src.shape[0]), ps, pd, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_pages_copy", rc)


def na_pages_compact(cache, new_cache, keep_lens, max_keep: int, keep=None,
                     rope: Optional[RopeConfig] = None, rotary_start: int = 0,
                     rotary_dim: Optional[int] = None, interleaved: bool = False, status=None,
                     stream=None):
    """Move the rows at positions keep[b] of each sequence of `cache` (all in order with keep None)
    to the front of `new_cache`'s pages, keys turned to their new positions where rope is given
    (rotary_dim: by default from rotary_start to the row's end)."""
    rc = (_native or _calls()).compact(cache, new_cache, keep_lens, max_keep, keep, rope,
                                       rotary_start, rotary_dim, interleaved, status, stream)
    if rc is None:
        _want(keep_lens, "keep_lens", "int32", (None,))
        batch, max_keep = int(keep_lens.shape[0]), int(max_keep)
        a, heads, d = _pages(cache, "cache")
        z, new_heads, new_d = _pages(new_cache, "new_cache")
        if (heads, d) != (new_heads, new_d):
            raise ValueError(f"new_cache: rows of {new_heads} x {new_d}, the cache's are {heads} x {d}")
        if cache.page_table is None or new_cache.page_table is None:
            raise ValueError("both caches need a page table")
        _want(keep, "keep", "int32", (batch, max_keep))
        _want(status, "status", "int32", (None,), 1)
        pk, pl, st = _ptr(keep), _ptr(keep_lens), _ptr(status)
        _on_current(keep, keep_lens, status)
        r = None if rope is None else ctypes.byref(rope.c())
        rd = d - rotary_start if rotary_dim is None else rotary_dim
        rc = load_library().na_pages_compact(
            heads, d, batch, ctypes.byref(a), ctypes.byref(z), pk, pl, max_keep, r,
            int(rotary_start), 0 if r is None else int(rd),
            NA_ROPE_INTERLEAVED if interleaved else 0, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_pages_compact", rc)


def _latent_cache(cache: PagedLatentCache, cfg: LatentConfig, batch: int) -> na_paged_latent_cache:
    """The C struct of a latent cache, its tensors checked."""
    _want(cache.kv, "cache.kv", "bfloat16", (None, None, cfg.kv_rank + cfg.rope_dim))
    _want(cache.page_table, "cache.page_table", "int32", (None, None), batch)
    return cache.c()


def _rows(t, name: str, width: int):
    """Pointer and stride of rows of `width` bfloat16 elements, one behind the other at any distance
    (the last part of wider rows, say); (None, 0) for None."""
    if t is None:
        return None, 0
    _want(t, name, "bfloat16", (None,) * (t.dim() - 1) + (width,))
    if not t.is_cuda:
        raise ValueError("libna operates on CUDA tensors only")
    if t.numel() == 0:
        return None, width
    # the last dimension of rows gives their distance, those before it have to follow one another; a
    # dimension of size 1 has a stride that says nothing, and a single row any distance
    dims = [i for i in range(t.dim() - 1) if t.shape[i] > 1]
    if t.stride(-1) != 1 or any(t.stride(i) != t.stride(j) * t.shape[j] for i, j in zip(dims, dims[1:])):
        raise ValueError(f"{name}: rows have to be contiguous and equally far apart")
    return t.data_ptr(), t.stride(dims[-1]) if dims else width


def na_latent_append_paged(cfg: LatentConfig, rope: RopeConfig, cu_seqlens, cache_lens, kv, q, q_out,
                           cache: PagedLatentCache, kv_norm_w=None, status=None,
                           total_tokens: Optional[int] = None, stream=None):
    """New tokens' latent rows kv [T, kv_rank + rope_dim] into their pages (normed, their rotated part
    turned), and q_out = RoPE(q), both [T, H, rope_dim] and views of wider rows where wanted (or
    None)."""
    rc = (_native or _calls()).latent_append(cfg, rope, cu_seqlens, cache_lens, kv, q, q_out,
                                             cache, kv_norm_w, status, total_tokens, stream)
    if rc is None:
        T = int(kv.shape[0]) if total_tokens is None else int(total_tokens)
        batch = int(cu_seqlens.numel()) - 1
        _want(cu_seqlens, "cu_seqlens", "int32", (None,))
        _want(cache_lens, "cache_lens", "int32", (None,), batch)
        _want(kv, "kv", "bfloat16", (None, None), T)
        for t, name in ((q, "q"), (q_out, "q_out")):
            _want(t, name, "bfloat16", (None, cfg.num_heads, cfg.rope_dim), T)
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        _want(kv_norm_w, "kv_norm_w", "bfloat16", (cfg.kv_rank,))
        _want(status, "status", "int32", (None,), 1)
        kc = _latent_cache(cache, cfg, batch)
        pkv, kv_stride = _rows(kv, "kv", cfg.kv_rank + cfg.rope_dim)
        pq, q_stride = _rows(q, "q", cfg.rope_dim)
        po, out_stride = _rows(q_out, "q_out", cfg.rope_dim)
        c, r = cfg.c(), rope.c()
        cu, lens, w, st = [_ptr(t) for t in (cu_seqlens, cache_lens, kv_norm_w, status)]
        _on_current(cu_seqlens, cache_lens, kv, q, q_out, kv_norm_w, status, cache.kv, cache.page_table)
        rc = load_library().na_latent_append_paged(
            ctypes.byref(c), ctypes.byref(r), batch, cu, lens, T, pkv, kv_stride, pq, q_stride,
            po, out_stride, w, ctypes.byref(kc), st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_latent_append_paged", rc)


def na_latent_paged_workspace_size(cfg: LatentConfig, batch: int, total_tokens: int, max_new_len: int,
                                   max_total_len: int) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    c = cfg.c()
    _check("na_latent_paged_workspace_size",
           lib.na_latent_paged_workspace_size(ctypes.byref(c), batch, total_tokens, max_new_len,
                                              max_total_len, ctypes.byref(out)))
    return int(out.value)


def na_attn_latent_paged(cfg: LatentConfig, cu_seqlens, cache_lens, max_new_len: int,
                         max_total_len: int, q_lat, cache: PagedLatentCache, out, workspace=None,
                         status=None, total_tokens: Optional[int] = None, stream=None):
    """Absorbed latent attention of new tokens (single ones or chunks) against the pages: q_lat
    [T, H, kv_rank + rope_dim], out [T, H, kv_rank] (workspace: na_latent_paged_workspace_size)."""
    rc = (_native or _calls()).latent(cfg, cu_seqlens, cache_lens, max_new_len, max_total_len,
                                      q_lat, cache, out, workspace, status, total_tokens, stream)
    if rc is None:
        T = int(q_lat.shape[0]) if total_tokens is None else int(total_tokens)
        batch, H = int(cu_seqlens.numel()) - 1, cfg.num_heads
        _want(cu_seqlens, "cu_seqlens", "int32", (None,))
        _want(cache_lens, "cache_lens", "int32", (None,), batch)
        _want(q_lat, "q_lat", "bfloat16", (None, H, cfg.kv_rank + cfg.rope_dim), T)
        _want(out, "out", "bfloat16", (None, H, cfg.kv_rank), T)
        _want(status, "status", "int32", (None,), 1)
        kc = _latent_cache(cache, cfg, batch)
        c = cfg.c()
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        cu, lens, pq, po, ws, st = [_ptr(t) for t in (cu_seqlens, cache_lens, q_lat, out, workspace, status)]
        _on_current(cu_seqlens, cache_lens, q_lat, out, workspace, status, cache.kv, cache.page_table)
        rc = load_library().na_attn_latent_paged(
            ctypes.byref(c), batch, cu, lens, T, int(max_new_len), int(max_total_len), pq,
            ctypes.byref(kc), po, ws, ws_bytes, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_attn_latent_paged", rc)


def na_attn_latent_expanded(cfg: LatentConfig, cu_seqlens, key_starts, key_lens, max_new_len: int,
                            max_key_len: int, q, kv, k_pe, out, status=None,
                            total_tokens: Optional[int] = None, stream=None):
    """Expanded latent attention, causal: q [T, H, nope_dim + rope_dim] against kv [keys, H,
    nope_dim + v_dim] and the shared k_pe [keys, rope_dim] (a view of wider rows where wanted); out
    [T, H, v_dim].  Sequence b's keys are rows key_starts[b] .. + key_lens[b] - 1."""
    rc = (_native or _calls()).expanded(cfg, cu_seqlens, key_starts, key_lens, max_new_len,
                                        max_key_len, q, kv, k_pe, out, status, total_tokens,
                                        stream)
    if rc is None:
        T = int(q.shape[0]) if total_tokens is None else int(total_tokens)
        batch, H = int(cu_seqlens.numel()) - 1, cfg.num_heads
        _want(cu_seqlens, "cu_seqlens", "int32", (None,))
        _want(key_starts, "key_starts", "int32", (None,), batch)
        _want(key_lens, "key_lens", "int32", (None,), batch)
        _want(q, "q", "bfloat16", (None, H, cfg.nope_dim + cfg.rope_dim), T)
        _want(kv, "kv", "bfloat16", (None, H, cfg.nope_dim + cfg.v_dim))
        _want(k_pe, "k_pe", "bfloat16", (None, None), int(kv.shape[0]))
        _want(out, "out", "bfloat16", (None, H, cfg.v_dim), T)
        _want(status, "status", "int32", (None,), 1)
        pe, stride = _rows(k_pe, "k_pe", cfg.rope_dim)
        c = cfg.c()
        cu, starts, lens, pq, pkv, po, st = [
            _ptr(t) for t in (cu_seqlens, key_starts, key_lens, q, kv, out, status)]
        _on_current(cu_seqlens, key_starts, key_lens, q, kv, k_pe, out, status)
        rc = load_library().na_attn_latent_expanded(
            ctypes.byref(c), batch, cu, starts, lens, T, int(kv.shape[0]), int(max_new_len),
            int(max_key_len), pq, pkv, pe, stride, po, st, _stream(stream))
    if rc != NA_OK:
        raise NAError("na_attn_latent_expanded", rc)


def na_selftest_wait_timeout(status, stream=None):
    """Run the library's bounded device wait on a barrier nothing completes:
    after about a second `status` holds NA_ERR_DEVICE_TIMEOUT."""
    _check("na_selftest_wait_timeout",
           load_library().na_selftest_wait_timeout(_ptr(status), _stream(stream)))


def workspace(nbytes: int, device="cuda"):
    """A byte tensor usable as workspace (None when nbytes is 0)."""
    import torch
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)
