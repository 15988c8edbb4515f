"""Binding of the serving entry points in include/sdpa_serve.h.

As in binding.py, every function turns torch tensors into pointers, sizes and
strides, calls the entry point of the same name on the current CUDA stream and
raises on a status; arithmetic runs in the library's kernels, and a missing
library raises.  The calls sit in a generation loop whose kernels take a few
microseconds, so their marshalling is compiled (_serve.so, csrc/serve/
serve_bind.cpp); the ctypes signatures here declare the same ABI for callers
that bring their own pointers.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .binding import BiasDesc, SdpaError, _check

_PKG = os.path.dirname(os.path.abspath(__file__))
SERVE_LIB_PATH = os.path.join(_PKG, "libsdpa_serve_b200.so")
BIND_PATH = os.path.join(_PKG, "_serve.so")

SERVE_EXPORTED = ("sdpa_rope", "sdpa_rope_frequencies", "sdpa_cache_append", "sdpa_cache_gather",
                  "sdpa_tree_fwd", "sdpa_tree_fwd_workspace_size", "sdpa_spec_verify",
                  "sdpa_serve_read_device_status", "sdpa_serve_set_wait_limit_ns")

CACHE_BF16, CACHE_E4M3 = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class RopeDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in
                 ("B", "L", "Hq", "Hkv", "d", "q_b", "q_l", "q_h", "k_b", "k_l", "k_h",
                  "qo_b", "qo_l", "qo_h", "ko_b", "ko_l", "ko_h")]
                + [("positions", ctypes.c_void_p), ("pos_b", ctypes.c_int64),
                   ("offset", ctypes.c_int64), ("freqs", ctypes.c_void_p),
                   ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                   ("inverse", ctypes.c_int32), ("amplitude", ctypes.c_float)])


class KvCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [("format", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in
                   ("num_pages", "page_size", "Hkv", "d", "stride_page", "stride_head",
                    "stride_row", "scale_stride_page", "scale_stride_head")])


class Tree(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "T", "max_nodes", "Hq", "q_t", "q_h", "o_t",
                                               "o_h")]
                + [(n, ctypes.c_void_p) for n in ("cu_nodes", "ctx_lens", "page_table")]
                + [("table_width", ctypes.c_int64), ("table_b", ctypes.c_int64),
                   ("tree_mask", ctypes.c_void_p), ("window_left", ctypes.c_int64)])


class Verify(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "N", "V", "target_b", "target_n", "draft_b",
                                               "draft_n")]
                + [(n, ctypes.c_void_p) for n in ("target", "draft", "tokens", "parents",
                                                  "u_accept", "u_sample")])


_lib = None
_bind = None
_wait_limit_ns = None    # set before the library was loaded


def load_serve_library(path: str | None = None) -> ctypes.CDLL:
    """Load libsdpa_serve_b200.so once and declare the signatures.  Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or SERVE_LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} (run scaled_dot_product_bwd_b200.build)")
    lib = ctypes.CDLL(p)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    bp = ctypes.POINTER(BiasDesc)
    cp = ctypes.POINTER(KvCache)
    f64 = ctypes.c_double
    lib.sdpa_rope.argtypes = [ctypes.POINTER(RopeDesc), vp, vp, vp, vp, vp]
    lib.sdpa_rope.restype = i32
    lib.sdpa_rope_frequencies.argtypes = [i32, f64, i32, f64, i64, f64, f64,
                                          ctypes.POINTER(f64), ctypes.POINTER(f32)]
    lib.sdpa_rope_frequencies.restype = i32
    lib.sdpa_cache_append.argtypes = [cp, vp, vp, i64, i64, i64, vp, vp]
    lib.sdpa_cache_append.restype = i32
    lib.sdpa_cache_gather.argtypes = [cp, i64, vp, i64, i64, vp, i64, vp, vp, i64, i64, vp]
    lib.sdpa_cache_gather.restype = i32
    tp = ctypes.POINTER(Tree)
    lib.sdpa_tree_fwd.argtypes = [tp, cp, vp, bp, f32, vp, vp, vp, sz, vp]
    lib.sdpa_tree_fwd.restype = i32
    lib.sdpa_tree_fwd_workspace_size.argtypes = [tp, cp]
    lib.sdpa_tree_fwd_workspace_size.restype = sz
    lib.sdpa_spec_verify.argtypes = [ctypes.POINTER(Verify), vp, vp, vp, vp]
    lib.sdpa_spec_verify.restype = i32
    lib.sdpa_serve_read_device_status.argtypes = [vp]
    lib.sdpa_serve_read_device_status.restype = i32
    lib.sdpa_serve_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.sdpa_serve_set_wait_limit_ns.restype = None
    if path is None:
        _lib = lib
        if _wait_limit_ns is not None:
            lib.sdpa_serve_set_wait_limit_ns(_wait_limit_ns)
    return lib


def _load_bind():
    """The compiled marshalling module, loaded once.  Raises if absent."""
    global _bind
    if _bind is None:
        if not os.path.exists(BIND_PATH):
            raise RuntimeError(f"not built: {BIND_PATH} (run scaled_dot_product_bwd_b200.build)")
        import importlib.machinery
        import importlib.util
        loader = importlib.machinery.ExtensionFileLoader("_serve", BIND_PATH)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_serve", loader))
        loader.exec_module(mod)
        mod.set_error((SdpaError, torch.OutOfMemoryError))
        load_serve_library()
        _bind = mod
    return _bind


def read_device_status(stream) -> int:
    """The serving kernels' status on `stream`'s device (0 while the library is not loaded)."""
    return 0 if _lib is None else int(_lib.sdpa_serve_read_device_status(stream))


def set_wait_limit_ns(ns: int):
    """The wait limit of the serving kernels, now or (a program that only trains need not have
    the library) as soon as it is loaded."""
    global _wait_limit_ns
    _wait_limit_ns = ns
    if _lib is not None:
        _lib.sdpa_serve_set_wait_limit_ns(ns)


def sdpa_rope_frequencies(rot, base=10000.0, *, scaling="none", factor=1.0, original_length=0,
                          beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freqs float64 [rot / 2] on ``device``, amplitude) for sdpa_rope: radians per position,
    unscaled or scaled for longer contexts ("linear", "ntk", "yarn"; see include/sdpa_serve.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(int(rot) // 2, 1))()
    amplitude = ctypes.c_float()
    _check(load_serve_library().sdpa_rope_frequencies(int(rot), float(base), ROPE_SCALINGS[scaling],
                                                float(factor), int(original_length),
                                                float(beta_fast), float(beta_slow), out,
                                                ctypes.byref(amplitude)), "sdpa_rope_frequencies")
    return torch.tensor(list(out), dtype=torch.float64, device=device), amplitude.value


def sdpa_rope(q, k, freqs, positions=None, *, offset=0, interleaved=False, inverse=False,
              amplitude=1.0, out_q=None, out_k=None):
    """q and k turned by their positions (see sdpa_rope in include/sdpa_serve.h): (out_q, out_k).

    q [B, L, Hq, d] and k [B, L, Hkv, d], or packed [T, Hq, d] and [T, Hkv, d]; k may be None.
    ``positions`` int32 [B, L] (or [T]); without it row l has position ``offset`` + l.
    ``inverse`` turns back: the gradient.  out_q=q, out_k=k works in place.
    """
    return (_bind or _load_bind()).rope(q, k, freqs, positions, out_q, out_k, offset, interleaved,
                                        inverse, amplitude)


def sdpa_cache_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Rows k, v [T, Hkv, d] into the cache at slots int64 [T] (page * page_size + row;
    negative: skipped), quantised if the cache is e4m3 (see sdpa_cache_append).  Where k and v differ
    in strides (a rotated k, and v still a slice of a fused buffer) that is two launches."""
    (_bind or _load_bind()).append(k_cache, v_cache, k_scale, v_scale, k, v, slots)


def sdpa_cache_gather(k_cache, v_cache, page_table, cu_seqlens, total, k_scale=None, v_scale=None,
                      k=None, v=None):
    """The cached sequences as packed bf16 (k, v) [total, Hkv, d], sequence b's first
    cu_seqlens[b + 1] - cu_seqlens[b] positions at its rows: the keys and values over which
    sdpa_fwd_varlen attends from a prompt's next chunk (see sdpa_cache_gather for its limits)."""
    return (_bind or _load_bind()).gather(k_cache, v_cache, k_scale, v_scale, page_table,
                                          cu_seqlens, total, k, v)


def sdpa_tree_fwd(q, k_cache, v_cache, page_table, ctx_lens, cu_nodes, max_nodes, *,
                  k_scale=None, v_scale=None, tree_mask=None, window_left=-1, t5_table=None,
                  t5_num_buckets=32, t5_max_distance=128, t5_bidirectional=True,
                  alibi_slopes=None, scale=None, out=None, lse=None, workspace=None):
    """O [T, Hq, d], LSE [Hq, T]: each sequence's nodes over its cached context and over the
    nodes that ``tree_mask`` (int64 [T], bit j: sees node j; None: a chain) shows them.  One node
    per sequence is plain decoding.  The nodes' own keys are in the cache already, at positions
    ctx_lens[b] and on (see sdpa_tree_fwd in include/sdpa_serve.h)."""
    return (_bind or _load_bind()).tree(k_cache, v_cache, k_scale, v_scale, q, page_table, ctx_lens,
                                        cu_nodes, max_nodes, tree_mask, window_left, t5_table,
                                        t5_num_buckets, t5_max_distance, t5_bidirectional,
                                        alibi_slopes, scale, out, lse, workspace, False)


def sdpa_tree_fwd_workspace_size(q, k_cache, v_cache, page_table, ctx_lens, cu_nodes, max_nodes, *,
                                 k_scale=None, v_scale=None) -> int:
    """Bytes of the workspace of sdpa_tree_fwd for these tensors (0: they do not fit together)."""
    return (_bind or _load_bind()).tree(k_cache, v_cache, k_scale, v_scale, q, page_table, ctx_lens,
                                        cu_nodes, max_nodes, None, -1, None, 0, 0, False, None,
                                        None, None, None, None, True)


def sdpa_spec_verify(target, draft, tokens, parents, u_accept, u_sample):
    """(path int32 [B, N], accepted int32 [B], next_token int32 [B]) of drafted trees, by
    rejection sampling with the given uniform numbers (see sdpa_spec_verify in include/sdpa_serve.h).

    target, draft float32 [B, N, V]: the distributions after each node (draft may be None when
    N = 1); tokens int32 [B, N]; parents int32 [B, N] or None (a chain); u_accept float32 [B, N];
    u_sample float32 [B].
    """
    return (_bind or _load_bind()).verify(target, draft, tokens, parents, u_accept, u_sample)
