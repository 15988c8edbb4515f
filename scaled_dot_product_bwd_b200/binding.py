"""ctypes binding of the C ABI in include/sdpa.h (argument marshalling only).

Every function here converts torch tensors into pointers, sizes and strides,
calls the entry point of the same name in libsdpa_b200.so on the current CUDA
stream, and turns a non-OK status into an exception.  All arithmetic runs in
the library's kernels; there is no fallback: if the library is missing or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsdpa_b200.so")

SDPA_OK = 0
STATUS_NAMES = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARG", 2: "SDPA_ERR_UNSUPPORTED",
                3: "SDPA_ERR_WORKSPACE", 4: "SDPA_ERR_CUDA", 5: "SDPA_ERR_TIMEOUT"}
BIAS_NONE, BIAS_DENSE, BIAS_T5, BIAS_ALIBI, BIAS_REL = 0, 1, 2, 3, 4

BWD_PREPROCESS, BWD_DQ, BWD_DKDV, BWD_ALL = 1, 2, 4, 7

NOALLOC_SCRATCH_BYTES = 16 << 20

EXPORTED = ("sdpa_fwd", "sdpa_fwd_varlen", "sdpa_bwd", "sdpa_bwd_phases", "sdpa_bwd_varlen",
            "sdpa_bwd_noalloc", "sdpa_bwd_workspace_size", "sdpa_bwd_varlen_workspace_size",
            "sdpa_bwd_bias_grad", "sdpa_bwd_bias_grad_workspace_size", "sdpa_t5_bucket",
            "sdpa_exp2_fma", "sdpa_read_device_status", "sdpa_set_wait_limit_ns",
            "sdpa_debug_wait_timeout", "sdpa_status_string", "sdpa_fire_table",
            "sdpa_fire_backward_workspace_size", "sdpa_fire_backward", "sdpa_rope",
            "sdpa_rope_frequencies", "sdpa_cache_append", "sdpa_cache_gather", "sdpa_tree_fwd",
            "sdpa_tree_fwd_workspace_size", "sdpa_spec_verify")

CACHE_BF16, CACHE_E4M3 = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class SdpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class MaskSpec(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("window_left", ctypes.c_int64),
                ("window_right", ctypes.c_int64)]


class BiasDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("ptr", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_i", ctypes.c_int64), ("num_buckets", ctypes.c_int32),
                ("max_distance", ctypes.c_int32), ("bidirectional", ctypes.c_int32)]


class Fire(ctypes.Structure):
    _fields_ = [("w1", ctypes.c_void_p), ("b1", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("b2", ctypes.c_void_p), ("c", ctypes.c_float), ("threshold", ctypes.c_float),
                ("width", ctypes.c_int32), ("heads", ctypes.c_int32)]


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("B", "L", "Hq", "Hkv", "d", "sq_b", "sq_l", "sq_h", "skv_b", "skv_l", "skv_h",
                 "Lk")]


class Varlen(ctypes.Structure):
    _fields_ = [("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("max_seqlen_q", ctypes.c_int64), ("max_seqlen_k", ctypes.c_int64),
                ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64)]


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


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libsdpa_b200.so once and declare the signatures.  Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} (run scaled_dot_product_bwd_b200.build)")
    lib = ctypes.CDLL(p)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    sp, bp, mp = ctypes.POINTER(Shape), ctypes.POINTER(BiasDesc), ctypes.POINTER(MaskSpec)
    vlp = ctypes.POINTER(Varlen)
    lib.sdpa_fwd.argtypes = [sp, vp, vp, vp, bp, mp, f32, vp, vp, vp]
    lib.sdpa_fwd.restype = i32
    lib.sdpa_fwd_varlen.argtypes = [sp, vlp, vp, vp, vp, bp, mp, f32, vp, vp, vp]
    lib.sdpa_fwd_varlen.restype = i32
    lib.sdpa_bwd.argtypes = [sp, vp, vp, vp, vp, vp, vp, bp, mp, f32, vp, vp, vp, i32, vp, sz, vp]
    lib.sdpa_bwd.restype = i32
    lib.sdpa_bwd_varlen.argtypes = [sp, vlp] + lib.sdpa_bwd.argtypes[1:]
    lib.sdpa_bwd_varlen.restype = i32
    lib.sdpa_bwd_varlen_workspace_size.argtypes = [sp, vlp]
    lib.sdpa_bwd_varlen_workspace_size.restype = sz
    lib.sdpa_bwd_phases.argtypes = [ctypes.c_uint32] + lib.sdpa_bwd.argtypes
    lib.sdpa_bwd_phases.restype = i32
    lib.sdpa_bwd_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, bp, mp, f32, vp, vp, vp, i32, vp]
    lib.sdpa_bwd_noalloc.restype = i32
    lib.sdpa_bwd_workspace_size.argtypes = [sp, i32]
    lib.sdpa_bwd_workspace_size.restype = sz
    lib.sdpa_bwd_bias_grad.argtypes = [sp, vp, vp, vp, vp, vp, vp, bp, mp, f32, vp, vp, vp, vp,
                                       i32, vp, sz, vp]
    lib.sdpa_bwd_bias_grad.restype = i32
    lib.sdpa_bwd_bias_grad_workspace_size.argtypes = [sp, bp]
    lib.sdpa_bwd_bias_grad_workspace_size.restype = sz
    lib.sdpa_t5_bucket.argtypes = [vp, vp, i64, i32, i32, i32, vp]
    lib.sdpa_t5_bucket.restype = i32
    lib.sdpa_exp2_fma.argtypes = [vp, vp, i64, vp]
    lib.sdpa_exp2_fma.restype = i32
    lib.sdpa_read_device_status.argtypes = [vp]
    lib.sdpa_read_device_status.restype = i32
    lib.sdpa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.sdpa_set_wait_limit_ns.restype = None
    lib.sdpa_debug_wait_timeout.argtypes = [vp]
    lib.sdpa_debug_wait_timeout.restype = i32
    fp = ctypes.POINTER(Fire)
    lib.sdpa_fire_table.argtypes = [fp, i64, i64, vp, vp]
    lib.sdpa_fire_table.restype = i32
    lib.sdpa_fire_backward_workspace_size.argtypes = [fp, i64, i64]
    lib.sdpa_fire_backward_workspace_size.restype = sz
    lib.sdpa_fire_backward.argtypes = [fp, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.sdpa_fire_backward.restype = i32
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
    lib.sdpa_status_string.argtypes = [i32]
    lib.sdpa_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def _check(status: int, where: str):
    if status != SDPA_OK:
        raise SdpaError(status, where)


def _stream(t: torch.Tensor | None = None):
    dev = t.device if t is not None else torch.device("cuda")
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def make_shape(q: torch.Tensor, k: torch.Tensor) -> Shape:
    """Shape of q [B, L, Hq, d] against k [B, Lk, Hkv, d] (Lk may differ from L)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, L, H, d]")
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"k shape {tuple(k.shape)} does not match q {tuple(q.shape)}")
    if q.stride(-1) != 1 or k.stride(-1) != 1:
        raise ValueError("head_dim must be contiguous")
    return Shape(B, L, Hq, Hkv, d, q.stride(0), q.stride(1), q.stride(2),
                 k.stride(0), k.stride(1), k.stride(2), k.shape[1])


def make_varlen_shape(q: torch.Tensor, k: torch.Tensor, batch: int) -> Shape:
    """Shape of packed q [total_q, Hq, d] and k [total_k, Hkv, d] with `batch` sequences."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("packed q and k must be [total, H, d]")
    if q.shape[2] != k.shape[2]:
        raise ValueError("q and k head dims differ")
    if q.stride(-1) != 1 or k.stride(-1) != 1:
        raise ValueError("head_dim must be contiguous")
    return Shape(int(batch), 0, q.shape[1], k.shape[1], q.shape[2], 0, q.stride(0), q.stride(1),
                 0, k.stride(0), k.stride(1), 0)


def make_varlen(cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                max_seqlen_k: int, total_q: int, total_k: int) -> Varlen:
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 1:
            raise ValueError(f"{n} must be a contiguous int32 CUDA vector")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B + 1 entries")
    return Varlen(cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), int(max_seqlen_q),
                  int(max_seqlen_k), int(total_q), int(total_k))


def make_mask(causal: bool, window_left: int, window_right: int) -> MaskSpec:
    return MaskSpec(1 if causal else 0, int(window_left), int(window_right))


def make_bias(bias: torch.Tensor | None, t5_table: torch.Tensor | None, num_buckets: int,
              max_distance: int, bidirectional: bool, dims: tuple | None = None,
              alibi_slopes: torch.Tensor | None = None,
              rel_table: torch.Tensor | None = None) -> BiasDesc:
    """Bias descriptor; ``dims`` = (B, Hq, L) of the attention checks the shapes."""
    if sum(x is not None for x in (bias, t5_table, alibi_slopes, rel_table)) > 1:
        raise ValueError("give one of a dense bias, a T5 table, ALiBi slopes or a relative table")
    if rel_table is not None:
        if (rel_table.dtype != torch.float32 or rel_table.dim() != 2
                or not rel_table.is_contiguous()):
            raise ValueError("relative table must be contiguous float32 [Lq + Lk - 1, Hq]")
        if dims is not None:
            if rel_table.shape[1] != dims[1]:
                raise ValueError("relative table columns must equal the query heads")
            if len(dims) > 2 and dims[2] > 0:
                Lk = dims[3] if len(dims) > 3 else dims[2]
                if rel_table.shape[0] != dims[2] + Lk - 1:
                    raise ValueError("relative table must have Lq + Lk - 1 rows")
        return BiasDesc(BIAS_REL, rel_table.data_ptr(), 0, 0, 0, 0, 0, 0)
    if alibi_slopes is not None:
        if (alibi_slopes.dtype != torch.float32 or alibi_slopes.dim() != 1
                or not alibi_slopes.is_contiguous()):
            raise ValueError("ALiBi slopes must be a contiguous float32 [Hq] vector")
        if dims is not None and alibi_slopes.shape[0] != dims[1]:
            raise ValueError("ALiBi slopes must have one entry per query head")
        return BiasDesc(BIAS_ALIBI, alibi_slopes.data_ptr(), 0, 0, 0, 0, 0, 0)
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() != 4 or bias.stride(-1) != 1:
            raise ValueError("dense bias must be float32 [B|1, H|1, L, L] with j contiguous")
        if dims is not None:
            B, Hq, L = dims[:3]
            Lk = dims[3] if len(dims) > 3 else L
            if (bias.shape[0] not in (1, B) or bias.shape[1] not in (1, Hq)
                    or tuple(bias.shape[2:]) != (L, Lk)):
                raise ValueError(f"dense bias shape {tuple(bias.shape)} is not "
                                 f"[{B}|1, {Hq}|1, {L}, {Lk}]")
        sb = bias.stride(0) if bias.shape[0] > 1 else 0
        sh = bias.stride(1) if bias.shape[1] > 1 else 0
        return BiasDesc(BIAS_DENSE, bias.data_ptr(), sb, sh, bias.stride(2), 0, 0, 0)
    if t5_table is not None:
        if t5_table.dtype != torch.float32 or not t5_table.is_contiguous():
            raise ValueError("T5 table must be contiguous float32 [num_buckets, Hq]")
        if t5_table.dim() != 2 or t5_table.shape[0] != num_buckets:
            raise ValueError("T5 table must be [num_buckets, Hq]")
        if dims is not None and t5_table.shape[1] != dims[1]:
            raise ValueError("T5 table columns must equal the query heads")
        return BiasDesc(BIAS_T5, t5_table.data_ptr(), 0, 0, 0, int(num_buckets),
                        int(max_distance), 1 if bidirectional else 0)
    return BiasDesc(BIAS_NONE, None, 0, 0, 0, 0, 0, 0)


def _same_layout(a: torch.Tensor, ref: torch.Tensor, name: str):
    if a.shape != ref.shape or a.stride() != ref.stride() or a.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bf16 with the shape and strides of its partner")


def sdpa_fwd(q, k, v, *, causal=False, window_left=-1, window_right=-1, bias=None,
             t5_table=None, t5_num_buckets=32, t5_max_distance=128, t5_bidirectional=True,
             alibi_slopes=None, rel_table=None, scale=None, out=None, lse=None):
    """O, LSE = attention forward (see sdpa_fwd in include/sdpa.h)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise ValueError(f"{n} must be a bf16 CUDA tensor")
    shape = make_shape(q, k)
    _same_layout(v, k, "v")
    B, L, Hq, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    _same_layout(out, q, "out")
    if lse is None:
        lse = torch.empty(B, Hq, L, device=q.device, dtype=torch.float32)
    if lse.shape != (B, Hq, L) or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError("lse must be contiguous float32 [B, Hq, L]")
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bd = make_bias(bias, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (B, Hq, L, k.shape[1]), alibi_slopes, rel_table)
    m = make_mask(causal, window_left, window_right)
    st = lib.sdpa_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(bd),
                      ctypes.byref(m), sc, _ptr(out), _ptr(lse), _stream(q))
    _check(st, "sdpa_fwd")
    return out, lse


def sdpa_bwd_workspace_size(q, k, deterministic: bool = True) -> int:
    lib = load_library()
    shape = make_shape(q, k)
    return int(lib.sdpa_bwd_workspace_size(ctypes.byref(shape), 1 if deterministic else 0))


def sdpa_bwd(q, k, v, o, do, lse, *, causal=False, window_left=-1, window_right=-1,
             bias=None, t5_table=None, t5_num_buckets=32, t5_max_distance=128,
             t5_bidirectional=True, alibi_slopes=None, rel_table=None,
             scale=None, dq=None, dk=None, dv=None,
             workspace=None, deterministic=True, phases=BWD_ALL):
    """dQ, dK, dV = attention backward (see sdpa_bwd / sdpa_bwd_phases in include/sdpa.h).

    ``phases`` selects launches (BWD_PREPROCESS | BWD_DQ | BWD_DKDV); the
    default runs all three in order.  DQ and DKDV read D from the workspace
    of an earlier PREPROCESS call on the same O and dO.
    """
    lib = load_library()
    shape = make_shape(q, k)
    _same_layout(v, k, "v")
    _same_layout(o, q, "o")
    _same_layout(do, q, "do")
    d = q.shape[-1]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _same_layout(dq, q, "dq")
    _same_layout(dk, k, "dk")
    _same_layout(dv, k, "dv")
    need = int(lib.sdpa_bwd_workspace_size(ctypes.byref(shape), 1))
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=q.device, dtype=torch.uint8)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bd = make_bias(bias, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (q.shape[0], q.shape[2], q.shape[1], k.shape[1]), alibi_slopes, rel_table)
    m = make_mask(causal, window_left, window_right)
    args = (ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
            ctypes.byref(bd), ctypes.byref(m), sc, _ptr(dq), _ptr(dk), _ptr(dv),
            1 if deterministic else 0, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(q))
    if phases == BWD_ALL:
        _check(lib.sdpa_bwd(*args), "sdpa_bwd")
    else:
        _check(lib.sdpa_bwd_phases(int(phases), *args), "sdpa_bwd_phases")
    return dq, dk, dv


def sdpa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, *, causal=False, window_left=-1,
                     window_right=-1, bias=None, t5_table=None, t5_num_buckets=32,
                     t5_max_distance=128, t5_bidirectional=True, alibi_slopes=None, rel_table=None,
                     scale=None):
    """Backward into caller-given dQ, dK, dV with no workspace and no allocation.

    For callers that cannot allocate device memory: the library's built-in
    scratch array (NOALLOC_SCRATCH_BYTES) stands in for the workspace, so the
    shape's sdpa_bwd_workspace_size must fit in it.  Calls that overlap on
    the GPU race on that array.
    """
    lib = load_library()
    shape = make_shape(q, k)
    for t, ref, n in ((v, k, "v"), (o, q, "o"), (do, q, "do"), (dq, q, "dq"), (dk, k, "dk"),
                      (dv, k, "dv")):
        _same_layout(t, ref, n)
    sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    bd = make_bias(bias, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (q.shape[0], q.shape[2], q.shape[1], k.shape[1]), alibi_slopes, rel_table)
    m = make_mask(causal, window_left, window_right)
    st = lib.sdpa_bwd_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do),
                              _ptr(lse), ctypes.byref(bd), ctypes.byref(m), sc, _ptr(dq),
                              _ptr(dk), _ptr(dv), 1, _stream(q))
    _check(st, "sdpa_bwd_noalloc")
    return dq, dk, dv


def sdpa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, *,
                    causal=False, window_left=-1, window_right=-1, t5_table=None,
                    t5_num_buckets=32, t5_max_distance=128, t5_bidirectional=True,
                    alibi_slopes=None, rel_table=None, scale=None, out=None, lse=None):
    """O [total_q, Hq, d], LSE [Hq, total_q] of a packed batch (sdpa_fwd_varlen)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise ValueError(f"{n} must be a bf16 CUDA tensor")
    _same_layout(v, k, "v")
    B = cu_seqlens_q.numel() - 1
    shape = make_varlen_shape(q, k, B)
    vl = make_varlen(cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, q.shape[0],
                     k.shape[0])
    total_q, Hq, d = q.shape
    out = torch.empty_like(q) if out is None else out
    _same_layout(out, q, "out")
    if lse is None:
        lse = torch.empty(Hq, total_q, device=q.device, dtype=torch.float32)
    if lse.shape != (Hq, total_q) or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError("lse must be contiguous float32 [Hq, total_q]")
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bd = make_bias(None, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (B, q.shape[1], 0, 0), alibi_slopes, rel_table)
    m = make_mask(causal, window_left, window_right)
    st = lib.sdpa_fwd_varlen(ctypes.byref(shape), ctypes.byref(vl), _ptr(q), _ptr(k), _ptr(v),
                             ctypes.byref(bd), ctypes.byref(m), sc, _ptr(out), _ptr(lse),
                             _stream(q))
    _check(st, "sdpa_fwd_varlen")
    return out, lse


def sdpa_bwd_varlen(q, k, v, o, do, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    max_seqlen_k, *, causal=False, window_left=-1, window_right=-1,
                    t5_table=None, t5_num_buckets=32, t5_max_distance=128,
                    t5_bidirectional=True, alibi_slopes=None, rel_table=None,
                    scale=None, dq=None, dk=None,
                    dv=None, workspace=None):
    """dQ, dK, dV of a packed batch (sdpa_bwd_varlen)."""
    lib = load_library()
    _same_layout(v, k, "v")
    _same_layout(o, q, "o")
    _same_layout(do, q, "do")
    B = cu_seqlens_q.numel() - 1
    shape = make_varlen_shape(q, k, B)
    vl = make_varlen(cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, q.shape[0],
                     k.shape[0])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _same_layout(dq, q, "dq")
    _same_layout(dk, k, "dk")
    _same_layout(dv, k, "dv")
    need = int(lib.sdpa_bwd_varlen_workspace_size(ctypes.byref(shape), ctypes.byref(vl)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=q.device, dtype=torch.uint8)
    sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    bd = make_bias(None, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (B, q.shape[1], 0, 0), alibi_slopes, rel_table)
    m = make_mask(causal, window_left, window_right)
    st = lib.sdpa_bwd_varlen(ctypes.byref(shape), ctypes.byref(vl), _ptr(q), _ptr(k), _ptr(v),
                             _ptr(o), _ptr(do), _ptr(lse), ctypes.byref(bd), ctypes.byref(m), sc,
                             _ptr(dq), _ptr(dk), _ptr(dv), 1, _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(q))
    _check(st, "sdpa_bwd_varlen")
    return dq, dk, dv


def sdpa_bwd_bias_grad_workspace_size(q, k, *, bias=None, t5_table=None, t5_num_buckets=32,
                                      t5_max_distance=128, t5_bidirectional=True,
                                      alibi_slopes=None, rel_table=None) -> int:
    lib = load_library()
    shape = make_shape(q, k)
    bd = make_bias(bias, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (q.shape[0], q.shape[2], q.shape[1], k.shape[1]), alibi_slopes, rel_table)
    return int(lib.sdpa_bwd_bias_grad_workspace_size(ctypes.byref(shape), ctypes.byref(bd)))


def sdpa_bwd_bias_grad(q, k, v, o, do, lse, *, causal=False, window_left=-1, window_right=-1,
                       bias=None, t5_table=None, t5_num_buckets=32, t5_max_distance=128,
                       t5_bidirectional=True, alibi_slopes=None, rel_table=None,
                       scale=None, dq=None, dk=None,
                       dv=None, dbias=None, workspace=None):
    """dQ, dK, dV and the bias gradient (see sdpa_bwd_bias_grad in include/sdpa.h).

    The bias gradient has the dense bias's shape and strides, the T5 table's
    [num_buckets, Hq] shape, or the ALiBi slopes' [Hq] shape.
    """
    lib = load_library()
    shape = make_shape(q, k)
    _same_layout(v, k, "v")
    _same_layout(o, q, "o")
    _same_layout(do, q, "do")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _same_layout(dq, q, "dq")
    _same_layout(dk, k, "dk")
    _same_layout(dv, k, "dv")
    bd = make_bias(bias, t5_table, t5_num_buckets, t5_max_distance, t5_bidirectional,
                   (q.shape[0], q.shape[2], q.shape[1], k.shape[1]), alibi_slopes, rel_table)
    ref = next((x for x in (bias, t5_table, alibi_slopes, rel_table) if x is not None), None)
    if ref is None:
        raise ValueError("a bias gradient needs a dense bias, a T5 table or ALiBi slopes")
    if dbias is None:
        dbias = torch.empty_strided(ref.shape, ref.stride(), device=q.device,
                                    dtype=torch.float32)
    if (dbias.shape != ref.shape or dbias.stride() != ref.stride()
            or dbias.dtype != torch.float32):
        raise ValueError("dbias must be float32 with the shape and strides of the bias")
    need = int(lib.sdpa_bwd_bias_grad_workspace_size(ctypes.byref(shape), ctypes.byref(bd)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), device=q.device, dtype=torch.uint8)
    sc = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    m = make_mask(causal, window_left, window_right)
    st = lib.sdpa_bwd_bias_grad(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                _ptr(do), _ptr(lse), ctypes.byref(bd), ctypes.byref(m), sc,
                                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias), 1, _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(q))
    _check(st, "sdpa_bwd_bias_grad")
    return dq, dk, dv, dbias


def sdpa_t5_bucket(rel: torch.Tensor, num_buckets=32, max_distance=128, bidirectional=True):
    """Bucket ids of int32 signed distances (device tensor) by the kernels' own function."""
    lib = load_library()
    if rel.dtype != torch.int32 or not rel.is_cuda or not rel.is_contiguous():
        raise ValueError("rel must be a contiguous int32 CUDA tensor")
    out = torch.empty_like(rel)
    st = lib.sdpa_t5_bucket(_ptr(rel), _ptr(out), rel.numel(), int(num_buckets),
                            int(max_distance), 1 if bidirectional else 0, _stream(rel))
    _check(st, "sdpa_t5_bucket")
    return out


def sdpa_exp2_fma(x: torch.Tensor) -> torch.Tensor:
    """2^x by the kernels' FMA-pipe exponential (float32 CUDA tensor)."""
    lib = load_library()
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    y = torch.empty_like(x)
    _check(lib.sdpa_exp2_fma(_ptr(x), _ptr(y), x.numel(), _stream(x)), "sdpa_exp2_fma")
    return y


def sdpa_read_device_status() -> int:
    """Synchronise the current stream; return (and clear) the device status code."""
    return int(load_library().sdpa_read_device_status(_stream()))


def sdpa_set_wait_limit_ns(ns: int):
    load_library().sdpa_set_wait_limit_ns(int(ns))


def sdpa_debug_wait_timeout():
    _check(load_library().sdpa_debug_wait_timeout(_stream()), "sdpa_debug_wait_timeout")


def _fire_desc(w1, b1, w2, b2, c, threshold):
    for t, n in ((w1, "w1"), (b1, "b1"), (w2, "w2"), (b2, "b2")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"FIRE {n} must be a contiguous float32 CUDA tensor")
    W = w1.shape[0]
    if w1.dim() != 1 or b1.shape != (W,) or w2.dim() != 2 or w2.shape[1] != W or \
            b2.shape != (w2.shape[0],):
        raise ValueError("FIRE weights must be w1 [W], b1 [W], w2 [H, W], b2 [H]")
    return Fire(w1.data_ptr(), b1.data_ptr(), w2.data_ptr(), b2.data_ptr(), float(c),
                float(threshold), int(W), int(w2.shape[0]))


def sdpa_fire_table(w1, b1, w2, b2, c, threshold, Lq, Lk, out=None):
    """FIRE bias as a relative-position table [Lq + Lk - 1, H] (see sdpa_fire_table in
    include/sdpa.h); pass it as ``rel_table``."""
    f = _fire_desc(w1, b1, w2, b2, c, threshold)
    if out is None:
        out = torch.empty(Lq + Lk - 1, f.heads, device=w1.device, dtype=torch.float32)
    _check(load_library().sdpa_fire_table(ctypes.byref(f), int(Lq), int(Lk), _ptr(out),
                                          _stream(w1)), "sdpa_fire_table")
    return out


def sdpa_fire_backward(w1, b1, w2, b2, c, threshold, Lq, Lk, d_table):
    """Gradients of FIRE's parameters from its table's gradient: a dict with w1, b1, w2,
    b2 and c_threshold (d/dc, d/dthreshold)."""
    lib = load_library()
    f = _fire_desc(w1, b1, w2, b2, c, threshold)
    if d_table.dtype != torch.float32 or not d_table.is_contiguous() or \
            tuple(d_table.shape) != (Lq + Lk - 1, f.heads):
        raise ValueError("d_table must be contiguous float32 [Lq + Lk - 1, H]")
    need = int(lib.sdpa_fire_backward_workspace_size(ctypes.byref(f), int(Lq), int(Lk)))
    ws = torch.empty(max(need, 256), device=w1.device, dtype=torch.uint8)
    g = {n: torch.empty_like(t) for n, t in (("w1", w1), ("b1", b1), ("w2", w2), ("b2", b2))}
    g["c_threshold"] = torch.empty(2, device=w1.device, dtype=torch.float32)
    _check(lib.sdpa_fire_backward(ctypes.byref(f), int(Lq), int(Lk), _ptr(d_table), _ptr(g["w1"]),
                                  _ptr(g["b1"]), _ptr(g["w2"]), _ptr(g["b2"]),
                                  _ptr(g["c_threshold"]), _ptr(ws), ws.numel(), _stream(w1)),
           "sdpa_fire_backward")
    return g


def sdpa_status_string(status: int) -> str:
    return load_library().sdpa_status_string(int(status)).decode()


# ------------------------------------------------------------------- serving
# These calls sit in a generation loop whose kernels take a few microseconds, so
# each reads what it needs of a tensor once and passes plain integers.
_BF16, _E4M3, _F32, _F64 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64
_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8


def _device_stream(ref: torch.Tensor, *tensors):
    """The raw current stream of ref's GPU, which must be the current one and every tensor's."""
    dev = ref.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{dev}, which is not the current CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors are on {t.device} and on cuda:{dev}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _bad(name: str, what: str):
    raise ValueError(f"{name} must be {what}")


def _rows(t: torch.Tensor, name: str, dims: int):
    """Shape and strides of a bf16 tensor of head rows; the stride of a dimension that is never
    stepped along is given as 8."""
    st = t.stride()
    sh = t.shape
    if t.dtype != _BF16 or len(sh) != dims or (st[-1] != 1 and sh[-1] != 1):
        _bad(name, f"bf16 with {dims} dimensions and a contiguous head_dim")
    if 1 in sh:
        st = tuple(8 if n == 1 else x for n, x in zip(sh, st))
    return sh, st


def _alike(t: torch.Tensor, name: str, sh, st):
    if t.dtype != _BF16 or t.shape != sh or (t.stride() != st and _rows(t, name, len(sh))[1] != st):
        _bad(name, "bf16 with the shape and strides of its partner")


def sdpa_rope_frequencies(rot, base=10000.0, *, scaling="none", factor=1.0, original_length=0,
                          beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freqs float64 [rot / 2] on ``device``, amplitude) for sdpa_rope: radians per position,
    unscaled or scaled for longer contexts ("linear", "ntk", "yarn"; see include/sdpa.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(int(rot) // 2, 1))()
    amplitude = ctypes.c_float()
    _check(load_library().sdpa_rope_frequencies(int(rot), float(base), ROPE_SCALINGS[scaling],
                                                float(factor), int(original_length),
                                                float(beta_fast), float(beta_slow), out,
                                                ctypes.byref(amplitude)), "sdpa_rope_frequencies")
    return torch.tensor(list(out), dtype=_F64, device=device), amplitude.value


def sdpa_rope(q, k, freqs, positions=None, *, offset=0, interleaved=False, inverse=False,
              amplitude=1.0, out_q=None, out_k=None):
    """q and k turned by their positions (see sdpa_rope in include/sdpa.h): (out_q, out_k).

    q [B, L, Hq, d] and k [B, L, Hkv, d], or packed [T, Hq, d] and [T, Hkv, d]; k may be None.
    ``positions`` int32 [B, L] (or [T]); without it row l has position ``offset`` + l.
    ``inverse`` turns back: the gradient.  out_q=q, out_k=k works in place.
    """
    lib = load_library()
    dims = q.dim()
    if dims != 3 and dims != 4:
        _bad("q", "[B, L, Hq, d] or [T, Hq, d]")
    stream = _device_stream(q, k, freqs, positions, out_q, out_k)
    qs, qst = _rows(q, "q", dims)
    d, Hq, L = qs[-1], qs[-2], qs[-3]
    B, zero = (qs[0], ()) if dims == 4 else (1, (8,))
    if freqs.dtype != _F64 or freqs.dim() != 1 or not freqs.is_contiguous():
        _bad("freqs", "a contiguous float64 vector")
    pos, pos_b = None, L
    if positions is not None:
        if positions.dtype != _I32 or positions.shape != qs[:-2]:
            _bad("positions", "int32 [B, L] (packed: [T])")
        pst = positions.stride()
        if L > 1 and pst[-1] != 1:
            _bad("positions", "contiguous along the sequence")
        pos, pos_b = positions.data_ptr(), (pst[0] if B > 1 else L)
    if out_q is None:
        out_q = torch.empty(qs, device=q.device, dtype=_BF16)
    ost = _rows(out_q, "out_q", dims)[1]
    if out_q.shape != qs:
        _bad("out_q", f"{tuple(qs)}")
    if k is not None:
        ks, kst = _rows(k, "k", dims)
        if ks[:-2] != qs[:-2] or ks[-1] != d:
            raise ValueError(f"k shape {tuple(ks)} does not match q {tuple(qs)}")
        if out_k is None:
            out_k = torch.empty(ks, device=q.device, dtype=_BF16)
        okst = _rows(out_k, "out_k", dims)[1]
        if out_k.shape != ks:
            _bad("out_k", f"{tuple(ks)}")
        Hkv, kp, okp = ks[-2], k.data_ptr(), out_k.data_ptr()
    else:
        kst = okst = (0,) * dims
        Hkv, kp, okp, out_k = 0, None, None, None
    if B * L == 0:
        return out_q, out_k
    r = RopeDesc(B, L, Hq, Hkv, d, *zero, *qst[:-1], *zero, *kst[:-1], *zero, *ost[:-1], *zero,
                 *okst[:-1], pos, pos_b, offset, freqs.data_ptr(), 2 * freqs.shape[0], interleaved,
                 inverse, amplitude)
    st = lib.sdpa_rope(ctypes.byref(r), q.data_ptr(), kp, out_q.data_ptr(), okp, stream)
    if st:
        raise SdpaError(st, "sdpa_rope")
    return out_q, out_k


def make_cache(k_cache, v_cache, k_scale=None, v_scale=None) -> KvCache:
    """Descriptor of a paged cache [num_pages, Hkv, page_size, d]: bf16, or float8_e4m3fn with
    uint8 scale exponents [num_pages, Hkv, page_size]."""
    dt, sh, st = k_cache.dtype, k_cache.shape, k_cache.stride()
    e4m3 = dt == _E4M3
    if not e4m3 and dt != _BF16:
        raise ValueError("a cache is bf16 or float8_e4m3fn")
    if (len(sh) != 4 or v_cache.shape != sh or v_cache.dtype != dt or v_cache.stride() != st
            or st[3] != 1):
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d] alike in "
                         "type, shape and strides, with a contiguous head_dim")
    P, H, page, d = sh
    sp = sh_ = 0
    kp = vp = None
    if e4m3:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        ss = k_scale.stride()
        if (k_scale.dtype != _U8 or k_scale.shape != sh[:3] or ss[2] != 1 or v_scale.dtype != _U8
                or v_scale.shape != sh[:3] or v_scale.stride() != ss):
            raise ValueError("k_scale and v_scale must be uint8 [num_pages, Hkv, page_size] alike "
                             "in strides, with contiguous rows")
        sp, sh_ = (ss[0] if P > 1 else 16), (ss[1] if H > 1 else 16)
        kp, vp = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bf16 cache has no scales")
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), kp, vp, 1 if e4m3 else 0, P, page, H, d,
                   st[0] if P > 1 else 16, st[1] if H > 1 else 16, st[2] if page > 1 else 16, sp,
                   sh_)


def _table(page_table: torch.Tensor, B: int):
    sh, st = page_table.shape, page_table.stride()
    if page_table.dtype != _I32 or len(sh) != 2 or sh[0] != B or (sh[1] > 1 and st[1] != 1):
        _bad("page_table", "int32 [B, pages] with contiguous rows")
    return sh[1], (st[0] if B > 1 else sh[1])


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _bad(name, f"contiguous {str(dtype)[6:]} {list(shape)}")
    return t.data_ptr()


def sdpa_cache_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Rows k, v [T, Hkv, d] into the cache at slots int64 [T] (page * page_size + row;
    negative: skipped), quantised if the cache is e4m3 (see sdpa_cache_append)."""
    lib = load_library()
    stream = _device_stream(k_cache, v_cache, k_scale, v_scale, k, v, slots)
    c = make_cache(k_cache, v_cache, k_scale, v_scale)
    sh, st = _rows(k, "k", 3)
    _alike(v, "v", sh, st)
    T, H, d = sh
    if H != c.Hkv or d != c.d:
        raise ValueError(f"k {tuple(sh)} does not fit the cache's heads")
    sp = _vector(slots, "slots", _I64, (T,))
    r = lib.sdpa_cache_append(ctypes.byref(c), k.data_ptr(), v.data_ptr(), T, st[0], st[1], sp,
                              stream)
    if r:
        raise SdpaError(r, "sdpa_cache_append")


def sdpa_cache_gather(k_cache, v_cache, page_table, cu_seqlens, total, k_scale=None, v_scale=None,
                      k=None, v=None):
    """The cached sequences as packed bf16 (k, v) [total, Hkv, d], sequence b's first
    cu_seqlens[b + 1] - cu_seqlens[b] positions at its rows (see sdpa_cache_gather)."""
    lib = load_library()
    stream = _device_stream(k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, k, v)
    c = make_cache(k_cache, v_cache, k_scale, v_scale)
    B = cu_seqlens.numel() - 1
    cu = _vector(cu_seqlens, "cu_seqlens", _I32, (B + 1,))
    width, table_b = _table(page_table, B)
    shape = (int(total), c.Hkv, c.d)
    if k is None:
        k = torch.empty(shape, device=k_cache.device, dtype=_BF16)
    if v is None:
        v = torch.empty_like(k)
    sh, st = _rows(k, "k", 3)
    if sh != shape:
        _bad("k", f"{list(shape)}")
    _alike(v, "v", sh, st)
    r = lib.sdpa_cache_gather(ctypes.byref(c), B, page_table.data_ptr(), width, table_b, cu,
                              shape[0], k.data_ptr(), v.data_ptr(), st[0], st[1], stream)
    if r:
        raise SdpaError(r, "sdpa_cache_gather")
    return k, v


def sdpa_tree_fwd(q, k_cache, v_cache, page_table, ctx_lens, cu_nodes, max_nodes, *,
                  k_scale=None, v_scale=None, tree_mask=None, window_left=-1, t5_table=None,
                  t5_num_buckets=32, t5_max_distance=128, t5_bidirectional=True,
                  alibi_slopes=None, scale=None, out=None, lse=None, workspace=None):
    """O [T, Hq, d], LSE [Hq, T]: each sequence's nodes over its cached context and over the
    nodes that ``tree_mask`` (int64 [T], bit j: sees node j; None: a chain) shows them.  One node
    per sequence is plain decoding.  The nodes' own keys are in the cache already, at positions
    ctx_lens[b] and on (see sdpa_tree_fwd in include/sdpa.h)."""
    lib = load_library()
    stream = _device_stream(k_cache, v_cache, k_scale, v_scale, q, page_table, ctx_lens, cu_nodes,
                            tree_mask, t5_table, alibi_slopes, out, lse, workspace)
    c = make_cache(k_cache, v_cache, k_scale, v_scale)
    sh, qst = _rows(q, "q", 3)
    T, Hq, d = sh
    if d != c.d:
        raise ValueError("q and the cache differ in head_dim")
    B = ctx_lens.numel()
    ctx = _vector(ctx_lens, "ctx_lens", _I32, (B,))
    cu = _vector(cu_nodes, "cu_nodes", _I32, (B + 1,))
    mask = None if tree_mask is None else _vector(tree_mask, "tree_mask", _I64, (T,))
    width, table_b = _table(page_table, B)
    if out is None:
        out = torch.empty(sh, device=q.device, dtype=_BF16)
    osh, ost = _rows(out, "out", 3)
    if osh != sh:
        _bad("out", "of q's shape")
    if lse is None:
        lse = torch.empty(Hq, T, device=q.device, dtype=_F32)
    lp = _vector(lse, "lse", _F32, (Hq, T))
    t = Tree(B, T, max_nodes, Hq, qst[0], qst[1], ost[0], ost[1], cu, ctx, page_table.data_ptr(),
             width, table_b, mask, window_left)
    bias = None
    if t5_table is not None or alibi_slopes is not None:
        bias = ctypes.byref(make_bias(None, t5_table, t5_num_buckets, t5_max_distance,
                                      t5_bidirectional, (B, Hq, 0, 0), alibi_slopes))
    tp, cp = ctypes.byref(t), ctypes.byref(c)
    if workspace is None:
        workspace = torch.empty(lib.sdpa_tree_fwd_workspace_size(tp, cp), device=q.device,
                                dtype=_U8)
    r = lib.sdpa_tree_fwd(tp, cp, q.data_ptr(), bias, d ** -0.5 if scale is None else scale,
                          out.data_ptr(), lp, workspace.data_ptr(), workspace.nbytes, stream)
    if r:
        raise SdpaError(r, "sdpa_tree_fwd")
    return out, lse


def sdpa_tree_fwd_workspace_size(q, k_cache, v_cache, page_table, ctx_lens, cu_nodes, max_nodes, *,
                                 k_scale=None, v_scale=None) -> int:
    """Bytes of the workspace of sdpa_tree_fwd for these tensors (0: they do not fit together)."""
    c = make_cache(k_cache, v_cache, k_scale, v_scale)
    width, table_b = _table(page_table, ctx_lens.numel())
    sh, st = _rows(q, "q", 3)
    t = Tree(ctx_lens.numel(), sh[0], int(max_nodes), sh[1], st[0], st[1], st[0], st[1],
             cu_nodes.data_ptr(), ctx_lens.data_ptr(), page_table.data_ptr(), width, table_b, None,
             -1)
    return int(load_library().sdpa_tree_fwd_workspace_size(ctypes.byref(t), ctypes.byref(c)))


def sdpa_spec_verify(target, draft, tokens, parents, u_accept, u_sample):
    """(path int32 [B, N], accepted int32 [B], next_token int32 [B]) of drafted trees, by
    rejection sampling with the given uniform numbers (see sdpa_spec_verify in include/sdpa.h).

    target, draft float32 [B, N, V]: the distributions after each node (draft may be None when
    N = 1); tokens int32 [B, N]; parents int32 [B, N] or None (a chain); u_accept float32 [B, N];
    u_sample float32 [B].
    """
    lib = load_library()
    stream = _device_stream(target, draft, tokens, parents, u_accept, u_sample)
    sh, tst = target.shape, target.stride()
    if target.dtype != _F32 or len(sh) != 3 or (tst[2] != 1 and sh[2] != 1):
        _bad("target", "float32 [B, N, V] with a contiguous vocabulary")
    B, N, V = sh
    dp = xp = pp = up = None
    dst = (0, 0)
    if draft is not None:
        dst = draft.stride()
        if draft.dtype != _F32 or draft.shape != sh or (dst[2] != 1 and V != 1):
            _bad("draft", "float32 [B, N, V] with a contiguous vocabulary")
        dp = draft.data_ptr()
    if N > 1:
        if draft is None:
            raise ValueError("draft distributions are needed when there are drafted nodes")
        xp = _vector(tokens, "tokens", _I32, (B, N))
        up = _vector(u_accept, "u_accept", _F32, (B, N))
        if parents is not None:
            pp = _vector(parents, "parents", _I32, (B, N))
    us = _vector(u_sample, "u_sample", _F32, (B,))
    dev = target.device
    path = torch.empty(B, N, device=dev, dtype=_I32)
    accepted = torch.empty(B, device=dev, dtype=_I32)
    token = torch.empty(B, device=dev, dtype=_I32)
    s = Verify(B, N, V, tst[0], tst[1], dst[0], dst[1], target.data_ptr(), dp, xp, pp, up, us)
    r = lib.sdpa_spec_verify(ctypes.byref(s), path.data_ptr(), accepted.data_ptr(),
                             token.data_ptr(), stream)
    if r:
        raise SdpaError(r, "sdpa_spec_verify")
    return path, accepted, token
