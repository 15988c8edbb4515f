"""Refusals of the serving entry points, on the host before any work is queued
(no GPU needed), and the host arithmetic of the rotary frequencies."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import serve_oracle as so
from scaled_dot_product_bwd_b200 import binding, serve
from scaled_dot_product_bwd_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    build()
    return serve.load_serve_library()


def _fields(cls, base, kw):
    base.update(kw)
    return cls(*[base[n] for n, _ in cls._fields_])


def _rope(**kw):
    base = dict(B=2, L=10, Hq=4, Hkv=2, d=64, positions=0x10000, pos_b=10, offset=0, freqs=0x10000,
                rot=64, interleaved=0, inverse=0, amplitude=1.0)
    for t, h in (("q", 4), ("k", 2), ("qo", 4), ("ko", 2)):
        base.update({f"{t}_b": 10 * h * 64, f"{t}_l": h * 64, f"{t}_h": 64})
    return _fields(serve.RopeDesc, base, kw)


def _cache(**kw):
    base = dict(k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000, format=1, num_pages=10,
                page_size=64, Hkv=2, d=64, stride_page=2 * 64 * 64, stride_head=64 * 64,
                stride_row=64, scale_stride_page=128, scale_stride_head=64)
    return _fields(serve.KvCache, base, kw)


def _tree(**kw):
    base = dict(B=2, T=8, max_nodes=4, Hq=4, q_t=256, q_h=64, o_t=256, o_h=64, cu_nodes=0x10000,
                ctx_lens=0x10000, page_table=0x10000, table_width=5, table_b=5, tree_mask=0x10000,
                window_left=-1)
    return _fields(serve.Tree, base, kw)


def _verify(**kw):
    base = dict(B=2, N=4, V=100, target_b=400, target_n=100, draft_b=400, draft_n=100,
                target=0x10000, draft=0x10000, tokens=0x10000, parents=0x10000, u_accept=0x10000,
                u_sample=0x10000)
    return _fields(serve.Verify, base, kw)


def test_library_exports_what_the_header_declares(lib):
    text = open(os.path.join(ROOT, "include", "sdpa_serve.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sdpa_[a-z0-9_]+)\s*\(", text))
    assert names == set(serve.SERVE_EXPORTED)
    for n in names:
        assert hasattr(lib, n), n


def test_missing_libraries_fail_loudly(tmp_path, monkeypatch):
    with pytest.raises(RuntimeError):
        serve.load_serve_library(str(tmp_path / "missing.so"))
    monkeypatch.setattr(serve, "_bind", None)
    monkeypatch.setattr(serve, "BIND_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError):
        serve.sdpa_spec_verify(None, None, None, None, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), 2), (dict(B=0), 1), (dict(L=0), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1),
    (dict(rot=0), 1), (dict(rot=66), 1), (dict(rot=33), 1), (dict(q_l=4), 1), (dict(ko_h=0), 1),
    (dict(freqs=0), 1), (dict(freqs=0x10004), 1), (dict(positions=0x10002), 1), (dict(pos_b=9), 1),
    (dict(amplitude=float("nan")), 1), (dict(L=1 << 30, B=2, pos_b=1 << 30), 2),
])
def test_rope_refuses(lib, kw, code):
    r = _rope(**kw)
    assert lib.sdpa_rope(ctypes.byref(r), FAKE, FAKE, FAKE, FAKE, None) == code


def test_rope_refuses_pointers(lib):
    r = _rope()
    odd = ctypes.c_void_p(0x10008)
    assert lib.sdpa_rope(None, FAKE, FAKE, FAKE, FAKE, None) == 1
    for i in range(4):
        for bad in (NULL, odd):
            args = [FAKE] * 4
            args[i] = bad
            assert lib.sdpa_rope(ctypes.byref(r), *args, None) == 1


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, original_length=4096),
                                dict(scaling="yarn", factor=2.0, original_length=7, beta_fast=4.0)])
@pytest.mark.parametrize("rot", [4, 32, 58, 128])
def test_rope_frequencies(lib, rot, kw):
    f, amp = serve.sdpa_rope_frequencies(rot, 10000.0, device="cpu", **kw)
    ref, ref_amp = so.rope_frequencies(rot, 10000.0, **kw)
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), ref, rtol=1e-13, atol=0)
    assert amp == pytest.approx(ref_amp, rel=1e-7)


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(base=1.0), dict(base=float("inf")),
                                dict(scaling="linear", factor=0.5), dict(rot=2, scaling="ntk", factor=2.0),
                                dict(scaling="yarn", factor=2.0),
                                dict(scaling="yarn", factor=2.0, original_length=9, beta_slow=0.0),
                                dict(scaling="yarn", factor=2.0, original_length=9, beta_fast=1.0)])
def test_rope_frequencies_refuse(lib, kw):
    kw = dict(kw)
    with pytest.raises(binding.SdpaError) as e:
        serve.sdpa_rope_frequencies(kw.pop("rot", 64), kw.pop("base", 10000.0), device="cpu", **kw)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        serve.sdpa_rope_frequencies(64, scaling="other", device="cpu")


BAD_CACHES = [
    (dict(k=0), 1), (dict(v=0x10008), 1), (dict(format=2), 1), (dict(num_pages=0), 1), (dict(d=32), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(Hkv=0), 1),
    (dict(stride_row=24), 1), (dict(stride_head=0), 1), (dict(k_scale=0), 1), (dict(v_scale=0x10008), 1),
    (dict(scale_stride_head=8), 1), (dict(scale_stride_page=0), 1), (dict(num_pages=1 << 31), 2),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(lib, kw, code):
    c = _cache(**kw)
    t = _tree()
    assert lib.sdpa_cache_append(ctypes.byref(c), FAKE, FAKE, 4, 128, 64, FAKE, None) == code
    assert lib.sdpa_cache_gather(ctypes.byref(c), 2, FAKE, 5, 5, FAKE, 9, FAKE, FAKE, 128, 64, None) == code
    assert lib.sdpa_tree_fwd(ctypes.byref(t), ctypes.byref(c), FAKE, None, 0.1, FAKE, FAKE, FAKE, 1 << 30, None) == code
    assert lib.sdpa_tree_fwd_workspace_size(ctypes.byref(t), ctypes.byref(c)) == 0


def test_append_and_gather_refuse(lib):
    c = _cache()

    def append(T=4, kv_t=128, kv_h=64, k=FAKE, v=FAKE, slots=FAKE):
        return lib.sdpa_cache_append(ctypes.byref(c), k, v, T, kv_t, kv_h, slots, None)

    assert lib.sdpa_cache_append(None, FAKE, FAKE, 4, 128, 64, FAKE, None) == 1
    assert append(T=-1) == append(kv_t=4) == append(kv_h=0) == append(k=NULL) == 1
    assert append(v=ctypes.c_void_p(0x10008)) == append(slots=NULL) == append(slots=ctypes.c_void_p(0x10004)) == 1
    assert append(T=0, slots=NULL) == 0                     # nothing to do
    assert append(T=1 << 31) == 2

    def gather(B=2, table=FAKE, width=5, table_b=5, cu=FAKE, total=9, k=FAKE, kv_t=128):
        return lib.sdpa_cache_gather(ctypes.byref(c), B, table, width, table_b, cu, total, k, FAKE, kv_t, 64, None)

    assert gather(B=0) == gather(table=NULL) == gather(width=0) == gather(table_b=4) == gather(cu=NULL) == 1
    assert gather(total=-1) == gather(k=NULL) == gather(kv_t=12) == 1
    assert gather(B=65536) == gather(total=1 << 30) == 2
    assert gather(total=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(max_nodes=0), 1), (dict(max_nodes=65), 2), (dict(Hq=3), 1),
    (dict(B=65536), 2), (dict(T=1 << 30), 2), (dict(cu_nodes=0), 1), (dict(ctx_lens=0x10002), 1),
    (dict(page_table=0), 1), (dict(table_width=0), 1), (dict(table_b=4), 1), (dict(tree_mask=0x10004), 1),
    (dict(q_t=12), 1), (dict(o_h=0), 1), (dict(table_width=1 << 29, table_b=1 << 29), 2),
])
def test_tree_refuses(lib, kw, code):
    c, t = _cache(), _tree(**kw)
    assert lib.sdpa_tree_fwd(ctypes.byref(t), ctypes.byref(c), FAKE, None, 0.1, FAKE, FAKE, FAKE, 1 << 30, None) == code
    assert lib.sdpa_tree_fwd_workspace_size(ctypes.byref(t), ctypes.byref(c)) == 0


def test_tree_refuses_bias_scale_workspace(lib):
    c, t = _cache(), _tree()
    need = lib.sdpa_tree_fwd_workspace_size(ctypes.byref(t), ctypes.byref(c))
    assert need > 0 and need % 256 == 0

    def call(bias=None, scale=0.1, ws=FAKE, n=need, q=FAKE, o=FAKE, lse=FAKE):
        return lib.sdpa_tree_fwd(ctypes.byref(t), ctypes.byref(c), q,
                                 ctypes.byref(binding.BiasDesc(*bias)) if bias else None, scale, o, lse, ws, n, None)

    assert call(bias=(1, 0x10000, 0, 0, 64, 0, 0, 0)) == 2       # dense
    assert call(bias=(4, 0x10000, 0, 0, 0, 0, 0, 0)) == 2        # relative table
    assert call(bias=(9, 0x10000, 0, 0, 0, 0, 0, 0)) == 1
    assert call(bias=(3, 0, 0, 0, 0, 0, 0, 0)) == 1              # ALiBi without slopes
    assert call(bias=(2, 0, 0, 0, 0, 32, 128, 0)) == 1           # T5 without a table
    assert call(bias=(2, 0x10000, 0, 0, 0, 31, 128, 1)) == 1
    assert call(scale=float("inf")) == 1
    assert call(ws=NULL) == call(ws=ctypes.c_void_p(0x10010)) == call(n=need - 1) == 3
    assert call(q=NULL) == call(o=ctypes.c_void_p(0x10008)) == call(lse=NULL) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(V=0), 1), (dict(N=65), 2), (dict(V=1 << 31), 2),
    (dict(target=0), 1), (dict(draft=0), 1), (dict(tokens=0), 1), (dict(u_accept=0), 1),
    (dict(u_sample=0), 1), (dict(parents=0x10002), 1), (dict(target_n=-1), 1),
])
def test_verify_refuses(lib, kw, code):
    s = _verify(**kw)
    assert lib.sdpa_spec_verify(ctypes.byref(s), FAKE, FAKE, FAKE, None) == code
    ok = _verify()
    assert lib.sdpa_spec_verify(None, FAKE, FAKE, FAKE, None) == 1
    for i in range(3):
        args = [FAKE] * 3
        args[i] = NULL
        assert lib.sdpa_spec_verify(ctypes.byref(ok), *args, None) == 1


def test_binding_refuses_host_tensors():
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: serve.sdpa_rope(q, k, torch.zeros(32, dtype=torch.float64)),
                 lambda: serve.sdpa_cache_append(k, k, torch.zeros(3, dtype=torch.int64), cache, cache),
                 lambda: serve.sdpa_cache_gather(cache, cache, i32[:1, None], i32, 3),
                 lambda: serve.sdpa_tree_fwd(q, cache, cache, i32[:1, None], i32[:1], i32, 4),
                 lambda: serve.sdpa_spec_verify(torch.zeros(1, 1, 9), None, None, None, None, torch.zeros(1))):
        with pytest.raises(ValueError):
            call()


def test_verify_refuses_a_vocabulary_whose_indices_could_wrap(lib):
    for v in (1 << 30, (1 << 31) - 1):
        s = _verify(V=v, target_n=v, target_b=4 * v, draft_n=v, draft_b=4 * v)
        assert lib.sdpa_spec_verify(ctypes.byref(s), FAKE, FAKE, FAKE, None) == 2
