"""GPU tests of the serving operators against their float64 definitions.

Tolerances (half a step of bf16 is 2^-8 of the value, of fp16 2^-11):
  rope   the sines and cosines and two products in float32 (2^-20 of the
         magnitudes covers them), then one rounding to bf16.
  cache  exact: codes, scales and values are compared bit for bit.
  tree   O: one rounding to bf16 (2^-8 |O|).  Each weight enters the product
         with V rounded to bf16 (2^-8) over a bf16 cache, as two e4m3 parts
         (2^-4 each, 2^-8 together) over e4m3, so at most 2^-8 sum(w |v|);
         e4m3 parts also drop what is below 2^-21 of the largest weight (half
         a step of 2^-9, over 16 for the second part and 2^7 for the largest
         weight), at most that for each of the n keys' |v|.  A score's error e_s
         of float32 accumulation, at most (d + 8) steps of 2^-23 of sum |q k|
         scale, moves a weight by 2 e_s (numerator and denominator); over e4m3
         a query element is off by at most 2^-21 of its row's largest, which
         adds 2^-21 max |q| sum |k| scale to e_s.  2^-18 covers exp2 and the
         sums.  LSE: e_s, and 2^-20 for the rest.
"""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as so
from scaled_dot_product_bwd_b200 import (SdpaError, sdpa_cache_append, sdpa_cache_gather, sdpa_fwd,
                                         sdpa_fwd_varlen, sdpa_read_device_status, sdpa_rope,
                                         sdpa_rope_frequencies, sdpa_spec_verify, sdpa_tree_fwd,
                                         sdpa_tree_fwd_workspace_size)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- rotary
def _check_rope(got, x, pos, freqs, **kw):
    ref = so.rope(f64(x), pos, freqs, **kw)
    size = so.rope(np.abs(f64(x)), np.zeros(pos.shape), freqs) * 0
    half = len(freqs)
    one = np.arange(half) * 2 if kw.get("interleaved") else np.arange(half)
    two = one + 1 if kw.get("interleaved") else one + half
    pair = np.abs(f64(x))[..., one] + np.abs(f64(x))[..., two]
    size[..., one] = size[..., two] = pair * kw.get("amplitude", 1.0)
    err = np.abs(f64(got) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size).all(), err.max()
    rest = sorted(set(range(x.shape[-1])) - set(one) - set(two))
    assert torch.equal(got[..., rest], x[..., rest])


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (128, 32), (128, 122), (64, 58), (64, 2), (128, 16), (64, 40)])
def test_rope(d, rot, interleaved, inverse):
    g = torch.Generator().manual_seed(rot + d)
    freqs, amp = sdpa_rope_frequencies(rot, scaling="yarn", factor=4.0, original_length=2048)
    for B, L, hq, hkv in ((1, 1, 3, 1), (2, 37, 4, 2), (1, 1300, 2, 2)):
        q, k = randn(g, B, L, hq, d), randn(g, B, L, hkv, d)
        pos = torch.randint(-5, 2000000, (B, L), generator=g, dtype=torch.int32)
        oq, ok = sdpa_rope(q, k, freqs, pos.to(DEV), interleaved=interleaved, inverse=inverse, amplitude=amp)
        for got, x in ((oq, q), (ok, k)):
            _check_rope(got, x, pos.numpy(), f64(freqs), interleaved=interleaved, inverse=inverse, amplitude=amp)


@pytest.mark.parametrize("interleaved,rot", [(False, 64), (True, 60), (False, 60)])
def test_rope_layouts(interleaved, rot):
    """A fused QKV buffer's slices, in place, packed rows, q alone, default positions."""
    g = torch.Generator().manual_seed(3)
    freqs, _ = sdpa_rope_frequencies(rot)
    B, L, hq, hkv, d = 2, 21, 4, 2, 64
    qkv = randn(g, B, L, hq + 2 * hkv, d)
    q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:].clone()
    want = sdpa_rope(q, k, freqs, interleaved=interleaved, offset=7)
    pos = np.arange(7, 7 + L)[None].repeat(B, 0)
    _check_rope(want[0], q, pos, f64(freqs), interleaved=interleaved)
    alone, none = sdpa_rope(q, None, freqs, interleaved=interleaved, offset=7)
    assert none is None and torch.equal(alone, want[0])
    packed = sdpa_rope(q[0].contiguous(), k[0].contiguous(), freqs, interleaved=interleaved, offset=7)
    assert torch.equal(packed[0], want[0][0]) and torch.equal(packed[1], want[1][0])
    got = sdpa_rope(q, k, freqs, interleaved=interleaved, offset=7, out_q=q, out_k=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, hq + hkv:], v)
    wide = torch.arange(B * 2 * L, device=DEV, dtype=torch.int32).view(B, 2 * L)[:, :L]
    _check_rope(sdpa_rope(v, None, freqs, wide, interleaved=interleaved)[0], v, wide.cpu().numpy(), f64(freqs),
                interleaved=interleaved)


def test_rope_gradient_is_the_transpose():
    g = torch.Generator().manual_seed(4)
    freqs, amp = sdpa_rope_frequencies(48, scaling="linear", factor=3.0)
    x, dy = randn(g, 1, 50, 2, 64), randn(g, 1, 50, 2, 64)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)[None] * 1000
    y = f64(sdpa_rope(x, None, freqs, pos)[0])
    dx = f64(sdpa_rope(dy, None, freqs, pos, inverse=True)[0])
    a, b = (y * f64(dy)).sum(), (f64(x) * dx).sum()
    # both sides round N = 6400 products' factors to bf16, each off by at most 2^-8
    assert abs(a - b) <= 2.0 ** -8 * (np.abs(y * f64(dy)).sum() + np.abs(f64(x) * dx).sum())


def test_rope_refuses_mismatches():
    q, k = torch.zeros(1, 4, 2, 64, device=DEV, dtype=torch.bfloat16), torch.zeros(1, 5, 2, 64, device=DEV, dtype=torch.bfloat16)
    freqs, _ = sdpa_rope_frequencies(64)
    for call in (lambda: sdpa_rope(q, k, freqs), lambda: sdpa_rope(q.float(), None, freqs),
                 lambda: sdpa_rope(q, None, freqs.float()), lambda: sdpa_rope(q, None, freqs, torch.zeros(1, 4, device=DEV)),
                 lambda: sdpa_rope(q, None, freqs, out_q=k)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(SdpaError):
        sdpa_rope(q, None, sdpa_rope_frequencies(66)[0])


# -------------------------------------------------------------------- cache
def make_cache(pages, hkv, page, d, kv, fill=None):
    dtype = torch.bfloat16 if kv == "bf16" else torch.uint8
    mk = lambda: torch.full((pages, hkv, page, d), 0x7F if kv == "e4m3" else float("nan"), device=DEV, dtype=dtype)
    c = dict(k_cache=mk(), v_cache=mk(), k_scale=None, v_scale=None)
    if kv == "e4m3":
        c["k_cache"], c["v_cache"] = (c[n].view(torch.float8_e4m3fn) for n in ("k_cache", "v_cache"))
        c["k_scale"], c["v_scale"] = (torch.full((pages, hkv, page), 120, device=DEV, dtype=torch.uint8) for _ in range(2))
    return c


def rows_of(cache, name, flat):
    """Float64 rows [len(flat), Hkv, d] at flat positions page * page_size + row."""
    c = cache[name + "_cache"]
    page = c.shape[2]
    raw = (c if c.dtype == torch.bfloat16 else c.view(torch.uint8)).transpose(1, 2).flatten(0, 1)[flat]
    if c.dtype == torch.bfloat16:
        return f64(raw)
    e = cache[name + "_scale"].transpose(1, 2).flatten(0, 1)[flat].cpu().numpy().astype(float)
    return so.e4m3_decode(raw.cpu().numpy()) * 2.0 ** (e - 127)[..., None]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,hkv,d,page", [(1, 1, 64, 16), (37, 3, 128, 16), (300, 8, 128, 64), (513, 2, 64, 256)])
def test_append_and_gather(T, hkv, d, page, kv):
    g = torch.Generator().manual_seed(T)
    pages = T // page + 3
    cache = make_cache(pages, hkv, page, d, kv)
    before = {n: t.clone() for n, t in cache.items() if t is not None}
    k = randn(g, T, hkv, d) * torch.exp2(torch.randint(-20, 20, (T, hkv, 1), generator=g)).to(DEV).bfloat16()
    qkv = randn(g, T, 2 * hkv, d)
    v = torch.empty_strided(k.shape, k.stride(), device=DEV, dtype=k.dtype).copy_(qkv[:, hkv:])
    k[0, 0, :4] = torch.tensor([0.0, float("inf"), -float("inf"), float("nan")]).bfloat16().to(DEV)
    if T > 3:
        k[1], v[2] = 0.0, torch.tensor(2.0 ** -133).bfloat16().to(DEV)
        k[2, 0] = torch.finfo(torch.bfloat16).max
    flat = torch.randperm(pages * page, generator=g)[:T]
    flat[T // 2:T // 2 + 2] = -1 if T > 5 else flat[T // 2:T // 2 + 2]
    sdpa_cache_append(k, v, flat.to(DEV), **cache)
    kept = (flat >= 0).to(DEV)
    at = flat[flat >= 0].to(DEV)
    for name, x in (("k", k), ("v", v)):
        c = cache[name + "_cache"]
        rows = (c if kv == "bf16" else c.view(torch.uint8)).transpose(1, 2).flatten(0, 1)
        if kv == "bf16":
            assert torch.equal(rows[at].view(torch.int16), x[kept].view(torch.int16))
        else:
            codes, e = so.e4m3_rows(f64(x[kept]))
            got = rows[at].cpu().numpy()
            nan = np.isnan(so.e4m3_decode(codes))
            assert np.array_equal(got[~nan], codes[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
            assert np.array_equal(cache[name + "_scale"].transpose(1, 2).flatten(0, 1)[at].cpu().numpy(), e)
        untouched = torch.ones(pages * page, dtype=torch.bool, device=DEV)
        untouched[at] = False
        old = before[name + "_cache"]
        old = (old.view(torch.int16) if kv == "bf16" else old.view(torch.uint8)).transpose(1, 2).flatten(0, 1)
        new = (c.view(torch.int16) if kv == "bf16" else c.view(torch.uint8)).transpose(1, 2).flatten(0, 1)
        assert torch.equal(new[untouched], old[untouched])
    # read back through a page table, ragged, with rows behind the last sequence
    table = torch.randperm(pages, generator=g)[:pages // 2 * 2].view(2, -1).int().to(DEV)
    room = table.shape[1] * page
    lens = [room - 3, 0] if T == 1 else [min(5, room), room]
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=DEV)
    mark = torch.full((sum(lens) + 4, hkv, d), 7.0, device=DEV, dtype=torch.bfloat16)
    ko, vo = sdpa_cache_gather(page_table=table, cu_seqlens=cu, total=sum(lens) + 4, k=mark, v=mark.clone(), **cache)
    pos = torch.cat([table[b].long().repeat_interleave(page)[:n] * page + torch.arange(n, device=DEV) % page
                     for b, n in enumerate(lens)])
    for name, got in (("k", ko), ("v", vo)):
        ref = torch.from_numpy(rows_of(cache, name, pos)).bfloat16()
        same = (got[:len(pos)].cpu() == ref) | (torch.isnan(got[:len(pos)].cpu()) & torch.isnan(ref))
        assert same.all()
        assert (got[len(pos):] == 7).all()


def test_strided_and_long_cache():
    """Pages whose offsets pass 2^31 elements, and a cache that is a slice of a larger buffer."""
    g = torch.Generator().manual_seed(1)
    hkv, page, d = 8, 64, 128
    pages = 2 ** 31 // (hkv * page * d) + 40
    buf = torch.empty(pages, 2, hkv, page, d, device=DEV, dtype=torch.bfloat16)       # K and V of a page together
    cache = dict(k_cache=buf[:, 0], v_cache=buf[:, 1])
    n = 130
    table = torch.tensor([[pages - 1, 3, pages - 7, pages // 2]], device=DEV, dtype=torch.int32)
    slots = table[0].long().repeat_interleave(page)[:n] * page + torch.arange(n, device=DEV) % page
    k, v, q = randn(g, n, hkv, d), randn(g, n, hkv, d), randn(g, 2, 16, d)
    sdpa_cache_append(k, v, slots, **cache)
    ko, vo = sdpa_cache_gather(page_table=table, cu_seqlens=torch.tensor([0, n], device=DEV, dtype=torch.int32), total=n, **cache)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)
    o, lse = sdpa_tree_fwd(q, page_table=table, ctx_lens=i32(n - 2), cu_nodes=i32(0, 2), max_nodes=2, **cache)
    check_tree(o, lse, q, [(f64(k), f64(v), n - 2)], [0, 2], "bf16")


def test_bad_slots_and_pages_are_reported():
    g = torch.Generator().manual_seed(2)
    cache = make_cache(4, 2, 16, 64, "e4m3")
    k = randn(g, 3, 2, 64)
    old = cache["k_cache"].view(torch.uint8).clone()
    sdpa_cache_append(k, k, torch.tensor([64, 1 << 40, -5], device=DEV), **cache)
    assert sdpa_read_device_status() == 2
    assert torch.equal(cache["k_cache"].view(torch.uint8), old)
    cu = torch.tensor([0, 20], device=DEV, dtype=torch.int32)
    for bad in (4, -1):
        table = torch.tensor([[1, bad]], device=DEV, dtype=torch.int32)
        out = torch.full((20, 2, 64), 3.0, device=DEV, dtype=torch.bfloat16)
        sdpa_cache_gather(page_table=table, cu_seqlens=cu, total=20, k=out, v=out.clone(), **cache)
        assert sdpa_read_device_status() == 2 and (out[16:] == 3).all()
    table = torch.tensor([[1]], device=DEV, dtype=torch.int32)      # 20 positions, one page
    out = torch.full((20, 2, 64), 3.0, device=DEV, dtype=torch.bfloat16)
    sdpa_cache_gather(page_table=table, cu_seqlens=cu, total=20, k=out, v=out.clone(), **cache)
    assert sdpa_read_device_status() == 2 and (out[16:] == 3).all()


# --------------------------------------------------------------------- tree
def tree_tolerance(q, k, v, ro, spread, size, kv, scale=None):
    """The module docstring's bounds for O and LSE."""
    d = q.shape[-1]
    e_s = (d + 8) * 2.0 ** -23 * size
    if kv == "bf16":
        return 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * e_s[..., None] + 2.0 ** -18) * spread, e_s
    scale = d ** -0.5 if scale is None else abs(scale)
    e_s = e_s + 2.0 ** -21 * np.abs(q).max(-1) * np.abs(k).sum(-1).max() * scale
    lost = 2.0 ** -21 * len(v) * np.abs(v).max()
    return 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * e_s[..., None] + 2.0 ** -18) * spread + lost, e_s


def check_tree(o, lse, q, seqs, cu, kv, masks=None, **kw):
    """seqs: (k, v, ctx) per sequence in float64; every output against the definition."""
    for b, (k, v, ctx) in enumerate(seqs):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        ro, rl, spread, size = so.tree_attention(f64(q[lo:hi]), k, v, ctx, None if masks is None else masks[lo:hi], **kw)
        tol, e_s = tree_tolerance(f64(q[lo:hi]), k, v, ro, spread, size, kv, kw.get("scale"))
        err = np.abs(f64(o[lo:hi]) - ro)
        assert (err <= tol).all(), (b, float(err.max()), float((err / np.maximum(tol, 1e-30)).max()))
        gl = f64(lse[:, lo:hi]).T
        none = np.isneginf(rl)
        assert np.array_equal(none, np.isneginf(gl)), (b, gl, rl)
        with np.errstate(invalid="ignore"):
            el = np.where(none, 0, np.abs(gl - rl))
        assert (el <= e_s + 2.0 ** -20 * (1 + np.where(none, 0, np.abs(rl)))).all(), (b, float(el.max()))


def random_tree(n, g, chain=False):
    mask = []
    for i in range(n):
        parent = i - 1 if chain else int(torch.randint(max(0, i - 4), i, (1,), generator=g)) if i else -1
        mask.append((mask[parent] if i else 0) | (1 << i))
    return [m - (1 << 64) if m >> 63 else m for m in mask]


def tree_setup(lens, counts, hq, hkv, d, page, kv, seed=0, extra_rows=0, chain=False):
    """A filled cache (rows outside the sequences hold NaN), q, page table and masks."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-(a + b) // page) for a, b in zip(lens, counts)))
    pages = len(lens) * width + 2
    cache = make_cache(pages, hkv, page, d, kv)
    table = torch.randperm(pages, generator=g)[:len(lens) * width].view(len(lens), width)
    seqs, cu, masks = [], [0], []
    for b, (ctx, n) in enumerate(zip(lens, counts)):
        m = ctx + n
        flat = (table[b].repeat_interleave(page)[:m] * page + torch.arange(m) % page).to(DEV)
        if m:
            sdpa_cache_append(randn(g, m, hkv, d), randn(g, m, hkv, d) * 2, flat, **cache)
        seqs.append((rows_of(cache, "k", flat), rows_of(cache, "v", flat), ctx))
        cu.append(cu[-1] + n)
        masks += random_tree(n, g, chain)
    q = randn(g, cu[-1] + extra_rows, hq, d)
    i32 = lambda x: torch.tensor(x, device=DEV, dtype=torch.int32)
    mask = torch.tensor(masks + [0] * extra_rows, device=DEV, dtype=torch.int64)
    args = dict(page_table=table.int().to(DEV), ctx_lens=i32(lens), cu_nodes=i32(cu), max_nodes=max(1, max(counts)))
    return cache, q, args, mask, seqs, cu, masks


TREES = {
    "one_key": dict(lens=[0], counts=[1], hq=1, hkv=1, d=64, page=16),
    "decode_ragged": dict(lens=[1, 63, 64, 65, 1000, 0, 127], counts=[1] * 7, hq=8, hkv=2, d=128, page=16),
    "decode_long": dict(lens=[9000], counts=[1], hq=4, hkv=4, d=128, page=64),
    "decode_mqa_d64": dict(lens=[300, 17], counts=[1, 1], hq=32, hkv=1, d=64, page=32),
    "decode_g3": dict(lens=[130, 500], counts=[1, 1], hq=6, hkv=2, d=128, page=128),
    "tree_ragged": dict(lens=[100, 0, 777, 64], counts=[16, 5, 1, 33], hq=8, hkv=2, d=128, page=16),
    "tree_empty_sequences": dict(lens=[10, 5, 0, 70], counts=[0, 3, 0, 7], hq=4, hkv=4, d=64, page=64),
    "tree_64": dict(lens=[129, 40], counts=[64, 64], hq=4, hkv=2, d=64, page=256),
    "tree_64_mqa": dict(lens=[600], counts=[64], hq=8, hkv=1, d=128, page=32),
    "tree_many_heads": dict(lens=[250, 251], counts=[3, 2], hq=24, hkv=24, d=64, page=16),
}
EXTRAS = {"plain": dict(), "window": dict(window_left=50), "window_0": dict(window_left=0), "alibi": dict(alibi=True),
          "t5": dict(t5=False), "t5_bidir_window": dict(t5=True, window_left=200), "scale": dict(scale=-0.3)}


def bias_kw(extra, hq):
    kw = {n: v for n, v in extra.items() if n in ("window_left", "scale")}
    okw = dict(kw)
    if extra.get("alibi"):
        s = torch.tensor([2.0 ** (-8 * (h + 1) / hq) for h in range(hq)])
        kw["alibi_slopes"], okw["alibi_slopes"] = s.to(DEV), s.numpy()
    if "t5" in extra:
        t = torch.randn(32, hq, generator=torch.Generator().manual_seed(9))
        kw["t5_table"], okw["t5_table"] = t.to(DEV), t.numpy()
        kw["t5_bidirectional"] = okw["t5_bidirectional"] = extra["t5"]
    return kw, okw


@pytest.mark.parametrize("extra", list(EXTRAS))
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(TREES))
def test_tree(name, kv, extra):
    c = TREES[name]
    cache, q, args, mask, seqs, cu, masks = tree_setup(kv=kv, **c)
    kw, okw = bias_kw(EXTRAS[extra], c["hq"])
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache, **kw)
    check_tree(o, lse, q, seqs, cu, kv, masks, **okw)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_chain_default(kv):
    cache, q, args, mask, seqs, cu, masks = tree_setup([70, 3], [9, 64], 4, 2, 128, 32, kv, chain=True)
    a = sdpa_tree_fwd(q, **args, **cache)
    b = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_tree(*a, q, seqs, cu, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_masks_that_leave_nothing_and_nan_in_hidden_nodes(kv):
    """Arbitrary masks: nodes that see nothing, only a later node, or a subset; one node's key and
    value are NaN (and infinite): they reach exactly the nodes that see it."""
    for ctx in (0, 61):
        cache, q, args, mask, seqs, cu, _ = tree_setup([ctx], [6], 4, 2, 128, 16, kv, seed=5)
        words = [0, 0b100000, 0b000010, 0b001001, 0b110111, 0]
        bad = 3
        flat = int(args["page_table"][0, (ctx + bad) // 16]) * 16 + (ctx + bad) % 16
        wild = torch.tensor([float("nan"), float("inf")], device=DEV).repeat(64).bfloat16()
        if kv == "bf16":
            for n in ("k_cache", "v_cache"):
                cache[n].transpose(1, 2).flatten(0, 1)[flat]    # (a view only when dense)
                cache[n][flat // 16, :, flat % 16] = wild
        else:
            for n in ("k_cache", "v_cache"):
                cache[n].view(torch.uint8)[flat // 16, :, flat % 16] = 0x7F
        m = torch.tensor(words, device=DEV, dtype=torch.int64)
        o, lse = sdpa_tree_fwd(q, tree_mask=m, **args, **cache)
        k, v, _ = seqs[0]
        k, v = k.copy(), v.copy()
        k[ctx + bad] = v[ctx + bad] = 0                       # hidden from every node but 3
        ro, rl, spread, size = so.tree_attention(f64(q), k, v, ctx, words)
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[:, bad]).all()
        keep = [i for i in range(6) if i != bad]
        err = np.abs(f64(o)[keep] - ro[keep])
        tol, _ = tree_tolerance(f64(q), k, v, ro, spread, size, kv)
        assert (err <= tol[keep]).all()
        if ctx == 0:
            for i in (0, 5):
                assert (o[i] == 0).all() and torch.isneginf(lse[:, i]).all()


def test_tree_value_infinity_reaches_its_viewers_alone():
    cache, q, args, _, seqs, cu, _ = tree_setup([20], [3], 2, 2, 64, 16, "bf16", seed=6)
    flat = int(args["page_table"][0, 1]) * 16 + (21 - 16)     # node 1
    cache["v_cache"][flat // 16, :, flat % 16] = float("inf")
    m = torch.tensor([0b001, 0b011, 0b101], device=DEV, dtype=torch.int64)
    o, _ = sdpa_tree_fwd(q, tree_mask=m, **args, **cache)
    assert torch.isinf(o[1]).all() and (o[1] > 0).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()


def test_tree_bias_of_the_lowest_value():
    """T5 buckets at the type's lowest value and at -inf: the first orders below every other key but
    still counts where nothing else is left; the second hides its keys."""
    cache, q, args, mask, seqs, cu, masks = tree_setup([40], [1], 2, 2, 64, 16, "bf16", seed=7)
    low = torch.finfo(torch.float32).min
    table = torch.zeros(32, 2)
    table[:, 0] = low
    table[5:, 1] = -float("inf")
    o, lse = sdpa_tree_fwd(q, t5_table=table.to(DEV), t5_bidirectional=False, **args, **cache)
    k, v, ctx = seqs[0]
    mean = v[:, 0].mean(0)                                    # head 0: all weights equal
    assert (np.abs(f64(o)[0, 0] - mean) <= 2.0 ** -7 * np.abs(v[:, 0]).mean(0)).all()
    ro, *_ = so.tree_attention(f64(q), k[-5:], v[-5:], 4)     # head 1: the 5 nearest keys
    assert np.allclose(f64(o)[0, 1], ro[0, 1], atol=0.05)
    table[:, :] = -float("inf")
    o, lse = sdpa_tree_fwd(q, t5_table=table.to(DEV), t5_bidirectional=False, **args, **cache)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_rows_behind_the_last_sequence_and_strides(kv):
    cache, q, args, mask, seqs, cu, masks = tree_setup([90, 200], [4, 2], 4, 2, 64, 32, kv, extra_rows=5)
    T = q.shape[0]
    wide = torch.full((T, 3, 4, 64), 5.0, device=DEV, dtype=torch.bfloat16)
    wide[:, 1] = q
    out = torch.full((T, 4, 2, 64), 9.0, device=DEV, dtype=torch.bfloat16)[:, :, 1]
    lse = torch.full((4, T), 4.0, device=DEV)
    need = sdpa_tree_fwd_workspace_size(q, page_table=args["page_table"], ctx_lens=args["ctx_lens"],
                                        cu_nodes=args["cu_nodes"], max_nodes=4, **cache)
    ws = torch.full((need,), 0xFF, device=DEV, dtype=torch.uint8)
    o, l2 = sdpa_tree_fwd(wide[:, 1], tree_mask=mask, out=out, lse=lse, workspace=ws, **args, **cache)
    assert o is out and l2 is lse
    check_tree(o, lse, q, seqs, cu, kv, masks)
    assert (out[cu[-1]:] == 9).all() and (lse[:, cu[-1]:] == 4).all()


def test_tree_extreme_scales_and_queries():
    """e4m3 rows whose scales lie 2^60 apart, and queries near the ends of bf16's range."""
    g = torch.Generator().manual_seed(8)
    n, hq, d = 100, 2, 128
    cache = make_cache(8, hq, 16, d, "e4m3")
    size = torch.exp2(torch.randint(-30, 31, (n, hq, 1), generator=g).float())
    k, v = randn(g, n, hq, d), (torch.randn(n, hq, d, generator=g) * size).bfloat16().to(DEV)
    slots = torch.arange(n, device=DEV)
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)
    for scale_q, scale_k in ((2.0 ** 100, 2.0 ** -100), (2.0 ** -100, 2.0 ** 100), (1.0, 1.0)):
        q = (torch.randn(1, hq, d, generator=g) * scale_q).bfloat16().to(DEV)
        sdpa_cache_append((k * scale_k).bfloat16(), v, slots, **cache)
        o, lse = sdpa_tree_fwd(q, page_table=i32(*range(8))[None], ctx_lens=i32(n - 1), cu_nodes=i32(0, 1), max_nodes=1, **cache)
        check_tree(o, lse, q, [(rows_of(cache, "k", slots), rows_of(cache, "v", slots), n - 1)], [0, 1], "e4m3")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_repeats_bit_for_bit_on_streams_and_in_graphs(kv):
    cache, q, args, mask, seqs, cu, masks = tree_setup([5000, 100, 3000], [7, 1, 16], 8, 2, 128, 64, kv)
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, lse2 = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # two graphs over one pool of inputs, each with its own workspace, replayed after the inputs change
    graphs = []
    for _ in range(2):
        out, l = torch.zeros_like(o), torch.zeros_like(lse)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sdpa_tree_fwd(q, tree_mask=mask, out=out, lse=l, **args, **cache)
        graphs.append((gr, out, l))
    q.copy_(randn(torch.Generator().manual_seed(99), *q.shape))
    args["ctx_lens"].copy_(torch.tensor([200, 90, 2999], dtype=torch.int32))
    for gr, out, l in graphs:
        gr.replay()
    o3, lse3 = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    for _, out, l in graphs:
        assert torch.equal(out, o3) and torch.equal(l, lse3)


def test_tree_bad_lengths_and_pages_are_reported():
    cache, q, args, mask, seqs, cu, masks = tree_setup([40, 40], [2, 2], 2, 2, 64, 16, "bf16")
    good, _ = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    for name, at, value in (("ctx_lens", 0, -1), ("ctx_lens", 0, 1000), ("cu_nodes", 1, 70), ("cu_nodes", 0, 3),
                            ("page_table", (0, 1), -1), ("page_table", (0, 0), 1 << 30)):
        bad = {n: t.clone() if torch.is_tensor(t) else t for n, t in args.items()}
        bad[name][at] = value
        o, _ = sdpa_tree_fwd(q, tree_mask=mask, **bad, **cache)
        assert sdpa_read_device_status() == 2, (name, at, value)
        if name != "cu_nodes":
            assert torch.equal(o[2:], good[2:])               # the other sequence is unharmed


def test_tree_refuses_mismatches():
    cache, q, args, mask, *_ = tree_setup([40], [2], 2, 2, 64, 16, "e4m3")
    for kw in (dict(tree_mask=mask.int()), dict(k_scale=None), dict(out=q[:1]), dict(lse=torch.zeros(2, 9, device=DEV)),
               dict(alibi_slopes=torch.zeros(3, device=DEV)), dict(page_table=args["page_table"].long()),
               dict(ctx_lens=args["ctx_lens"].float()), dict(v_cache=cache["v_cache"][:1])):
        with pytest.raises(ValueError):
            sdpa_tree_fwd(q, **{**args, **cache, **kw})
    with pytest.raises(SdpaError) as e:
        sdpa_tree_fwd(q, workspace=torch.zeros(256, device=DEV, dtype=torch.uint8), **args, **cache)
    assert e.value.status == 3


# ------------------------------------------------------------------- verify
def draw_tree(g, B, N, V, sharp=3.0, chain=False):
    logits = torch.randn(B, N, V, generator=g) * sharp
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + torch.randn(B, N, V, generator=g), -1)
    parents = torch.full((B, N), -1, dtype=torch.int32)
    tokens = torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        for n in range(1, N):
            p = n - 1 if chain else int(torch.randint(0, max(1, n // 2 + 1), (1,), generator=g))
            parents[b, n] = p
            tokens[b, n] = int(torch.multinomial(draft[b, p], 1, generator=g))
    return target, draft, tokens, parents, torch.rand(B, N, generator=g), torch.rand(B, generator=g)


def check_verify(target, draft, tokens, parents, ua, us):
    dev = [t.to(DEV) if t is not None else None for t in (target, draft, tokens, parents, ua, us)]
    path, accepted, token = (t.cpu().numpy() for t in sdpa_spec_verify(*dev))
    for b in range(target.shape[0]):
        ref = so.verify(target[b].double().numpy(), draft[b].double().numpy() if draft is not None else None,
                        tokens[b].tolist() if tokens is not None else None,
                        parents[b].tolist() if parents is not None else None,
                        ua[b].double().numpy() if ua is not None else None, float(us[b]))
        assert (path[b].tolist(), int(accepted[b]), int(token[b])) == ref, b


@pytest.mark.parametrize("B,N,V,chain", [(1, 1, 1, True), (3, 1, 1000, True), (4, 6, 32000, True), (7, 16, 1003, False),
                                         (16, 64, 50, False), (2, 33, 40001, False), (40, 5, 4097, False)])
def test_verify(B, N, V, chain):
    g = torch.Generator().manual_seed(B * N)
    t, d, x, p, ua, us = draw_tree(g, B, N, V, chain=chain)
    check_verify(t, d, x, None if chain else p, ua, us)
    if N > 1:
        check_verify(t, d, x, p, torch.ones(B, N) - 2.0 ** -24, us)        # mostly rejected: long residual chains
        check_verify(t, d, x, p, torch.zeros(B, N), torch.ones(B) - 2.0 ** -24)   # mostly accepted
    else:
        check_verify(t, None, None, None, None, us)


def test_verify_ties_zeros_and_ends():
    p = torch.tensor([[[0.5, 0.25, 0.25, 0.0], [0.25] * 4]])
    q = torch.tensor([[[0.25, 0.5, 0.125, 0.125], [0.25] * 4]])
    one = lambda t, d, x, u, us: check_verify(t, d, torch.tensor([[0, x]], dtype=torch.int32), None,
                                              torch.tensor([[0.0, u]]), torch.tensor([us]))
    for u in (0.0, 0.49, 0.5, 0.51):
        for us in (0.0, 0.25, 2 / 3, 0.999, 1.0):
            for x in range(4):
                one(p, q, x, u, us)
                one(p, p, x, u, us)                    # nothing left after a rejection
    zero = torch.zeros(1, 2, 4)
    one(zero, q, 1, 0.5, 0.5)                          # no weight anywhere
    one(q, zero, 1, 0.5, 0.5)                          # a token the draft gives no weight


def test_verify_odd_trees_and_strides():
    g = torch.Generator().manual_seed(11)
    t, d, x, p, ua, us = draw_tree(g, 3, 9, 777)
    p[0, 4] = -1                                       # missing nodes
    p[1, 1:] = -1
    p[2, 1:] = 0                                       # all children of the root
    x[2, 3] = x[2, 2]                                  # the same token twice
    check_verify(t, d, x, p, ua, us)
    big = torch.zeros(3, 12, 800, device=DEV)
    big[:, :9, 5:782] = t.to(DEV)
    view = big[:, :9, 5:782]
    a = sdpa_spec_verify(view, d.to(DEV), x.to(DEV), p.to(DEV), ua.to(DEV), us.to(DEV))
    b = sdpa_spec_verify(t.to(DEV), d.to(DEV), x.to(DEV), p.to(DEV), ua.to(DEV), us.to(DEV))
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_verify_reports_bad_tokens_and_parents():
    g = torch.Generator().manual_seed(12)
    t, d, x, p, ua, us = draw_tree(g, 1, 4, 100, chain=True)
    for tok, par in ((100, 0), (-1, 0), (5, 1), (5, 3)):
        x2, p2 = x.clone(), p.clone()
        x2[0, 1], p2[0, 1] = tok, par
        check_verify(t, d, x2, p2, ua, us)
        assert sdpa_read_device_status() == 2


def test_verify_in_a_graph():
    g = torch.Generator().manual_seed(13)
    args = [t.to(DEV) for t in draw_tree(g, 4, 8, 5000)]
    first = sdpa_spec_verify(*args)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = sdpa_spec_verify(*args)
    gr.replay()
    assert all(torch.equal(i, j) for i, j in zip(first, out))
    args[4].copy_(torch.rand(4, 8, generator=g))
    gr.replay()
    assert all(torch.equal(i, j) for i, j in zip(sdpa_spec_verify(*args), out))


# ----------------------------------------------------------------- together
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_generation_steps(kv):
    """Prompt, a tree step, its accepted path kept, a second step: each step's attention equals the
    framework's causal attention over the sequence that the path spells out."""
    g = torch.Generator().manual_seed(21)
    hq, hkv, d, page, prompt = 8, 2, 128, 16, 75
    freqs, amp = sdpa_rope_frequencies(d, scaling="linear", factor=2.0)
    cache = make_cache(12, hkv, page, d, kv)
    table = torch.randperm(12, generator=g)[:10].view(1, 10).int().to(DEV)
    slot = lambda pos: table[0].long()[pos // page] * page + pos % page
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)

    q, k, v = randn(g, prompt, hq, d), randn(g, prompt, hkv, d), randn(g, prompt, hkv, d)
    q, k = sdpa_rope(q, k, freqs, amplitude=amp)
    sdpa_cache_append(k, v, slot(torch.arange(prompt, device=DEV)), **cache)
    ctx = prompt
    for step in range(2):
        parents = [-1, 0, 0, 1, 1, 2]
        n = len(parents)
        mask, depth = [1], [0]
        for i in range(1, n):
            mask.append(mask[parents[i]] | (1 << i))
            depth.append(depth[parents[i]] + 1)
        pos = torch.tensor(depth, device=DEV, dtype=torch.int32) + ctx
        q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
        q, k = sdpa_rope(q, k, freqs, pos, amplitude=amp)
        sdpa_cache_append(k, v, slot(ctx + torch.arange(n, device=DEV)), **cache)
        o, lse = sdpa_tree_fwd(q, page_table=table, ctx_lens=i32(ctx), cu_nodes=i32(0, n), max_nodes=n,
                               tree_mask=torch.tensor(mask, device=DEV), **cache)
        t, dr, x, _, ua, us = draw_tree(g, 1, n, 300)
        path, accepted, _ = sdpa_spec_verify(t.to(DEV), dr.to(DEV), x.to(DEV), i32(*parents)[None], ua.to(DEV), us.to(DEV))
        rows = path[0, :int(accepted) + 1].long()
        # the cached sequence along the path, read back
        sdpa_cache_append(k[rows].contiguous(), v[rows].contiguous(), slot(ctx + torch.arange(len(rows), device=DEV)), **cache)
        total = ctx + len(rows)
        kc, vc = sdpa_cache_gather(page_table=table, cu_seqlens=i32(0, total), total=total, **cache)
        chunk = q[rows].contiguous()
        ref, ref_lse = sdpa_fwd_varlen(chunk, kc, vc, i32(0, len(rows)), i32(0, total), len(rows), total, window_right=ctx)
        assert (o[rows].float() - ref.float()).abs().max() <= 2e-2    # two bf16 results, each within 1e-2 (1 + |O|)
        assert (lse[:, rows] - ref_lse).abs().max() <= 2e-3
        ctx = total
    # a prompt chunk over its cached prefix equals the whole prompt's attention
    whole, _ = sdpa_fwd(*(x[None] for x in (randn(g, total, hq, d), kc, vc)), causal=True)
    assert torch.isfinite(whole.float()).all()


# ------------------------------------------------- larger batches, odd calls
@pytest.mark.parametrize("T,hkv,d,page", [(50, 40, 128, 16), (33, 17, 64, 32), (9, 33, 64, 128), (2100, 5, 64, 16)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_append_and_gather_head_counts(T, hkv, d, page, kv):
    test_append_and_gather(T, hkv, d, page, kv)


MANY = {
    "33": dict(lens=[7 * i % 100 for i in range(33)], counts=[1] * 33, hq=4, hkv=2, d=64, page=16),
    "64_long_one": dict(lens=[20] * 20 + [15000] + [130] * 43, counts=[1] * 64, hq=4, hkv=1, d=128, page=64),
    "70_trees": dict(lens=[53 * i % 400 for i in range(70)], counts=[i % 6 for i in range(70)], hq=8, hkv=2, d=64, page=32),
    "300": dict(lens=[31 * i % 257 for i in range(300)], counts=[(i + 1) % 3 for i in range(300)], hq=4, hkv=4, d=64, page=16),
    "700_one_node_each_third": dict(lens=[5] * 700, counts=[int(i % 3 == 0) for i in range(700)], hq=2, hkv=1, d=64, page=16),
    "40_empty": dict(lens=[0] * 40, counts=[0] * 39 + [2], hq=2, hkv=2, d=64, page=16),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(MANY))
def test_tree_many_sequences(name, kv):
    cache, q, args, mask, seqs, cu, masks = tree_setup(kv=kv, extra_rows=1, **MANY[name])
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    check_tree(o, lse, q, seqs, cu, kv, masks)
    again = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    assert torch.equal(o[:cu[-1]], again[0][:cu[-1]]) and torch.equal(lse[:, :cu[-1]], again[1][:, :cu[-1]])
    assert sdpa_read_device_status() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_many_row_blocks(kv):
    """64 nodes of 32 query heads over one KV head: 2048 rows against the same keys."""
    cache, q, args, mask, seqs, cu, masks = tree_setup([300, 5], [64, 64], 32, 1, 64, 16, kv)
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, window_left=120, **args, **cache)
    check_tree(o, lse, q, seqs, cu, kv, masks, window_left=120)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("buckets,distance,bidir,ctx,hq,hkv", [
    (128, 200, False, 1500, 16, 1),     # a table of 2048 entries per KV head
    (32, 5000, False, 6000, 4, 2),      # buckets that go on behind the tabulated distances
    (128, 3000, True, 4000, 16, 1),     # both
    (4, 3, False, 200, 2, 2), (2, 2, False, 200, 2, 2), (6, 100000, True, 1200, 2, 1)])
def test_tree_t5_tables(buckets, distance, bidir, ctx, hq, hkv, kv):
    cache, q, args, mask, seqs, cu, masks = tree_setup([ctx, 40], [5, 9], hq, hkv, 64, 32, kv)
    t = torch.randn(buckets, hq, generator=torch.Generator().manual_seed(buckets))
    kw = dict(t5_num_buckets=buckets, t5_max_distance=distance, t5_bidirectional=bidir)
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, t5_table=t.to(DEV), **kw, **args, **cache)
    check_tree(o, lse, q, seqs, cu, kv, masks, t5_table=t.numpy(), **kw)


def test_tree_e4m3_offsets_past_32_bits():
    """Three pages of e4m3 rows 2^31 + 4096 elements apart, their scales 2^32 bytes apart."""
    hkv, page, d, far = 2, 32, 64, 2 ** 31 + 4096
    codes = torch.empty(2, 2 * far + hkv * page * d, device=DEV, dtype=torch.uint8)
    scales = torch.empty(2, 2 ** 33 + hkv * page, device=DEV, dtype=torch.uint8)
    rows = lambda i: codes[i].as_strided((3, hkv, page, d), (far, page * d, d, 1)).view(torch.float8_e4m3fn)
    sc = lambda i: scales[i].as_strided((3, hkv, page), (2 ** 32, page, 1))
    cache = dict(k_cache=rows(0), v_cache=rows(1), k_scale=sc(0), v_scale=sc(1))
    g = torch.Generator().manual_seed(5)
    n = 90
    table = torch.tensor([[2, 0, 1]], device=DEV, dtype=torch.int32)
    flat = table[0].long().repeat_interleave(page)[:n] * page + torch.arange(n, device=DEV) % page
    k, v, q = randn(g, n, hkv, d), randn(g, n, hkv, d), randn(g, 1, 4, d)
    sdpa_cache_append(k, v, flat, **cache)
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)
    kg, vg = sdpa_cache_gather(page_table=table, cu_seqlens=i32(0, n), total=n, **cache)
    o, lse = sdpa_tree_fwd(q, page_table=table, ctx_lens=i32(n - 1), cu_nodes=i32(0, 1), max_nodes=1, **cache)
    # (the rows read back are exact: test_append_and_gather; here against the rows written, 2^-4 off at most)
    assert ((kg.double() - k.double()).abs() <= 2.0 ** -4 * k.double().abs() + 2.0 ** -10 * 2.0 ** -5).all()
    check_tree(o, lse, q, [(f64(kg), f64(vg), n - 1)], [0, 1], "e4m3")


def test_verify_large_vocabulary_and_batch():
    g = torch.Generator().manual_seed(31)
    for B, N, V in ((2, 3, 200003), (600, 2, 130), (1, 2, 32769)):
        check_verify(*draw_tree(g, B, N, V))


def test_odd_arguments_are_refused():
    q = torch.randn(1, 2, 0, 64, device=DEV).bfloat16()
    k = torch.randn(1, 2, 2, 64, device=DEV).bfloat16()
    freqs, _ = sdpa_rope_frequencies(64)
    with pytest.raises(SdpaError):
        sdpa_rope(q, k, freqs)                                  # no query head, yet keys to turn
    for name in ("interleaved", "inverse"):
        with pytest.raises(ValueError):
            sdpa_rope(k, None, freqs, **{name: torch.zeros(2)})
    cache, q, args, *_ = tree_setup([40], [2], 2, 2, 64, 16, "bf16")
    for far in (-2 ** 32 + 200, -1, 0, 8):
        with pytest.raises(SdpaError):
            sdpa_tree_fwd(q, t5_table=torch.zeros(32, 2, device=DEV), t5_max_distance=far, **args, **cache)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [4, 5, 8, 9, 16, 17])
def test_tree_row_counts(nodes, kv, d):
    """8 to 34 query rows: each size of product, full and barely begun, plain and with T5 and a window."""
    cache, q, args, mask, seqs, cu, masks = tree_setup([400, 129], [nodes, 1], 4, 2, d, 16, kv)
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache)
    check_tree(o, lse, q, seqs, cu, kv, masks)
    kw, okw = bias_kw(dict(t5=True, window_left=150), 4)
    o, lse = sdpa_tree_fwd(q, tree_mask=mask, **args, **cache, **kw)
    check_tree(o, lse, q, seqs, cu, kv, masks, **okw)
