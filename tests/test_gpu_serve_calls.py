"""GPU tests of calls that a serving program makes: tables whose pages are gone, ties after
a rejection, prompt chunks over a cached prefix."""
import pytest
import torch

from scaled_dot_product_bwd_b200 import (SdpaError, sdpa_cache_append, sdpa_cache_gather, sdpa_fwd, sdpa_fwd_varlen,
                                         sdpa_read_device_status, sdpa_rope, sdpa_rope_frequencies,
                                         sdpa_spec_verify, sdpa_tree_fwd)
from test_gpu_serve import DEV, check_verify, draw_tree, make_cache, randn, tree_setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("window", [100, 0])
def test_pages_behind_the_window_may_be_gone(page, window, kv):
    """Pages that hold no key inside any node's window are not reported, whatever the table says;
    those that hold one are."""
    lens, counts = [1000, 300, 2000], [3, 1, 17]
    cache, q, args, mask, *_ = tree_setup(lens, counts, 4, 2, 64, page, kv)
    want = sdpa_tree_fwd(q, tree_mask=mask, window_left=window, **args, **cache)
    assert sdpa_read_device_status() == 0
    table = args["page_table"].clone()
    for b, (ctx, gone) in enumerate(zip(lens, (-1, 1 << 30, -7))):
        table[b, :(ctx - window) // page] = gone
    got = sdpa_tree_fwd(q, tree_mask=mask, window_left=window, **{**args, "page_table": table}, **cache)
    assert sdpa_read_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b, ctx in enumerate(lens):
        bad = table.clone()
        bad[b, (ctx - window) // page] = -1
        sdpa_tree_fwd(q, tree_mask=mask, window_left=window, **{**args, "page_table": bad}, **cache)
        assert sdpa_read_device_status() == 2
    table[0, 0] = -1
    sdpa_tree_fwd(q, tree_mask=mask, **{**args, "page_table": table}, **cache)    # no window: needed
    assert sdpa_read_device_status() == 2


@pytest.mark.parametrize("vocab", [4, 4000, 40000])
def test_a_tie_after_a_rejection_is_a_rejection(vocab):
    """The second child's u q(x) equals (p - q)(x) / Z exactly, with a Z that is no power of two; next
    to it on either side; and so the third child's after a second rejection."""
    def spread(*at):
        row = torch.zeros(vocab, dtype=torch.float64)
        for x, value in zip((0, vocab // 2, vocab - 2, vocab - 1), at):
            row[x] = value
        return row
    t, z = 1125 / 65536, 4800 / 65536            # t / Z = 15 / 64 = 0.375 * 0.625
    p = spread(0.625 + t, 0.125 + z - t, 0.0, 0.0)
    q = spread(0.625, 0.125, 0.125, 0.125)
    assert (p.float().double() == p).all() and (q.float().double() == q).all()
    n = 4
    target, draft = p.float().repeat(1, n, 1), q.float().repeat(1, n, 1)
    tokens = torch.tensor([[0, vocab - 1, 0, 0]], dtype=torch.int32)
    parents = torch.tensor([[-1, 0, 0, 0]], dtype=torch.int32)
    for u in (0.375, 0.375 - 2.0 ** -25, 0.375 + 2.0 ** -24):
        for third in (0.0, 0.5):
            check_verify(target, draft, tokens, parents, torch.tensor([[0.0, 0.5, u, third]]), torch.tensor([0.3]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("prefix,chunk", [(75, 100), (1000, 129), (1, 200)])
def test_a_prompt_chunk_over_its_cached_prefix_is_the_whole_prompt(prefix, chunk, kv):
    """Two sequences of one prefix length: their chunks over the rows read back equal those rows of
    causal attention over the whole prompt, over the same keys.  Both are bf16 results within the
    attention tests' 1e-2 (1 + |O|) of the definition."""
    g = torch.Generator().manual_seed(prefix)
    hq, hkv, d, page, n = 8, 2, 128, 16, prefix + chunk
    pages = -(-n // page)
    cache = make_cache(2 * pages + 1, hkv, page, d, kv)
    table = torch.randperm(2 * pages + 1, generator=g)[:2 * pages].view(2, pages).int().to(DEV)
    pos = torch.arange(n, device=DEV)
    q = randn(g, 2, n, hq, d)
    for b in range(2):
        slots = table[b].long()[pos // page] * page + pos % page
        for part in (slice(0, prefix), slice(prefix, n)):
            rows = len(slots[part])
            sdpa_cache_append(randn(g, rows, hkv, d), randn(g, rows, hkv, d), slots[part].contiguous(), **cache)
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)
    k, v = sdpa_cache_gather(page_table=table, cu_seqlens=i32(0, n, 2 * n), total=2 * n, **cache)
    whole, whole_lse = sdpa_fwd(q, k.view(2, n, hkv, d), v.view(2, n, hkv, d), causal=True)
    o, lse = sdpa_fwd_varlen(q[:, prefix:].reshape(2 * chunk, hq, d), k, v, i32(0, chunk, 2 * chunk), i32(0, n, 2 * n),
                             chunk, n, window_right=prefix)
    want, want_lse = whole[:, prefix:].reshape(2 * chunk, hq, d).float(), whole_lse[:, :, prefix:]
    assert ((o.float() - want).abs() <= 2e-2 * (1 + want.abs())).all()
    assert ((lse.view(hq, 2, chunk).transpose(0, 1) - want_lse).abs() <= 2e-3).all()


def test_one_row_of_positions_or_pages_for_all_sequences():
    g = torch.Generator().manual_seed(1)
    freqs, _ = sdpa_rope_frequencies(64)
    q = randn(g, 3, 20, 2, 64)
    pos = torch.arange(20, device=DEV, dtype=torch.int32) * 7
    assert torch.equal(sdpa_rope(q, None, freqs, pos.expand(3, 20))[0], sdpa_rope(q, None, freqs, pos.repeat(3, 1))[0])
    cache, q, args, mask, *_ = tree_setup([40, 40, 17], [2, 2, 2], 2, 2, 64, 16, "bf16")
    table = args["page_table"][:1]
    one, each = ({**args, "page_table": t} for t in (table.expand(3, -1), table.repeat(3, 1)))
    a, b = sdpa_tree_fwd(q, tree_mask=mask, **one, **cache), sdpa_tree_fwd(q, tree_mask=mask, **each, **cache)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cu = torch.tensor([0, 40, 45, 62], device=DEV, dtype=torch.int32)
    a, b = (sdpa_cache_gather(page_table=x["page_table"], cu_seqlens=cu, total=62, **cache) for x in (one, each))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_two_streams_at_once(kv):
    """Calls of different sizes on two streams, whose kernels may run side by side: the same bits."""
    cases = []
    for seed, (lens, counts) in enumerate((([3000, 100, 5], [7, 1, 16]), ([800] * 40, [1] * 40))):
        cache, q, args, mask, *_ = tree_setup(lens, counts, 8, 2, 128, 64, kv, seed=seed)
        t, d, x, p, ua, us = (y.to(DEV) for y in draw_tree(torch.Generator().manual_seed(seed), 4, 9, 9000))
        def call(cache=cache, q=q, args=args, mask=mask, v=(t, d, x, p, ua, us)):
            return *sdpa_tree_fwd(q, tree_mask=mask, **args, **cache), *sdpa_spec_verify(*v)
        cases.append((call, call()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (call, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(call())
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(cases):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_generation_step_in_a_graph(kv):
    """Rotation, write, attention, read-back and verification captured together and replayed with
    other inputs: what the calls give one by one."""
    g = torch.Generator().manual_seed(3)
    hq, hkv, d, page, n, ctx = 8, 2, 128, 16, 6, 90
    freqs, amp = sdpa_rope_frequencies(d, scaling="yarn", factor=4.0, original_length=64)
    cache = make_cache(8, hkv, page, d, kv)
    table = torch.tensor([[5, 0, 7, 2, 1, 3, 6]], device=DEV, dtype=torch.int32)
    i32 = lambda *x: torch.tensor(x, device=DEV, dtype=torch.int32)
    slot = lambda pos: table[0].long()[pos // page] * page + pos % page
    sdpa_cache_append(randn(g, ctx, hkv, d), randn(g, ctx, hkv, d), slot(torch.arange(ctx, device=DEV)), **cache)
    q, k, v = randn(g, n, hq, d), randn(g, n, hkv, d), randn(g, n, hkv, d)
    pos, slots = i32(*range(ctx, ctx + n)), slot(ctx + torch.arange(n, device=DEV))
    cu, ctx_lens, all_rows = i32(0, n), i32(ctx), i32(0, ctx + n)
    tree = [t.to(DEV) for t in draw_tree(g, 1, n, 500, chain=True)]

    def step():
        rq, rk = sdpa_rope(q, k, freqs, pos, amplitude=amp)
        sdpa_cache_append(rk, v, slots, **cache)
        o, lse = sdpa_tree_fwd(rq, page_table=table, ctx_lens=ctx_lens, cu_nodes=cu, max_nodes=n, **cache)
        return rq, o, lse, *sdpa_cache_gather(page_table=table, cu_seqlens=all_rows, total=ctx + n, **cache), \
            *sdpa_spec_verify(*tree)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        g = torch.Generator().manual_seed(100 + seed)
        for t in (q, k, v):
            t.copy_(randn(g, *t.shape))
        for t, new in zip(tree, draw_tree(g, 1, n, 500, chain=True)):
            t.copy_(new)
        graph.replay()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 5, 700])
def test_append_of_a_rotated_key_and_a_slice_of_a_fused_buffer(T, kv):
    """K fresh from the rotation, V and slots as they are: what an append of copies gives."""
    g = torch.Generator().manual_seed(T)
    hq, hkv, d, page = 4, 2, 64, 16
    freqs, _ = sdpa_rope_frequencies(d)
    qkv = randn(g, T, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    _, k = sdpa_rope(q, k, freqs)
    assert T == 1 or k.stride() != v.stride()
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[:1] = -1 if T > 1 else slots[:1]
    a, b = make_cache(pages, hkv, page, d, kv), make_cache(pages, hkv, page, d, kv)
    sdpa_cache_append(k, v, slots.to(DEV), **a)
    sdpa_cache_append(k, v.contiguous(), slots.to(DEV), **b)
    raw = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)
    for name in a:
        assert a[name] is None or torch.equal(raw(a[name]), raw(b[name])), name
    for bad in (v.float(), v[:, :1], v[:0] if T > 1 else v[:, :, :32]):
        with pytest.raises(ValueError):
            sdpa_cache_append(k, bad, slots.to(DEV), **a)
    # refused before K is written: a base off by 8 bytes, rows of one stride of 0
    odd = torch.zeros(T, 2 * hkv, d + 8, device=DEV, dtype=torch.bfloat16)[:, :hkv, 4:4 + d]
    for bad in (odd, v[:1, :1].expand(T, hkv, d)):
        with pytest.raises(SdpaError):
            sdpa_cache_append(torch.full_like(k, 5.0), bad, slots.to(DEV), **a)
    assert torch.equal(raw(a["k_cache"]), raw(b["k_cache"]))
