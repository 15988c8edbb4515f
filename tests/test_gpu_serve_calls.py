"""GPU tests of calls that a serving program makes: tables whose pages are gone, ties after
a rejection, prompt chunks over a cached prefix."""
import pytest
import torch

from scaled_dot_product_bwd_b200 import (sdpa_cache_append, sdpa_cache_gather, sdpa_fwd, sdpa_fwd_varlen,
                                         sdpa_read_device_status, sdpa_tree_fwd)
from test_gpu_serve import DEV, check_verify, make_cache, randn, tree_setup

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
