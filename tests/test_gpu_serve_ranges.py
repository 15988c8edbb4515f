"""GPU tests of the serving operators at the ends of their number ranges: far keys and
values, biases of the type's lowest value, value rows of zeros, many small weights.

Bounds are test_gpu_serve.py's (its module docstring) unless a test says otherwise.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serve_oracle as so
from scaled_dot_product_bwd_b200 import sdpa_cache_append, sdpa_tree_fwd
from test_gpu_serve import DEV, check_tree, f64, make_cache, rows_of, tree_tolerance

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, device=DEV, dtype=torch.int32)


def filled(k, v, kv="e4m3", page=16):
    """A cache that holds rows k, v [n, Hkv, d] from slot 0 on, its table, and the rows as stored."""
    n, hkv, d = k.shape
    pages = -(-n // page)
    cache = make_cache(pages, hkv, page, d, kv)
    slots = torch.arange(n, device=DEV)
    sdpa_cache_append(k.bfloat16().to(DEV), v.bfloat16().to(DEV), slots, **cache)
    return cache, i32(*range(pages))[None], (rows_of(cache, "k", slots), rows_of(cache, "v", slots))


@pytest.mark.parametrize("q_size,k_size", [(-110, 113), (-110, 110), (116, -113), (0, 0)])
@pytest.mark.parametrize("nodes", [1, 16, 40])
def test_keys_near_one_end_under_queries_near_the_other(nodes, q_size, k_size):
    """Finite scores of keys and queries near the ends of bf16's range, though the product of a key's
    codes and its scale, or of a query's, leaves float32."""
    g = torch.Generator().manual_seed(nodes)
    n, hq, d = 200 + nodes, 2, 128
    k, v = torch.randn(n, hq, d, generator=g), torch.randn(n, hq, d, generator=g)
    q = torch.randn(nodes, hq, d, generator=g)
    k[7] = 48 * q[0].sign()                      # products of one sign: a sum near its largest
    q = (q * 2.0 ** q_size).bfloat16().to(DEV)
    cache, table, rows = filled(k * 2.0 ** k_size, v)
    o, lse = sdpa_tree_fwd(q, page_table=table, ctx_lens=i32(n - nodes), cu_nodes=i32(0, nodes), max_nodes=nodes, **cache)
    check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3")


# one piece per CTA where every sequence is the same: the whole line's tiles in one accumulator
COPIES = 148


def attend(q, cache, table, ctx, copies=1, **kw):
    """O, LSE of nodes q [n, Hq, d] at ctx, as one sequence or as copies of it over the same pages."""
    n = len(q)
    o, lse = sdpa_tree_fwd(q.repeat(copies, 1, 1), page_table=table.repeat(copies, 1), ctx_lens=i32(*[ctx] * copies),
                           cu_nodes=i32(*range(0, n * copies + 1, n)), max_nodes=n, **kw, **cache)
    for c in range(1, copies):
        assert torch.equal(o[:n], o[c * n:c * n + n]) and torch.equal(lse[:, :n], lse[:, c * n:c * n + n])
    return o[:n], lse[:, :n]


@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -1e38, -1e8, -1e5, 0.0])
@pytest.mark.parametrize("nodes,copies", [(1, 1), (16, 1), (40, 1), (1, COPIES), (40, COPIES)])
def test_biases_that_leave_no_digits_for_the_scores(nodes, copies, low):
    """Every key under the same bias, down to the type's lowest value, and equal scores (q = 0): the
    mean of the values, whose scales differ by up to 2^7 from row to row."""
    g = torch.Generator().manual_seed(nodes)
    n, hq, d = 300 + nodes, 1, 64
    k, v = torch.randn(n, hq, d, generator=g), torch.randn(n, hq, d, generator=g)
    cache, table, rows = filled(k, v * torch.exp2(torch.randint(-4, 4, (n, hq, 1), generator=g).float()))
    q = torch.zeros(nodes, hq, d, device=DEV).bfloat16()
    o, _ = attend(q, cache, table, n - nodes, copies, t5_table=torch.full((32, hq), low, device=DEV), t5_bidirectional=False)
    _, lse = attend(q, cache, table, n - nodes, copies)
    check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3")


@pytest.mark.parametrize("size", [-116, -100, -60, 60, 100, 120])
@pytest.mark.parametrize("nodes", [1, 16, 40])
def test_values_near_the_ends_of_the_range(nodes, size):
    g = torch.Generator().manual_seed(nodes)
    n, hq, d = 500 + nodes, 2, 64
    k, v, q = (torch.randn(m, hq, d, generator=g) for m in (n, n, nodes))
    cache, table, rows = filled(k, v * 2.0 ** size)
    for steep in (1, 8):                         # weights of one size, and over 2^80
        o, lse = attend((steep * q).bfloat16().to(DEV), cache, table, n - nodes)
        check_tree(o, lse, (steep * q).bfloat16(), [(*rows, n - nodes)], [0, nodes], "e4m3")


@pytest.mark.parametrize("nodes", [1, 16, 40])
def test_many_small_weights_on_values_near_the_largest(nodes):
    """One key of weight 1 and 2^16 of weight 2^-16, with values of 2^126 and -2^125: half of O's
    weight lies 2^-16 below the largest."""
    g = torch.Generator().manual_seed(nodes)
    n, d = 65536 + nodes, 64
    u = torch.randn(1, d, generator=g).bfloat16().float()
    k, v = torch.zeros(n, 1, d), torch.full((n, 1, d), -2.0 ** 125)
    k[3] = u * (16 * math.log(2) * math.sqrt(d) / (u * u).sum())
    v[3] = 2.0 ** 126
    q = u.expand(nodes, 1, d).bfloat16().to(DEV)
    cache, table, rows = filled(k, v, page=256)
    o, lse = attend(q, cache, table, n - nodes, COPIES)
    check_tree(o[:1], lse[:, :1], q[:1], [(rows[0][:n - nodes + 1], rows[1][:n - nodes + 1], n - nodes)], [0, 1], "e4m3")
    assert (o.double().abs() < 2.0 ** 125).all()


@pytest.mark.parametrize("step", [8, -8])
@pytest.mark.parametrize("nodes,copies", [(1, 1), (1, COPIES), (16, COPIES), (40, COPIES)])
def test_scores_that_rise_as_the_values_fall(nodes, copies, step):
    """From tile to tile weights rise (or fall) by 2^8 and the values' scales do the opposite: each tile
    adds as much to O, while the sum of weights grows by 2^128."""
    g = torch.Generator().manual_seed(nodes)
    tiles, d = 17, 64
    n = 128 * tiles + nodes
    u = torch.randn(1, d, generator=g).bfloat16().float()
    tile = (torch.arange(n) // 128)[:, None, None].float()
    k = u * (step * math.log(2) * math.sqrt(d) / (u * u).sum()) * (tile - 8)
    v = torch.randn(n, 1, d, generator=g) * torch.exp2(step * (8 - tile))
    q = u.expand(nodes, 1, d).bfloat16().to(DEV)
    cache, table, rows = filled(k, v)
    o, lse = attend(q, cache, table, n - nodes, copies)
    check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3")


@pytest.mark.parametrize("size", [1.0, 0.1, 1e-4])
@pytest.mark.parametrize("lead", [0.0, 8.0, 9.7, 11.0, 100.0])
@pytest.mark.parametrize("nodes,copies", [(1, 1), (1, COPIES), (16, COPIES), (40, COPIES)])
def test_value_rows_of_zeros(nodes, copies, lead, size):
    """Value rows of zeros (stored with a scale of 1), one of them under the highest score: they add to
    the sum of weights and take nothing from the other keys' weights."""
    g = torch.Generator().manual_seed(nodes)
    n, d = 4096 + nodes, 128
    u = torch.randn(1, d, generator=g)
    q = (u + 0.05 * torch.randn(nodes, 1, d, generator=g)).bfloat16().to(DEV)
    k, v = torch.randn(n, 1, d, generator=g), size * torch.randn(n, 1, d, generator=g)
    k[5] = u * (lead * math.sqrt(d) / (u * u).sum())
    v[5] = v[700] = v[n - nodes - 1] = v[n - 1] = 0.0
    cache, table, rows = filled(k, v, page=64)
    o, lse = attend(q, cache, table, n - nodes, copies)
    check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3")


@pytest.mark.parametrize("nodes", [1, 16, 40])
def test_values_of_zeros_alone(nodes):
    g = torch.Generator().manual_seed(nodes)
    n, d = 400 + nodes, 64
    k, q = torch.randn(n, 1, d, generator=g), torch.randn(nodes, 1, d, generator=g).bfloat16().to(DEV)
    cache, table, rows = filled(k, torch.zeros(n, 1, d))
    for kw in (dict(), dict(alibi_slopes=torch.ones(1, device=DEV))):
        o, lse = attend(q, cache, table, n - nodes, **kw)
        assert (o == 0).all()
        check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3",
                   **{name: t.cpu().numpy() for name, t in kw.items()})


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("gap", [1.0, 12.0, 40.0, 200.0])
@pytest.mark.parametrize("ctx", [5, 128, 300])
@pytest.mark.parametrize("window", [-1, 3])
def test_nan_values_reach_their_viewers_whatever_their_weight(ctx, gap, window, kv):
    """Values of NaN of a node `gap` nats below the other keys: NaN for the node that sees it, and for it alone."""
    g = torch.Generator().manual_seed(5)
    nodes, d = 3, 64
    u = torch.randn(1, d, generator=g).bfloat16().float()
    k, v = torch.zeros(ctx + nodes, 1, d), torch.randn(ctx + nodes, 1, d, generator=g)
    k[ctx + 1] = -u * (gap * math.sqrt(d) / (u * u).sum())
    v[ctx + 1] = float("nan")
    cache, table, _ = filled(k, v, kv)
    q = u.expand(nodes, 1, d).bfloat16().to(DEV)
    mask = torch.tensor([0b001, 0b011, 0b101], device=DEV)
    o, lse = attend(q, cache, table, ctx, tree_mask=mask, window_left=window)
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("gap", [1.0, 12.0, 40.0])
def test_infinite_values_reach_their_viewers_whatever_their_weight(gap):
    g = torch.Generator().manual_seed(6)
    ctx, nodes, d = 70, 3, 64
    u = torch.randn(1, d, generator=g).bfloat16().float()
    k, v = torch.zeros(ctx + nodes, 1, d), torch.randn(ctx + nodes, 1, d, generator=g)
    k[ctx + 1] = -u * (gap * math.sqrt(d) / (u * u).sum())
    v[ctx + 1, :, ::2], v[ctx + 1, :, 1::2] = float("inf"), -float("inf")
    cache, table, _ = filled(k, v, "bf16")
    q = u.expand(nodes, 1, d).bfloat16().to(DEV)
    o, _ = attend(q, cache, table, ctx, tree_mask=torch.tensor([0b001, 0b011, 0b101], device=DEV))
    assert (o[1, :, ::2] == float("inf")).all() and (o[1, :, 1::2] == -float("inf")).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,nodes", [(40, 1), (3000, 1), (300, 16), (0, 1)])
def test_lse_of_rows_whose_biases_are_the_lowest_value(ctx, nodes, kv):
    """Such a row's LSE is that value (its scores and the count of its keys are far below its last
    digit); a row hidden by -inf has -inf."""
    g = torch.Generator().manual_seed(ctx)
    n, hq, d = ctx + nodes, 2, 64
    cache, table, _ = filled(torch.randn(n, hq, d, generator=g), torch.randn(n, hq, d, generator=g), kv)
    q = torch.randn(nodes, hq, d, generator=g).bfloat16().to(DEV)
    low = torch.finfo(torch.float32).min
    t5 = torch.tensor([[low, -float("inf")]] * 32, device=DEV)
    o, lse = attend(q, cache, table, ctx, t5_table=t5, t5_bidirectional=False)
    assert (lse[0] == low).all() and torch.isfinite(o[:, 0]).all()
    assert torch.isneginf(lse[1]).all() and (o[:, 1] == 0).all()


@pytest.mark.parametrize("below", [20.4, 21.0, 21.6, 23.0])
@pytest.mark.parametrize("noise", [0.0, 1.0])
@pytest.mark.parametrize("nodes", [1, 16, 40])
def test_many_weights_below_the_last_step_of_the_weights(nodes, noise, below):
    """32767 keys 2^-below of the largest weight each, all in one piece: together up to 2 % of O.

    Each weight is off by at most 2^-20 of the largest, unbiased over the keys: for n keys a standard
    deviation of at most sqrt(n) 2^-21, and six of them are allowed beside the roundings of the
    module docstring of test_gpu_serve.py without its loss per key (2^-21 n, all of what is tested)."""
    g = torch.Generator().manual_seed(nodes)
    ctx, d = 32768, 64
    n = ctx + nodes
    u = torch.randn(1, d, generator=g).bfloat16().float()
    k = noise * torch.randn(n, 1, d, generator=g)
    k = k - (k @ u.T) * u / (u * u).sum() * 0.9
    k[0] = u * (below * math.log(2) * math.sqrt(d) / (u * u).sum())
    v = torch.ones(n, 1, d)
    v[0, :, 1:] = 0
    cache, table, rows = filled(k, v, page=256)
    q = u.expand(nodes, 1, d).bfloat16().to(DEV)
    o, _ = attend(q, cache, table, ctx, COPIES)
    ro, _, spread, size = so.tree_attention(f64(q[:1]), rows[0][:ctx + 1], rows[1][:ctx + 1], ctx)
    tol, _ = tree_tolerance(f64(q[:1]), rows[0], rows[1], ro, spread, size, "e4m3")
    tol += (6 * math.sqrt(n) * 2.0 ** -21 - 2.0 ** -21 * n) * np.abs(rows[1]).max()
    err = np.abs(f64(o[:1]) - ro)
    assert (err <= tol).all(), (float(err.max()), float(ro[..., 1:].min()))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20])
@pytest.mark.parametrize("nodes,copies", [(1, 1), (1, COPIES), (16, COPIES), (40, COPIES)])
def test_the_lowest_bias_after_tiles_that_a_row_does_not_see(nodes, copies, size, kv):
    """Far keys hidden by a bias of -inf, near ones under the type's lowest value: the near ones' mean
    (q = 0), whose weights the tiles before have left no reference for."""
    g = torch.Generator().manual_seed(nodes)
    ctx, d = 1000, 64
    n = ctx + nodes
    v = size * torch.randn(n, 1, d, generator=g) * torch.exp2(torch.randint(-3, 4, (n, 1, 1), generator=g).float())
    cache, table, rows = filled(torch.randn(n, 1, d, generator=g), v, kv)
    q = torch.zeros(nodes, 1, d, device=DEV).bfloat16()
    t5 = torch.full((32, 1), torch.finfo(torch.float32).min)
    t5[28:] = -float("inf")
    o, _ = attend(q, cache, table, ctx, copies, t5_table=t5.to(DEV), t5_bidirectional=False)
    t5[:28] = 0.0                                # (the same weights for the float64 definition)
    ro, _, spread, size = so.tree_attention(f64(q), *rows, ctx, t5_table=t5.numpy())
    tol, _ = tree_tolerance(f64(q), *rows, ro, spread, size, kv)
    err = np.abs(f64(o) - ro)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("sizes", [(0.0, 2.0 ** 100), (2.0 ** 100, 0.0), (2.0 ** -110, 2.0 ** 100), (2.0 ** 110, 2.0 ** -110),
                                   (0.0, 2.0 ** -110), (2.0 ** -40, 2.0 ** 60), (0.0, 1.0, 2.0 ** 90, 2.0 ** -90)])
@pytest.mark.parametrize("nodes,copies", [(1, 1), (1, COPIES), (16, COPIES), (40, COPIES)])
def test_values_of_one_size_after_values_of_another(nodes, copies, sizes):
    """Each size for some tiles, scores alike: every key counts in the sum of weights, whatever its value."""
    g = torch.Generator().manual_seed(nodes)
    d, run = 64, 640
    n = run * len(sizes) + nodes
    v = torch.randn(n, 1, d, generator=g)
    for i in range(n):
        v[i] *= sizes[min(i // run, len(sizes) - 1)]
    cache, table, rows = filled(torch.randn(n, 1, d, generator=g), v)
    q = torch.randn(nodes, 1, d, generator=g).bfloat16().to(DEV)
    o, lse = attend(q, cache, table, n - nodes, copies)
    check_tree(o, lse, q, [(*rows, n - nodes)], [0, nodes], "e4m3")


@pytest.mark.parametrize("byte", [255, 254, 0, 127])
@pytest.mark.parametrize("codes", [0x7F, 0x00, 0x7E])
@pytest.mark.parametrize("nodes", [1, 5, 40])
def test_hidden_rows_may_hold_any_codes_and_scales(nodes, codes, byte):
    """Keys behind the window, a node that none sees and the rest of the last page."""
    g = torch.Generator().manual_seed(nodes)
    ctx, d, page = 500, 64, 64
    n = ctx + nodes + 1
    k, v = torch.randn(n, 1, d, generator=g), torch.randn(n, 1, d, generator=g)
    cache, table, rows = filled(k, v, page=page)
    q = torch.randn(nodes + 1, 1, d, generator=g).bfloat16().to(DEV)
    words = [(2 << i) - 1 for i in range(nodes)] + [(1 << nodes) - 1]       # a chain; the last node sees it alone
    mask = torch.tensor(words, device=DEV)
    wild = list(range(ctx - 100)) + list(range(n - 1, cache["k_cache"].shape[0] * page))
    at = torch.tensor(wild, device=DEV)
    for name in ("k", "v"):
        cache[name + "_cache"].view(torch.uint8)[at // page, 0, at % page] = codes
        cache[name + "_scale"][at // page, 0, at % page] = byte
    got = attend(q, cache, table, ctx, tree_mask=mask, window_left=100)
    assert torch.isfinite(got[0]).all()
    check_tree(*got, q, [(*rows, ctx)], [0, nodes + 1], "e4m3", words, window_left=100)
