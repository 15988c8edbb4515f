"""GPU tests of the serving operators at the ends of their number ranges: far keys and
values, biases of the type's lowest value, value rows of zeros, many small weights.

Bounds are test_gpu_serve.py's (its module docstring) unless a test says otherwise.
"""
import pytest
import torch

from scaled_dot_product_bwd_b200 import sdpa_cache_append, sdpa_tree_fwd
from test_gpu_serve import DEV, check_tree, make_cache, rows_of

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
