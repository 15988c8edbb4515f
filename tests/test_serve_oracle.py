"""Pins of the serving operators' float64 definitions on hand-checkable inputs."""
import math

import numpy as np
import pytest
import torch

from oracle import attention_forward
from oracle import serve_oracle as so


def test_rotation_is_orthogonal_and_relative():
    rng = np.random.default_rng(0)
    f, amp = so.rope_frequencies(16)
    assert amp == 1.0 and f[0] == 1.0 and f[-1] == pytest.approx(10000.0 ** (-14 / 16))
    x = rng.standard_normal((5, 2, 20))
    pos = np.array([0, 1, 7, 100, 12345])
    for inter in (False, True):
        y = so.rope(x, pos, f, inter)
        assert np.array_equal(y[0], x[0])                        # position 0
        assert np.array_equal(y[..., 16:], x[..., 16:])          # beyond rot
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(so.rope(y, pos, f, inter, inverse=True), x)
    # scores depend on the difference of positions alone
    q, k = x[0, 0, :16], x[1, 0, :16]
    dot = lambda i, j: so.rope(q[None, None], [i], f)[0, 0] @ so.rope(k[None, None], [j], f)[0, 0]
    assert dot(3, 10) == pytest.approx(dot(1003, 1010))


def test_rotation_gradient_against_differences():
    rng = np.random.default_rng(1)
    f, amp = so.rope_frequencies(8, scaling="yarn", factor=4.0, original_length=64)
    x, g = rng.standard_normal((3, 1, 8)), rng.standard_normal((3, 1, 8))
    pos = np.array([5, 90, 201])
    grad = so.rope(g, pos, f, inverse=True, amplitude=amp)
    for at in np.ndindex(x.shape):
        e = np.zeros(x.shape)
        e[at] = 1e-6
        d = ((so.rope(x + e, pos, f, amplitude=amp) - so.rope(x - e, pos, f, amplitude=amp)) * g).sum()
        assert d / 2e-6 == pytest.approx(grad[at], rel=1e-6, abs=1e-8)


def test_scaled_frequencies():
    plain, _ = so.rope_frequencies(64)
    linear, _ = so.rope_frequencies(64, scaling="linear", factor=8.0)
    assert np.allclose(linear, plain / 8)
    ntk, _ = so.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 8)   # slowest pair interpolated
    yarn, amp = so.rope_frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    assert yarn[0] == plain[0] and yarn[-1] == pytest.approx(plain[-1] / 8)
    assert amp == pytest.approx(0.1 * math.log(8) + 1)


def test_e4m3_codes_against_torch():
    v = so.e4m3_values()
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    got = so.e4m3_decode(codes.numpy())
    assert np.array_equal(np.isnan(ref), np.isnan(got)) and np.array_equal(ref[~np.isnan(ref)], got[~np.isnan(got)])
    assert v[126] == 448.0
    x = np.random.default_rng(2).standard_normal(4000) * 2.0 ** np.random.default_rng(3).integers(-12, 8, 4000)
    mid = (v[:126] + v[1:127]) / 2                                # ties
    x = np.clip(np.concatenate([x, mid, -mid, v[:127]]), -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(so.e4m3_round(x.astype(np.float64)), ref)


def test_e4m3_row_scales():
    codes, e = so.e4m3_rows(np.array([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [2.0 ** -130, 0.0], [896.0, np.inf]]))
    assert list(e) == [127, 128, 127, 1, 128]
    assert so.e4m3_decode(codes)[0].tolist() == [448.0, 1.0]
    assert so.e4m3_decode(codes)[4].tolist() == [448.0, 448.0]
    x = np.random.default_rng(4).standard_normal((50, 64)) * 10.0 ** np.random.default_rng(5).integers(-6, 6, (50, 1))
    codes, e = so.e4m3_rows(x)
    s = 2.0 ** (e.astype(float) - 127)[:, None]
    err = np.abs(so.e4m3_decode(codes) * s - x)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()


def test_chain_is_causal_attention():
    g = torch.Generator().manual_seed(0)
    n, ctx, hq, hkv, d = 5, 9, 4, 2, 64
    q = torch.randn(1, ctx + n, hq, d, generator=g).bfloat16()
    k, v = (torch.randn(1, ctx + n, hkv, d, generator=g).bfloat16() for _ in range(2))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0])
    for kw in (dict(), dict(alibi_slopes=slopes), dict(window_left=4)):
        O, LSE = attention_forward(q, k, v, causal=True, **kw)
        o, lse, _, _ = so.tree_attention(q[0, ctx:].double().numpy(), k[0].double().numpy(),
                                         v[0].double().numpy(), ctx, **kw)
        assert np.allclose(o, O[0, ctx:]) and np.allclose(lse, LSE[0, :, ctx:].T)
    table = torch.randn(32, hq, generator=g)
    O, LSE = attention_forward(q, k, v, causal=True, t5_table=table, t5_bidirectional=False)
    o, lse, _, _ = so.tree_attention(q[0, ctx:].double().numpy(), k[0].double().numpy(),
                                     v[0].double().numpy(), ctx, t5_table=table.numpy())
    assert np.allclose(o, O[0, ctx:]) and np.allclose(lse, LSE[0, :, ctx:].T)


def test_tree_branches_are_their_paths():
    """A node's output equals that of its path decoded as a chain of its own."""
    rng = np.random.default_rng(7)
    ctx, hq, d = 6, 2, 8
    parents = [-1, 0, 0, 1, 2, 3]
    n = len(parents)
    mask = [0] * n
    for i in range(n):
        mask[i] = (mask[parents[i]] if i else 0) | (1 << i)
    q, k, v = rng.standard_normal((n, hq, d)), *rng.standard_normal((2, ctx + n, hq, d))
    o, lse, _, _ = so.tree_attention(q, k, v, ctx, mask, window_left=5)
    for leaf in range(n):
        path = [leaf]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        rows = list(range(ctx)) + [ctx + i for i in path]
        oc, lc, _, _ = so.tree_attention(q[path], k[rows], v[rows], ctx, window_left=5)
        assert np.allclose(oc[-1], o[leaf]) and np.allclose(lc[-1], lse[leaf])


def test_node_that_sees_nothing():
    o, lse, _, _ = so.tree_attention(np.ones((1, 1, 8)), np.ones((1, 1, 8)), np.ones((1, 1, 8)), 0, [0])
    assert (o == 0).all() and lse[0, 0] == -np.inf


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.25, 0.5, 0.125, 0.125], [0.25] * 4])
    # token 0: q <= p, always accepted; then p[1]'s cumulative sum
    assert so.verify(p, q, [0, 0], None, [0, 0.99], 0.5) == ([0, 1], 1, 2)
    # token 1: accepted iff u < 0.5; a tie is a rejection
    assert so.verify(p, q, [0, 1], None, [0, 0.49], 0.0)[1] == 1
    path, n, token = so.verify(p, q, [0, 1], None, [0, 0.5], 0.7)
    assert (path, n) == ([0, -1], 0)
    assert token == 2                     # left: max(p - q, 0) = [.25, 0, .125, 0]: cumulative 2/3, 1
    assert so.verify(p, q, [0, 1], None, [0, 0.5], 0.6)[2] == 0
    assert so.verify(p, p, [0, 3], None, [0, 0.5], 0.1)[2] == 0      # nothing left: p itself
    assert so.verify(p[:1], None, [0], None, [0], 0.99) == ([0], 0, 2)


@pytest.mark.parametrize("children", [1, 2, 3])
def test_verify_draws_from_the_target(children):
    """Over random drafts and numbers the first new token has the target's distribution: each of
    4 frequencies over 20000 draws lies within 5 standard deviations."""
    rng = np.random.default_rng(children)
    p, q = np.array([0.4, 0.3, 0.2, 0.1]), np.array([0.1, 0.2, 0.3, 0.4])
    n = 20000
    seen = np.zeros(4)
    target, draft = np.tile(p, (children + 1, 1)), np.tile(q, (children + 1, 1))
    for _ in range(n):
        x = np.concatenate([[0], rng.choice(4, children, p=q)])
        path, m, token = so.verify(target, draft, x, [-1] + [0] * children, rng.random(children + 1), rng.random())
        seen[x[path[1]] if m else token] += 1
    assert (np.abs(seen / n - p) < 5 * np.sqrt(p * (1 - p) / n)).all(), seen / n
