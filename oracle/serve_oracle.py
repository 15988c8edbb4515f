"""Float64 CPU definitions of the serving operators: rotary positions, the e4m3
cache rows, attention of drafted nodes over a cached context, and the
verification of drafted tokens.  Plain and slow; shares no code with the
library."""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------- rotary
def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=0,
                     beta_fast=32.0, beta_slow=1.0):
    """(frequencies [rot / 2], amplitude): RoFormer's, position-interpolated (linear), with the
    base raised (ntk), or blended by the turns a pair makes in the original length (yarn)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def pair_turning(turns):
        return rot * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

    lo = max(math.floor(pair_turning(beta_fast)), 0.0)
    hi = min(math.ceil(pair_turning(beta_slow)), rot - 1.0)
    if hi <= lo:
        hi = lo + 0.001
    ramp = np.clip((i - lo) / (hi - lo), 0.0, 1.0)
    return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def rope(x, positions, freqs, interleaved=False, inverse=False, amplitude=1.0):
    """x [..., L, H, d] float64 turned by positions [..., L] (see sdpa_rope)."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    t = np.asarray(positions, dtype=np.float64)[..., None, None] * freqs
    c, s = amplitude * np.cos(t), amplitude * np.sin(t) * (-1.0 if inverse else 1.0)
    one = np.arange(half) * 2 if interleaved else np.arange(half)
    two = one + 1 if interleaved else one + half
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one] = a * c - b * s
    y[..., two] = b * c + a * s
    return y


# --------------------------------------------------------------------- e4m3
def e4m3_values():
    """The value of every code 0 .. 127 (sign excluded); code 127 is NaN."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v + [np.nan])


def e4m3_round(x):
    """Codes (uint8) of float64 x rounded to nearest, ties to the even code; saturating at 448."""
    table = e4m3_values()[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - table[lo], table[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == table[hi], hi, code)
    code = code.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.where(np.signbit(x), 0xFF, 0x7F), code).astype(np.uint8)


def e4m3_decode(code):
    return np.where(code & 0x80, -1.0, 1.0) * e4m3_values()[code & 0x7F]


def e4m3_rows(x):
    """(codes, scale exponents) of rows x [..., d]: the smallest 2^k with max |x| <= 448 * 2^k."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    k = np.zeros(a.shape, dtype=int)
    for at in np.ndindex(a.shape):
        if a[at] > 0:
            e = math.frexp(a[at] / 448.0)[1]          # 2^(e-1) <= a / 448 < 2^e
            k[at] = e - 1 if 448.0 * 2.0 ** (e - 1) >= a[at] else e
            k[at] = min(max(k[at], -126), 127)
    return e4m3_round(x / 2.0 ** k[..., None]), (k + 127).astype(np.uint8)


# --------------------------------------------------------------------- tree
def t5_bucket(rel, num_buckets=32, max_distance=128, bidirectional=False):
    out = np.zeros(rel.shape, dtype=int)
    n = -rel
    if bidirectional:
        num_buckets //= 2
        out += (rel > 0) * num_buckets
        n = np.abs(rel)
    n = np.maximum(n, 0)
    exact = num_buckets // 2
    far = exact + (np.log(np.maximum(n, exact) / exact) / math.log(max_distance / exact)
                   * (num_buckets - exact)).astype(int)
    return out + np.where(n < exact, n, np.minimum(far, num_buckets - 1))


def tree_attention(q, k, v, ctx, mask=None, window_left=-1, alibi_slopes=None, t5_table=None,
                   t5_bidirectional=False, scale=None, t5_num_buckets=32, t5_max_distance=128):
    """One sequence's nodes q [n, Hq, d] over rows k, v [ctx + n, Hkv, d]; mask: n integers (bit
    j: sees node j), None: a chain.  Returns O, LSE [n, Hq], and per entry the sum of
    weight * |v| and the largest sum of |q k| of a row (for tolerances)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq, d = q.shape
    group = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    words = [(2 << i) - 1 for i in range(n)] if mask is None else [int(w) & (2 ** 64 - 1) for w in mask]
    sees = np.array([[bool((w >> j) & 1) for j in range(n)] for w in words]).reshape(n, n)
    pos = ctx + (sees & ~np.eye(n, dtype=bool)).sum(1)
    key_pos = np.concatenate([np.arange(ctx), pos])
    shown = np.concatenate([np.ones((n, ctx), dtype=bool), sees], 1)
    rel = key_pos[None, :] - pos[:, None]
    if window_left >= 0:
        shown &= rel >= -window_left
    o, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    spread, size = np.zeros((n, hq, d)), np.zeros((n, hq))
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        for i in range(n):
            on = shown[i]
            if not on.any():
                continue
            s = scale * (kh[on] @ q[i, h])
            if alibi_slopes is not None:
                s = s - float(alibi_slopes[h]) * np.abs(rel[i, on])
            if t5_table is not None:
                s = s + np.asarray(t5_table, dtype=np.float64)[
                    t5_bucket(rel[i, on], t5_num_buckets, t5_max_distance, t5_bidirectional), h]
            top = s.max()
            p = np.exp(s - top)
            lse[i, h] = top + math.log(p.sum())
            p = p / p.sum()
            o[i, h] = p @ vh[on]
            spread[i, h] = p @ np.abs(vh[on])
            size[i, h] = (np.abs(kh[on]) @ np.abs(q[i, h])).max() * abs(scale)
    return o, lse, spread, size


# ------------------------------------------------------------------- verify
def verify(target, draft, tokens, parents, u_accept, u_sample):
    """One sequence (see sdpa_spec_verify): (path, accepted, next token)."""
    target = np.asarray(target, dtype=np.float64)
    n, vocab = target.shape
    parents = list(range(-1, n - 1)) if parents is None else [int(p) for p in parents]
    at, path = 0, [0]
    w = target[0].copy()
    total = 1.0
    while True:
        kids = [c for c in range(1, n) if 0 <= parents[c] < c and parents[c] == at]
        taken = None
        for c in kids:
            x = int(tokens[c])
            q = np.asarray(draft[at], dtype=np.float64)
            if 0 <= x < vocab and float(u_accept[c]) * q[x] < w[x]:
                taken = c
                break
            w = np.maximum(w - q, 0.0)
            total = math.fsum(w)
            if total > 0:
                w = w / total
        if taken is None:
            break
        at, w = taken, target[taken].copy()
        path.append(taken)
    if not w.any():
        w = target[at]
    upto = np.cumsum(w)
    over = np.nonzero((upto > float(u_sample) * upto[-1]) & (w > 0))[0]
    some = np.nonzero(w > 0)[0]
    token = int(over[0]) if len(over) else (int(some[-1]) if len(some) else 0)
    return path + [-1] * (n - len(path)), len(path) - 1, token
