"""The serving operators over a paged key/value cache, as measurable cases.

Five entry points that a program calls around attention when it generates text
with drafted tokens:

  rope     rotary positions of Q and K, forward and gradient
  append   K and V rows written into a paged cache (bf16, or e4m3 with one
           power-of-two scale per row and head)
  gather   the cache read back as packed bf16 K and V
  tree     attention of each sequence's drafted nodes over its cached context
           and over the nodes that the tree shows them (one node: plain decoding)
  verify   acceptance of drafted tokens and the next token, by rejection sampling
           with given random numbers

With ``own`` false, ``run`` computes each operator's plain form in elementary
torch operations; with ``own`` true it makes the library's calls.  ``exact``
computes the definition in float64, sequence by sequence.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 8 sequences far into a long context: latency
        dict(name="rope_step_b8", op="rope", B=8, L=1, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             inverse=False, factor=4.0, far=131072),
        # the gradient of the rotation over a training batch (B = 4, L = 4096, 32 query and 8 KV heads)
        dict(name="rope_grad_4k", op="rope", B=4, L=4096, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             inverse=True, factor=1.0, far=0),
        # the rows of one decoding step into an 8-bit cache
        dict(name="append_step_e4m3", op="append", T=64, Hkv=8, d=128, page=64, kv="e4m3"),
        # a prompt batch of 32768 tokens into an 8-bit cache
        dict(name="append_prompt_e4m3", op="append", T=32768, Hkv=8, d=128, page=64, kv="e4m3"),
        # one short 64-wide bf16 context read back for its next chunk
        dict(name="gather_bf16_d64", op="gather", B=1, ctx=1500, ragged=False, Hkv=12, d=64, page=16, kv="bf16"),
        # ragged 8-bit contexts read back
        dict(name="gather_e4m3_ragged", op="gather", B=16, ctx=8192, ragged=True, Hkv=8, d=128, page=64, kv="e4m3"),
        # single-token decoding of one sequence: latency
        dict(name="decode_b1_bf16", op="tree", B=1, ctx=4095, ragged=False, nodes=1, chain=True, Hq=32, Hkv=8, d=128,
             page=64, kv="bf16", window=4096, bias="none"),
        # single-token decoding of a ragged batch over an 8-bit cache
        dict(name="decode_b32_e4m3_16k", op="tree", B=32, ctx=16384, ragged=True, nodes=1, chain=True, Hq=32, Hkv=8,
             d=128, page=64, kv="e4m3", window=-1, bias="none"),
        # trees of up to 16 drafted nodes over long bf16 contexts
        dict(name="tree16_b16_bf16_8k", op="tree", B=16, ctx=8191, ragged=True, nodes=16, chain=False, Hq=32, Hkv=8,
             d=128, page=64, kv="bf16", window=-1, bias="none"),
        # trees of 64 nodes with a relative-position bias, every head its own keys
        dict(name="tree64_t5_d64", op="tree", B=8, ctx=2000, ragged=True, nodes=64, chain=False, Hq=12, Hkv=12,
             d=64, page=32, kv="bf16", window=-1, bias="t5"),
        # verification of one drafted chain: latency
        dict(name="verify_b1_chain5", op="verify", B=1, nodes=6, chain=True, V=32000),
        # verification of 16-node trees for 32 sequences
        dict(name="verify_b32_tree16", op="verify", B=32, nodes=16, chain=False, V=32000),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "gather", "tree", "tree", "tree", "verify"])
    d = rng.choice([64, 128])
    hq, hkv = rng.choice([(32, 32), (32, 8), (32, 1), (12, 12), (16, 4), (8, 2)])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "e4m3"])
    if op == "rope":
        B = rng.choice([1, 2, 5, 16])
        return dict(op="rope", B=B, L=log_int(1, 16384 // B), Hq=hq, Hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, d - 6]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, factor=rng.choice([1.0, 2.0, 8.0]), far=rng.choice([0, 5000, 1000000]))
    if op == "append":
        return dict(op="append", T=log_int(1, 32768), Hkv=hkv if hkv < 32 else 8, d=d, page=page, kv=kv)
    row = 2 * hkv * d * (2 if kv == "bf16" else 1)              # bytes of one cached position
    B = log_int(1, 32)
    if op == "gather":
        return dict(op="gather", B=B, ctx=log_int(1, max(1, min(32768, 4 * 10**8 // B // (row + 4 * hkv * d)))),
                    ragged=rng.random() < 0.7, Hkv=hkv, d=d, page=page, kv=kv)
    if op == "tree":
        nodes = rng.choice([1, 1, 2, 4, 7, 16, 33, 64])
        most = min(32768, 6 * 10**8 // B // row, 12 * 10**9 // B // (4 * d * hq * nodes))
        return dict(op="tree", B=B, ctx=log_int(1, max(1, most)), ragged=rng.random() < 0.7, nodes=nodes,
                    chain=rng.random() < 0.3, Hq=hq, Hkv=hkv, d=d, page=page, kv=kv,
                    window=rng.choice([-1, -1, 100, 4096]), bias=rng.choice(["none", "none", "alibi", "t5"]))
    nodes = rng.choice([1, 2, 5, 8, 16, 33])
    return dict(op="verify", B=log_int(1, 512 // nodes), nodes=nodes, chain=rng.random() < 0.5, V=log_int(500, 32000))


def lengths(case):
    """The sequences' context lengths and node counts: a property of the case, not of the seed."""
    r = random.Random("%d %d" % (case["B"], case["ctx"]))
    lens, counts = [case["ctx"]], [case.get("nodes", 1)]
    for _ in range(case["B"] - 1):
        lens.append(r.randint(max(1, case["ctx"] // 4), case["ctx"]) if case["ragged"] else case["ctx"])
        counts.append(r.randint(1, counts[0]) if case["ragged"] else counts[0])
    return lens, counts


# ------------------------------------------------------------------ inputs
def power_of_two_above(amax):
    """Biased exponent of the smallest power of two s with amax <= 448 s (127 where amax is 0)."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    k = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, (k + 127).clamp(1, 254), torch.full_like(e, 127)).to(torch.uint8)


def as_scale(e8):
    return torch.exp2(e8.float() - 127.0)


def quantised(x):
    e8 = power_of_two_above(x.float().abs().amax(-1))
    return (x.float() / as_scale(e8)[..., None]).to(torch.float8_e4m3fn), e8


def make_cache(case, g, num_pages):
    """A cache whose every row holds keys and values (rows past a sequence's end are what an earlier one left)."""
    shape = (num_pages, case["Hkv"], case["page"], case["d"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    if case["kv"] == "bf16":
        return dict(k_cache=k, v_cache=v, k_scale=None, v_scale=None)
    k, ks = quantised(k)
    v, vs = quantised(v)
    return dict(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs)


def make_tree(parents):
    """Bit m of row n: node n sees node m (its ancestors and itself)."""
    B, N = parents.shape
    mask = torch.zeros(B, N, dtype=torch.int64, device=parents.device)
    mask[:, 0] = 1
    for n in range(1, N):
        bit = torch.tensor(1 << n if n < 63 else -(1 << 63), dtype=torch.int64, device=parents.device)
        mask[:, n] = mask.gather(1, parents[:, n:n + 1])[:, 0] | bit
    return mask


def random_parents(B, N, chain, g):
    parents = torch.arange(-1, N - 1, device="cuda").expand(B, N).clone()
    if not chain and N > 1:
        top = torch.arange(N, device="cuda").float()
        # a node's parent is one of the earlier half, so that trees branch and grow deep
        parents = (torch.rand(B, N, generator=g, device="cuda") * (top + 1) / 2).long()
        parents[:, 0] = -1
    return parents


def frequencies(rot, factor):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot) / factor


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    if op == "rope":
        B, L = case["B"], case["L"]
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        return dict(op=op, q=randn(B, L, case["Hq"], case["d"]), k=randn(B, L, case["Hkv"], case["d"]),
                    freqs=frequencies(case["rot"], case["factor"]), interleaved=case["interleaved"],
                    inverse=case["inverse"], amplitude=1.0 + 0.1 * math.log(case["factor"]),
                    positions=(start + torch.arange(L, device="cuda")).int())
    if op == "append":
        T, page = case["T"], case["page"]
        num_pages = T // page + 2
        pad = T // 32                               # padded rows of the batch have no slot
        pages = torch.randperm(num_pages, generator=g, device="cuda")
        row = torch.arange(T, device="cuda")
        slots = pages[row // page] * page + row % page
        slots[T - pad:] = -1
        cache = make_cache(case, g, num_pages)
        # keys' channels differ in size, as learned projections make them
        size = torch.exp(randn(case["Hkv"], case["d"], dtype=torch.float32))
        return dict(op=op, k=(randn(T, case["Hkv"], case["d"]) * size).bfloat16(),
                    v=randn(T, case["Hkv"], case["d"]), slots=slots, **cache)
    if op in ("gather", "tree"):
        B, page = case["B"], case["page"]
        lens, counts = lengths(case)
        width = (max(a + b for a, b in zip(lens, counts)) + page - 1) // page
        num_pages = B * width + 3
        table = torch.randperm(num_pages, generator=g, device="cuda")[:B * width].view(B, width).int()
        cache = make_cache(case, g, num_pages)
        if op == "gather":
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            return dict(op=op, table=table, cu=torch.tensor(cu, device="cuda", dtype=torch.int32), total=cu[-1], **cache)
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        q = randn(cu[-1], case["Hq"], case["d"])
        N = case["nodes"]
        parents = random_parents(B, N, case["chain"], g)
        keep = torch.arange(N, device="cuda") < torch.tensor(counts, device="cuda")[:, None]
        mask = None if case["chain"] else make_tree(parents)[keep]
        bias = {}
        if case["bias"] == "alibi":
            h = torch.arange(1, case["Hq"] + 1, device="cuda")
            bias["alibi_slopes"] = torch.exp2(-8.0 * h / case["Hq"]).float()
        elif case["bias"] == "t5":
            bias["t5_table"] = randn(32, case["Hq"], dtype=torch.float32)
        return dict(op=op, q=q, table=table, ctx=torch.tensor(lens, device="cuda", dtype=torch.int32),
                    cu=torch.tensor(cu, device="cuda", dtype=torch.int32), max_nodes=N, tree_mask=mask,
                    window=case["window"], bias=bias, scale=1.0 / math.sqrt(case["d"]), **cache)
    B, N, V = case["B"], case["nodes"], case["V"]
    logits = 3.0 * randn(B, N, V, dtype=torch.float32)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + randn(B, N, V, dtype=torch.float32), -1)
    parents = random_parents(B, N, case["chain"], g)
    rows = draft.gather(1, parents.clamp(min=0)[:, :, None].expand(B, N, V))
    tokens = torch.multinomial(rows.view(B * N, V), 1, generator=g).view(B, N).int()
    return dict(op=op, target=target, draft=draft, tokens=tokens, parents=parents.int(),
                u_accept=torch.rand(B, N, generator=g, device="cuda"), u_sample=torch.rand(B, generator=g, device="cuda"))


# --------------------------------------------------------------------- run
def run(state):
    if own:
        return run_own(state)
    return {"rope": plain_rope, "append": plain_append, "gather": plain_gather, "tree": plain_tree,
            "verify": plain_verify}[state["op"]](state)


def run_own(s):
    import scaled_dot_product_bwd_b200 as lib

    cache = {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s}
    if s["op"] == "rope":
        return lib.sdpa_rope(s["q"], s["k"], s["freqs"], s["positions"], interleaved=s["interleaved"],
                             inverse=s["inverse"], amplitude=s["amplitude"])
    if s["op"] == "append":
        lib.sdpa_cache_append(s["k"], s["v"], s["slots"], **cache)
        return cache
    if s["op"] == "gather":
        return lib.sdpa_cache_gather(page_table=s["table"], cu_seqlens=s["cu"], total=s["total"], **cache)
    if s["op"] == "tree":
        return lib.sdpa_tree_fwd(s["q"], page_table=s["table"], ctx_lens=s["ctx"], cu_nodes=s["cu"],
                                 max_nodes=s["max_nodes"], tree_mask=s["tree_mask"], window_left=s["window"],
                                 scale=s["scale"], t5_bidirectional=False, **s["bias"], **cache)
    return lib.sdpa_spec_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["u_accept"], s["u_sample"])


def plain_rope(s):
    angle = s["positions"].double()[..., None] * s["freqs"]
    cos = (s["amplitude"] * torch.cos(angle)).float()[:, :, None]
    sin = (s["amplitude"] * torch.sin(angle)).float()[:, :, None]
    sin = -sin if s["inverse"] else sin
    half = s["freqs"].numel()

    def rotate(x):
        y, rest = x[..., :2 * half].float(), x[..., 2 * half:]
        a, b = (y[..., 0::2], y[..., 1::2]) if s["interleaved"] else (y[..., :half], y[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((y.to(x.dtype), rest), -1)

    return rotate(s["q"]), rotate(s["k"])


def plain_append(s):
    kc, vc, ks, vs = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    page = kc.shape[2]
    has = s["slots"] >= 0
    slots = s["slots"][has]
    where = (slots // page, slice(None), slots % page)
    if ks is None:
        kc[where], vc[where] = s["k"][has], s["v"][has]
    else:
        for x, cache, scale in ((s["k"], kc, ks), (s["v"], vc, vs)):
            x8, e8 = quantised(x[has])
            cache.view(torch.uint8)[where] = x8.view(torch.uint8)
            scale[where] = e8
    return dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)


def cached(cache, scale, table):
    """fp32 rows [B, Hkv, positions, d] of the tables' pages."""
    B, W = table.shape
    _, H, page, d = cache.shape
    x = cache[table.long()].float()
    if scale is not None:
        x = x * as_scale(scale[table.long()])[..., None]
    return x.transpose(1, 2).reshape(B, H, W * page, d)


def plain_gather(s):
    cu = s["cu"].long()
    row = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[b]
    page = s["k_cache"].shape[2]
    at = (s["table"].long()[b, pos // page], slice(None), pos % page)
    out = []
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        if scale is None:
            out.append(cache[at])
        else:
            x = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn)
            out.append((x.float() * as_scale(scale[at])[..., None]).bfloat16())
    return tuple(out)


def t5_bucket(distance, buckets=32, max_distance=128):
    """Unidirectional T5 bucket of key positions `distance` before the query."""
    n = distance.clamp(min=0)
    exact_up_to = buckets // 2
    far = torch.log(n.clamp(min=1).double() / exact_up_to) / math.log(max_distance / exact_up_to) * (buckets - exact_up_to)
    return torch.where(n < exact_up_to, n, (exact_up_to + far.long()).clamp(max=buckets - 1))


def plain_tree(s):
    q, ctx, cu, N = s["q"], s["ctx"].long(), s["cu"].long(), s["max_nodes"]
    T, Hq, d = q.shape
    k = cached(s["k_cache"], s["k_scale"], s["table"])
    v = cached(s["v_cache"], s["v_scale"], s["table"])
    B, Hkv, S, _ = k.shape
    node = torch.arange(N, device="cuda")
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + node).clamp(max=T - 1)                            # [B, N]
    sees = s["tree_mask"][row] if s["tree_mask"] is not None else ((2 << node) - 1).expand(B, N)
    bits = (sees[..., None] >> node) & 1                                    # [B, N, N]
    depth = (bits * (node[:, None] != node)).sum(-1)
    key = torch.arange(S, device="cuda").expand(B, S)
    m = key - ctx[:, None]
    is_node = (m >= 0) & (m < count[:, None])
    m = m.clamp(0, N - 1)
    key_pos = torch.where(is_node, ctx[:, None] + depth.gather(1, m), key)    # [B, S]
    before = (ctx[:, None] + depth)[:, :, None] - key_pos[:, None]            # [B, N, S]
    shown = bits.gather(2, m[:, None].expand(B, N, S)) > 0
    shown = (key < ctx[:, None])[:, None] | (is_node[:, None] & shown)
    if s["window"] >= 0:
        shown = shown & (before <= s["window"])
    qf = q.float()[row].view(B, N, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    score = (s["scale"] * (qf @ k.transpose(-1, -2))).view(B, Hq, N, S)
    if "alibi_slopes" in s["bias"]:
        score = score - s["bias"]["alibi_slopes"][:, None, None] * before.abs().float()[:, None]
    if "t5_table" in s["bias"]:
        score = score + s["bias"]["t5_table"][t5_bucket(before)].permute(0, 3, 1, 2)
    score = torch.where(shown[:, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, S) @ v).view(B, Hq, N, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    n = t - cu[b]
    return o[b, :, n].to(q.dtype), lse[b, :, n].t().contiguous()


def plain_verify(s):
    target, draft, parents = s["target"], s["draft"], s["parents"].long()
    B, N, V = target.shape
    tokens, u = s["tokens"].long(), s["u_accept"].double()
    every = torch.arange(B, device="cuda")
    at = torch.zeros(B, dtype=torch.long, device="cuda")
    weight = target[:, 0].double()                 # what is left of the current node's distribution
    accepted = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.full((B, N + 1), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    # nodes come after their parents, so one walk over them in order visits every child of an accepted node
    for n in range(1, N):
        q = draft[every, at].double()
        x = tokens[:, n:n + 1]
        tried = parents[:, n] == at
        ok = tried & (u[:, n] * q.gather(1, x)[:, 0] < weight.gather(1, x)[:, 0])
        left = (weight - q).clamp(min=0)
        left = left / left.sum(-1, keepdim=True).clamp(min=1e-300)
        weight = torch.where(ok[:, None], target[:, n].double(), torch.where(tried[:, None], left, weight))
        at = torch.where(ok, n, at)
        accepted = accepted + ok
        path.scatter_(1, torch.where(ok, accepted, N)[:, None], at[:, None])
    path[:, N] = -1
    weight = torch.where((weight > 0).any(-1, keepdim=True), weight, target[every, at].double())
    upto = weight.cumsum(-1)
    index = torch.arange(V, device="cuda")
    last = torch.where(weight > 0, index, 0).amax(-1)
    token = (upto <= s["u_sample"].double()[:, None] * upto[:, -1:]).sum(-1)
    return path[:, :N].int(), accepted.int(), torch.minimum(token, last).int()


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["B"] * case["L"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 4 * n + 4 * case["B"] * case["L"], "flops": 6 * n * case["rot"] / case["d"] / 2}
    cell = 2 if case.get("kv") == "bf16" else 1
    row = 2 * case.get("Hkv", 0) * (case.get("d", 0) * cell + (cell == 1))   # cached bytes of one position
    if op == "append":
        kept = case["T"] - case["T"] // 32
        return {"bytes": kept * (4 * case["Hkv"] * case["d"] + row) + 8 * case["T"], "flops": 0}
    if op == "gather":
        return {"bytes": sum(lengths(case)[0]) * (row + 4 * case["Hkv"] * case["d"]), "flops": 0}
    if op == "tree":
        lens, counts = lengths(case)
        w = case["window"]
        seen = [n if w < 0 else min(n, w) for n in lens]
        qo = sum(counts) * case["Hq"] * (4 * case["d"] + 4)
        flops = sum(4 * case["d"] * case["Hq"] * c * (n + (c + 1) / 2) for n, c in zip(seen, counts))
        return {"bytes": sum(n + c for n, c in zip(seen, counts)) * row + qo, "flops": flops}
    # one row of both distributions, where a sequence's walk ends, and two values for each node
    return {"bytes": case["B"] * (8 * case["V"] + 24 * case["nodes"]), "flops": 3 * case["B"] * case["V"]}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "append": exact_append, "gather": exact_gather, "tree": exact_tree,
            "verify": lambda s: None}[s["op"]](s)


def exact_rope(s):
    out = []
    half = s["freqs"].numel()
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    turn = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None, None] * s["freqs"])
    if s["inverse"]:
        turn = turn.conj()
    for x in (s["q"], s["k"]):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def exact_append(s):
    out = {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    page = s["k_cache"].shape[2]
    slots = s["slots"][s["slots"] >= 0]
    n = slots.numel()
    flat = slots // page * page + slots % page
    for name in ("k", "v"):
        x = s[name][:n].double()
        rows = out[name + "_cache"].transpose(1, 2).flatten(0, 1).clone()       # [positions, Hkv, d]
        if out[name + "_scale"] is None:
            rows[flat] = x.bfloat16()
        else:
            big = x.abs().amax(-1)
            e = torch.ceil(torch.log2(big.clamp(min=1e-300) / E4M3_MAX) - 1e-12)
            e = torch.where(big > 0, e, torch.zeros_like(e))
            rows.view(torch.uint8)[flat] = (x * torch.exp2(-e)[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
            scale = out[name + "_scale"].transpose(1, 2).flatten(0, 1).clone()
            scale[flat] = (e + 127).to(torch.uint8)
            out[name + "_scale"] = scale.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
        out[name + "_cache"] = rows.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
    return out


def exact_rows(s, name, b, n):
    """Float64 rows [Hkv, n, d] of the first n positions of sequence b."""
    page = s["k_cache"].shape[2]
    ids = s["table"][b, :(n + page - 1) // page].long()
    x = s[name + "_cache"][ids].double()
    if s[name + "_scale"] is not None:
        x = x * 2.0 ** (s[name + "_scale"][ids].double() - 127)[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def exact_gather(s):
    cu = s["cu"].tolist()
    return tuple(torch.cat([exact_rows(s, name, b, hi - lo).transpose(0, 1) for b, (lo, hi) in enumerate(zip(cu, cu[1:]))])
                 for name in ("k", "v"))


def exact_tree(s):
    T, Hq, d = s["q"].shape
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    cu, lens = s["cu"].tolist(), s["ctx"].tolist()
    for b, ctx in enumerate(lens):
        lo, n = cu[b], cu[b + 1] - cu[b]
        words = [(2 << i) - 1 for i in range(n)] if s["tree_mask"] is None else s["tree_mask"][lo:lo + n].tolist()
        see = torch.tensor([[(w >> j) & 1 for j in range(n)] for w in words], device="cuda", dtype=torch.bool)
        pos = ctx + (see & ~torch.eye(n, device="cuda", dtype=torch.bool)).sum(1)
        key_pos = torch.cat((torch.arange(ctx, device="cuda"), pos))
        see = torch.cat((torch.ones(n, ctx, device="cuda", dtype=torch.bool), see), 1)
        gap = pos[:, None] - key_pos
        if s["window"] >= 0:
            see &= gap <= s["window"]
        k, v = exact_rows(s, "k", b, ctx + n), exact_rows(s, "v", b, ctx + n)
        group = Hq // k.shape[0]
        for h in range(Hq):
            a = s["q"][lo:lo + n, h].double() @ k[h // group].t() * s["scale"]
            if "alibi_slopes" in s["bias"]:
                a = a - s["bias"]["alibi_slopes"][h].double() * gap.abs()
            if "t5_table" in s["bias"]:
                near = gap.clamp(min=0)
                far = 16 + (torch.log(near.clamp(min=16).double() / 16) / math.log(8.0) * 16).floor().long()
                a = a + s["bias"]["t5_table"][:, h].double()[torch.where(near < 16, near, far.clamp(max=31))]
            a = a.masked_fill(~see, -math.inf)
            lse[h, lo:lo + n] = torch.logsumexp(a, 1)
            o[lo:lo + n, h] = torch.softmax(a, 1) @ v[h // group]
    return o, lse
