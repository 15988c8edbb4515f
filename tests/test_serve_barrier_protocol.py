"""The tree attention kernel's barrier protocol, model-checked on the CPU.

Its roles (TMA producer, query warp, the two MMA issuers, four softmax
warpgroups) are restated as the mbarrier and named-barrier operations they
perform, with what they read and write in between: ring slots, query operands,
scores, weights, accumulators and row sums.  Random interleavings are explored,
asynchronous arrivals (a copy landing, MMAs done) at random times.  A schedule
in which every unfinished role waits is a deadlock; a read that does not find
what it is for, or a write over something still to be read, is a missing wait.
The sequences mirror csrc/serve/tree_fwd.cuh.
"""
import random

import pytest

from test_barrier_protocols import Bar


def explore(bars, roles, seed, max_steps=400000):
    """One random interleaving; None, or the blocked operations of a deadlock."""
    rng = random.Random(seed)
    B = {n: Bar(c) for n, c in bars.items()}
    cur = {n: next(g, None) for n, g in roles.items()}
    flying = []
    slow = rng.choice(list(roles))           # a role that is held back
    for _ in range(max_steps):
        ready = [n for n, op in cur.items() if op is not None
                 and not (op[0] == "wait" and not B[op[1]].parity_done(op[2]))
                 and not (op[0] == "phase_ge" and B[op[1]].phase < op[2])]
        if flying and (not ready or rng.random() < 0.3):
            bar, landed = flying.pop(rng.randrange(len(flying)))
            landed()
            B[bar].arrive()
            continue
        if not ready:
            return None if all(op is None for op in cur.values()) else {n: op for n, op in cur.items() if op}
        n = rng.choice([r for r in ready if r != slow] or ready) if rng.random() < 0.95 else rng.choice(ready)
        op, nxt = cur[n], None
        if op[0] == "arrive":
            for _ in range(op[2] if len(op) > 2 else 1):
                B[op[1]].arrive()
        elif op[0] == "async":
            flying.append((op[1], op[2]))
        elif op[0] == "sync":
            nxt = ("phase_ge", op[1], B[op[1]].phase + 1)
            B[op[1]].arrive()
        cur[n] = nxt or next(roles[n], None)
    raise AssertionError("schedule did not finish")


def tree_protocol(pieces, R, NS, seed, drop=None):
    """pieces: tiles of each; R: query rows of a product; NS: ring slots.  drop: a wait left out
    (to show that the model sees it)."""
    rng = random.Random(seed)
    RG = max(R // 16, 1)
    TN = 4 // RG
    NB = max(TN, 2)
    ids = [(u, i) for u, nt in enumerate(pieces) for i in range(nt)]
    bars = {"all": 4}
    bars.update({f"full{s}": 1 for s in range(NS)} | {f"empty{s}": 1 for s in range(NS)})
    bars.update({f"s_full{x}": 1 for x in range(NB)} | {f"s_free{x}": RG for x in range(NB)})
    bars.update({f"p_full{x}": RG for x in range(NB)} | {f"pv_done{x}": 1 for x in range(NB)})
    bars.update({f"q_full{x}": 4 for x in range(2)} | {f"q_free{x}": 4 for x in range(2)})
    bars.update({f"turn{t}": RG for t in range(TN)})
    slot, S, landed_pv = {}, {}, set()
    Q, P, O, sums = {0: {}, 1: {}}, {}, {}, {}
    reading = {}                              # (u, wg): results of piece u not read yet

    def wait(name, phase, kind=None):
        if kind is None or kind != drop:
            yield ("wait", name, phase & 1)

    def nothing():
        pass

    def producer():
        for item in range(2 * len(ids)):
            s = item % NS
            if item >= NS:
                yield from wait(f"empty{s}", item // NS - 1, "empty")
                assert slot[s][1] == "used", "a slot is filled while it is in use"
            slot[s] = [item, "filling"]

            def landed(s=s):
                slot[s][1] = "full"
            yield ("async", f"full{s}", landed)

    def query():
        for u in range(1, len(pieces)):
            x = u & 1
            if u >= 2:
                yield from wait(f"q_free{x}", (u >> 1) - 1, "q_free")
                assert all((u - 2, g) not in reading for g in range(4)), "rows of a piece still being read"
            Q[x] = dict.fromkeys(range(4), u)
            yield ("arrive", f"q_full{x}", 4)

    def s_issuer():
        it = 0
        for u, nt in enumerate(pieces):
            yield from wait(f"q_full{u & 1}", u >> 1, "q_full")
            for _ in range(nt):
                x, item = it % NB, 2 * it
                yield from wait(f"full{item % NS}", item // NS)
                if it >= NB:
                    yield from wait(f"s_free{x}", it // NB - 1, "s_free")
                    assert len(S[x][1]) == RG, "scores overwritten before they were read"
                assert slot[item % NS] == [item, "full"] and all(Q[u & 1].get(g) == u for g in range(4))
                S[x] = [None, set()]

                def done(x=x, it=it, s=item % NS, u=u):
                    S[x][0] = it
                    slot[s][1] = "used"
                    assert all(Q[u & 1].get(g) == u for g in range(4)), "queries replaced under the product"
                yield ("async", f"s_full{x}", done)
                # (one commit after the other, of the same MMAs)
                while S[x][0] != it:
                    yield ("wait", "never_low", 1)
                yield ("async", f"empty{item % NS}", nothing)
                it += 1

    def pv_issuer():
        it = 0
        for u, nt in enumerate(pieces):
            for i in range(nt):
                x, item = it % NB, 2 * it + 1
                yield from wait(f"full{item % NS}", item // NS)
                yield from wait(f"p_full{x}", it // NB, "p_full")
                assert slot[item % NS] == [item, "full"] and P[x] == dict.fromkeys(range(RG), it)
                o = ((u & 1), it % TN)
                if i < TN:
                    assert all((u - 2, g) not in reading for g in range(4)), "an O overwritten before it was read"
                    O[o] = [u, 0]

                def done(it=it, o=o, s=item % NS, x=x):
                    O[o][1] += 1
                    assert P[x] == dict.fromkeys(range(RG), it), "weights replaced under the product"
                    landed_pv.add(it)
                    slot[s][1] = "used"
                yield ("async", f"pv_done{x}", done)
                while it not in landed_pv:
                    yield ("wait", "never_low", 1)
                yield ("async", f"empty{item % NS}", nothing)
                it += 1

    def softmax(g):
        turn, row = g // RG, g % RG
        it = 0

        def values_done(j, kind=None):
            yield from wait(f"pv_done{j % NB}", j // NB, kind)
            assert j in landed_pv, "O or weights touched before P V was done"
        for u, nt in enumerate(pieces):
            reading[(u, g)] = True
            if u == 0:
                Q[0][g] = 0
                yield ("arrive", "q_full0")
                yield ("sync", "all")
            else:
                yield from wait(f"q_full{u & 1}", u >> 1)
            assert Q[u & 1].get(g) == u
            fresh, last = True, None
            for i in range(nt):
                if it % TN == turn:
                    x = it % NB
                    yield from wait(f"s_full{x}", it // NB)
                    assert S[x][0] == it
                    S[x][1].add(row)
                    yield ("arrive", f"s_free{x}")
                    if it >= NB:
                        yield from values_done(it - NB, "weights")
                    if (fresh or rng.random() < 0.3) and not fresh:
                        if TN < NB:
                            yield from values_done(it - TN)
                        assert it - TN in landed_pv, "O rescaled under a product"
                    P.setdefault(x, {})[row] = it
                    mend = False
                    if masked[it]:
                        yield from wait(f"full{(2 * it + 1) % NS}", (2 * it + 1) // NS)
                        assert slot[(2 * it + 1) % NS] == [2 * it + 1, "full"]
                        yield ("sync", f"turn{turn}")
                        mend = mended[it]
                    yield ("arrive", f"p_full{x}")
                    fresh, last = False, it
                    if mend:
                        yield from values_done(it)
                it += 1
            if not fresh:
                yield from values_done(last)
            assert sums.get((u & 1, g), u - 2) == u - 2, "sums replaced"
            if u >= 2:
                assert all((u - 2, h) not in reading for h in range(4)), "sums replaced before they were read"
            sums[(u & 1, g)] = u
            if TN > 1:
                yield ("sync", "all")
            writer = R > 16 or ((g + u) & 3 == 0 if R == 8 else (g ^ ((u & 1) << 1)) < 2)
            if writer:
                for t in range(min(nt, TN)):
                    k = (it - nt + t) % TN
                    mine = [j for j in range(it - nt, it) if j % TN == k]
                    assert O[(u & 1, k)] == [u, len(mine)], "O read too early or too late"
                if TN > 1:
                    assert all(sums[(u & 1, h)] == u for h in range(4))
            del reading[(u, g)]
            yield ("arrive", f"q_free{u & 1}")

    masked = [rng.random() < 0.4 for _ in ids]
    mended = [rng.random() < 0.5 for _ in ids]
    bars["never_low"] = 1                    # phase 0: a wait for parity 1 passes (a pause)
    roles = {"producer": producer(), "query": query(), "s": s_issuer(), "pv": pv_issuer()}
    roles.update({f"wg{g}": softmax(g) for g in range(4)})
    return bars, roles


SHAPES = [[1], [2, 1, 1, 3], [1] * 9, [5, 4], [13], [3, 1, 7, 2, 6], [4, 1, 1, 1, 8]]


@pytest.mark.parametrize("NS", [4, 6, 12])
@pytest.mark.parametrize("R", [8, 16, 32, 64])
def test_tree_kernel_protocol(R, NS):
    for k, pieces in enumerate(SHAPES):
        for seed in range(12):
            blocked = explore(*tree_protocol(pieces, R, NS, seed), seed * 31 + k)
            assert blocked is None, (pieces, seed, blocked)


@pytest.mark.parametrize("drop", ["empty", "q_free", "q_full", "s_free", "p_full", "weights"])
def test_the_model_sees_a_missing_wait(drop):
    """Leaving a wait out of the model (not of the kernel) is noticed (scores that run ahead only
    where the ring has more slots than there are buffers of scores)."""
    for R in (8, 16, 32, 64):
        for seed in range(400):
            try:
                explore(*tree_protocol([3, 1, 7, 2, 6], R, 4 if seed & 1 else 12, seed, drop), seed)
            except (AssertionError, KeyError):
                break
        else:
            raise AssertionError(f"unnoticed at {R} rows")
