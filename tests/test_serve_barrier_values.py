"""The tree attention kernel's protocol where a warpgroup waits for a tile's values before its weights:
a new reference looks for value rows of zeros.  The model is test_serve_barrier_protocol.py's."""
import random

import pytest

from test_serve_barrier_protocol import SHAPES, explore, tree_protocol


def looks_at_values(role, g, R, NS, seed):
    """The softmax role with a wait for V of a tile after its scores are read, in some tiles."""
    rng = random.Random(seed * 7 + g)
    turns = 4 // max(R // 16, 1)
    it = g // max(R // 16, 1)
    for op in role:
        yield op
        if op[0] == "arrive" and op[1].startswith("s_free"):
            if rng.random() < 0.5:
                item = 2 * it + 1
                yield ("wait", f"full{item % NS}", (item // NS) & 1)
            it += turns


@pytest.mark.parametrize("NS", [4, 6, 12])
@pytest.mark.parametrize("R", [8, 16, 32, 64])
def test_a_wait_for_the_values_before_the_weights(R, NS):
    for k, pieces in enumerate(SHAPES):
        for seed in range(8):
            bars, roles = tree_protocol(pieces, R, NS, seed)
            for g in range(4):
                roles[f"wg{g}"] = looks_at_values(roles[f"wg{g}"], g, R, NS, seed)
            blocked = explore(bars, roles, seed * 31 + k)
            assert blocked is None, (pieces, seed, blocked)
