"""The barriers between the two issuing warps of rf_tree_attention's kernel (two row tiles), as a
model on the CPU: every order in which the two warps can run has to end.

An mbarrier is its number of completed phases; a wait for parity p passes when the phase of that
parity is the last one that completed, so a barrier that runs two phases ahead of its waiter
holds the waiter up."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ridge_map_kv_gb300", "csrc", "attn.cu")


def _programs(tiles, barriers):
    """('wait' | 'arrive', barrier, parity) of the warps that issue stream 0's and stream 1's products, for one
    segment of `tiles` tiles that all have to be cleaned."""
    first, second = [], []
    turn = [1, 0]                                   # parities that the warps wait for next

    def my_turn(w, prog):
        prog.append(("wait", f"turn{w}", turn[w]))
        turn[w] ^= 1

    my_turn(0, first)
    first.append(("arrive", "turn1", 0))
    my_turn(1, second)
    second.append(("arrive", "turn0", 0))
    for i in range(tiles):
        clean = f"clean{i % barriers}"
        first.append(("arrive", clean, 0))
        my_turn(0, first)
        first.append(("arrive", "turn1", 0))
        second.append(("wait", clean, (i // barriers) & 1))
        my_turn(1, second)
        second.append(("arrive", "turn0", 0))
    return first, second


def _orders_that_hang(tiles, barriers):
    progs = _programs(tiles, barriers)
    todo, seen, stuck = [((0, 0), ())], set(), 0
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, phases = state
        phases = dict(phases)
        moved = False
        for w in (0, 1):
            if at[w] == len(progs[w]):
                continue
            op, bar, parity = progs[w][at[w]]
            done = dict(phases)
            if op == "arrive":
                done[bar] = done.get(bar, 0) + 1
            elif done.get(bar, 0) & 1 == parity:    # the phase now open has the parity waited for
                continue
            moved = True
            todo.append((tuple(a + (i == w) for i, a in enumerate(at)), tuple(sorted(done.items()))))
        stuck += not moved and any(a < len(p) for a, p in zip(at, progs))
    return stuck


def test_the_model_sees_a_barrier_that_wraps():
    assert _orders_that_hang(1, 1) == 0
    assert _orders_that_hang(2, 1) > 0


@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 9])
def test_no_order_of_the_issuing_warps_hangs(tiles):
    decl = re.search(r"v_clean(?:\[(\d+)\])?[,;]", open(SRC).read())
    assert _orders_that_hang(tiles, int(decl.group(1) or 1)) == 0
