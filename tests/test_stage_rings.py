"""A model of the stage rings of matmul_tiles.cu on the CPU: mbarriers as a count of arrivals
and a number of finished phases, of which a waiter sees one bit (the parity of the last).

Loads land in any order.  Groups of warps take every `turn`-th TMA stage, so they do not see every
phase of its barrier; the ring is sound if no schedule makes a group take a stage for full before
its own load has landed.  The model finds such schedules where the rule in the source (turn + the
converted stages, in TMA stages, at most the TMA stages; or a multiple of turn) does not hold, and
the configurations in the source keep it."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_03_gb300", "csrc",
                      "matmul_tiles.cu")


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1

    def passed(self, parity):   # the phase of this parity is the last finished one (or none was, for parity 1)
        return (self.done - 1) & 1 == parity


def lapped(raw, cvt, halves, sets, seed, loads=60):
    """Whether, in one random schedule, a group read a stage whose load had not landed."""
    rng = random.Random(seed)
    turn = sets * halves // 2
    full = [Barrier(1) for _ in range(raw)]
    empty = [Barrier(2 // halves) for _ in range(raw)]   # groups that share a TMA stage
    cfull = [Barrier(1) for _ in range(cvt)]
    cempty = [Barrier(1) for _ in range(cvt)]
    landed, flying = set(), []
    armed, mma = 0, 0
    uses = loads * 2 // halves
    at = list(range(sets))                               # next use of each group
    step = [0] * sets
    while mma < uses:
        moves = []
        if armed < loads and empty[armed % raw].passed((armed // raw & 1) ^ 1):
            moves.append("arm")
        moves += [("land", i) for i in flying]
        for g in range(sets):
            if at[g] < uses:
                i, c = at[g] * halves // 2, at[g] % cvt
                if step[g] == 0 and full[i % raw].passed(i // raw & 1):
                    moves.append(("take", g))
                if step[g] == 1 and cempty[c].passed((at[g] // cvt & 1) ^ 1):
                    moves.append(("give", g))
        if cfull[mma % cvt].passed(mma // cvt & 1):
            moves.append("mma")
        if not moves:
            return False   # nothing can move: a lost schedule of an unsound ring
        m = rng.choice([x for x in moves if x[0] != "land"] or moves) if rng.random() < 0.9 else rng.choice(moves)
        if m == "arm":
            flying.append(armed)
            armed += 1
        elif m == "mma":
            cempty[mma % cvt].arrive()
            mma += 1
        elif m[0] == "land":
            flying.remove(m[1])
            landed.add(m[1])
            full[m[1] % raw].arrive()
        elif m[0] == "take":
            if at[m[1]] * halves // 2 not in landed:
                return True
            step[m[1]] = 1
        else:
            u = at[m[1]]
            empty[u * halves // 2 % raw].arrive()
            cfull[u % cvt].arrive()
            at[m[1]], step[m[1]] = u + sets, 0
    return False


def sound(raw, cvt, halves, sets):
    turn = sets * halves // 2
    return turn + cvt * halves // 2 <= raw or raw % turn == 0


def configurations():
    text = open(SOURCE).read()
    found = re.findall(r"using \w+ = Config<(\d+), (\d+), (\d+), (\d+)>", text)
    sets = int(re.search(r"constexpr int kSets = (\d+)", text).group(1))
    return [(int(raw), int(cvt), int(halves), sets) for _, raw, cvt, halves in found]


def test_the_configurations_are_sound():
    assert len(configurations()) == 2
    for c in configurations():
        assert sound(*c)
        assert not any(lapped(*c, seed) for seed in range(400))


@pytest.mark.parametrize("raw,cvt,halves,sets", [(7, 4, 2, 4), (5, 4, 2, 4), (6, 4, 2, 4)])
def test_rings_that_a_group_can_lap(raw, cvt, halves, sets):
    assert not sound(raw, cvt, halves, sets)
    assert any(lapped(raw, cvt, halves, sets, seed) for seed in range(400))


@pytest.mark.parametrize("raw,cvt,halves,sets", [(8, 4, 2, 4), (4, 4, 2, 4), (5, 4, 1, 4), (6, 4, 1, 4), (9, 4, 2, 4), (8, 8, 1, 4)])
def test_sound_rings(raw, cvt, halves, sets):
    assert sound(raw, cvt, halves, sets)
    assert not any(lapped(raw, cvt, halves, sets, seed) for seed in range(400))
