"""A model of the stage ring of matmul_fp8.cu on the CPU, whose blocks two warps issue in turn: mbarriers as a count of
arrivals and a number of finished phases, of which a waiter sees one bit (the parity of the last).

Loads land in any order.  A warp looks at every other block's stage, so that with an odd number of stages it sees every
second phase of a barrier; the ring is sound if no schedule makes it take a stage for full before its own load has
landed.  The model finds such schedules where the rule in the source (an even number of stages, or two more than
accumulators) does not hold, and the configurations in the source keep it."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_03_gb300", "csrc",
                      "matmul_fp8.cu")


class Barrier:
    def __init__(self):
        self.done = 0   # every barrier here takes one arrival a phase

    def arrive(self):
        self.done += 1

    def passed(self, parity):   # the phase of this parity is the last finished one (or none was, for parity 1)
        return (self.done - 1) & 1 == parity


def lapped(stages, accs, seed, blocks=60):
    """Whether, in one random schedule, a warp issued a block whose load had not landed."""
    rng = random.Random(seed)
    full, empty = [Barrier() for _ in range(stages)], [Barrier() for _ in range(stages)]
    acc_full, acc_empty = [Barrier() for _ in range(accs)], [Barrier() for _ in range(accs)]
    landed, flying, running = set(), [], []
    armed = read = 0
    at, ready = [0, 1], [False, False]
    slow = rng.randrange(blocks)                       # one load that comes late
    while read < blocks:
        moves = []
        if armed < blocks and empty[armed % stages].passed((armed // stages & 1) ^ 1):
            moves.append(("arm",))
        moves += [("land", i) for i in flying if i != slow or rng.random() < 0.02]
        for w in range(2):
            b = at[w]
            if b < blocks and not ready[w] and full[b % stages].passed(b // stages & 1):
                moves.append(("see", w))
            if b < blocks and ready[w] and acc_empty[b % accs].passed((b // accs & 1) ^ 1):
                moves.append(("issue", w))
        if running:
            moves.append(("finish",))
        if acc_full[read % accs].passed(read // accs & 1):
            moves.append(("read",))
        if not moves:
            if slow in flying:
                moves.append(("land", slow))
            else:
                return False   # nothing can move: a lost schedule of an unsound ring
        m = rng.choice(moves)
        if m[0] == "arm":
            flying.append(armed)
            armed += 1
        elif m[0] == "land":
            flying.remove(m[1])
            landed.add(m[1])
            full[m[1] % stages].arrive()
        elif m[0] == "see":
            if at[m[1]] not in landed:
                return True
            ready[m[1]] = True
        elif m[0] == "issue":
            running.append(at[m[1]])
            at[m[1]], ready[m[1]] = at[m[1]] + 2, False
        elif m[0] == "finish":   # products end in the order of their issue
            b = running.pop(0)
            acc_full[b % accs].arrive()
            empty[b % stages].arrive()
        else:
            acc_empty[read % accs].arrive()
            read += 1
    return False


def sound(stages, accs):
    return stages % 2 == 0 or stages >= accs + 2


def configurations():
    found = re.findall(r"using \w+ = Config<(\d+), (\d+), (\d+), (\d+), (\d+), (\d+)>", open(SOURCE).read())
    return [(int(stages), int(accs)) for _, _, _, stages, accs, _ in found]


def test_the_configurations_are_sound():
    assert len(configurations()) == 4
    for c in configurations():
        assert sound(*c)
        assert not any(lapped(*c, seed) for seed in range(400))


@pytest.mark.parametrize("stages,accs", [(5, 4), (3, 2), (3, 4), (7, 8)])
def test_rings_that_a_warp_can_lap(stages, accs):
    assert not sound(stages, accs)
    assert any(lapped(stages, accs, seed) for seed in range(2000))


@pytest.mark.parametrize("stages,accs", [(5, 2), (9, 4), (7, 4), (4, 4), (6, 4), (4, 2), (6, 8)])
def test_sound_rings(stages, accs):
    assert sound(stages, accs)
    assert not any(lapped(stages, accs, seed) for seed in range(400))
