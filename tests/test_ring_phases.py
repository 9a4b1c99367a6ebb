"""The rings of the packed attention kernels under any timing: a model of an mbarrier (a wait names a parity, so it passes in the
phase behind the one that it names, and again two phases later) with a loader, a warp that issues the products and a warp that waits
for every item but works on few.  The number of arrivals that free a slot is read from the kernels' sources."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hierarchical_kv_routing_tok_b200", "csrc")


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passes(self, parity):
        return self.phase & 1 != parity


def late(ring, empties, items, seed):
    """How many items the watching warp took for another: runs the three in a random order, the watcher slow."""
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(ring)], [Barrier(empties) for _ in range(ring)]
    held = [None] * ring                               # the item in each slot
    at = {"load": 0, "product": 0, "watch": 0}
    wrong = steps = 0
    while at["product"] < items or at["watch"] < items:
        steps += 1
        assert steps < 1000 * items, "the ring stands still"
        who = rng.choice(["load"] * 4 + ["product"] * 4 + ["watch"])
        j = at[who]
        if j >= items:
            continue
        s, parity = j % ring, j // ring & 1
        if who == "load":
            if not empty[s].passes(parity ^ 1):
                continue
            held[s] = j
            full[s].arrive()
        else:
            if not full[s].passes(parity):
                if who == "watch" and at["product"] >= items and at["load"] >= items:
                    return wrong + items - j           # it waits for a phase that does not come again
                continue
            wrong += held[s] != j
            if who == "product" or empties == 2:
                empty[s].arrive()
        at[who] = j + 1
    return wrong


RINGS = [("packed_tc_fwd.cu", "empty", 2), ("packed_tc_bwd.cu", "k_empty", 3), ("packed_tc_bwd.cu", "q_empty", 4)]


@pytest.mark.parametrize("name,bar,ring", RINGS, ids=[b for _, b, _ in RINGS])
def test_the_cleaning_warp_holds_the_ring(name, bar, ring):
    with open(os.path.join(CSRC, name)) as f:
        count = re.search(r"mbar_init\(%s\(s\), (?:ragged \? )?(\d)" % bar, f.read())
    assert sum(late(ring, int(count.group(1)), 200, seed) for seed in range(20)) == 0


@pytest.mark.parametrize("ring", [2, 3, 4])
def test_the_model_sees_a_ring_that_does_not_wait(ring):
    assert sum(late(ring, 1, 200, seed) for seed in range(20)) > 0
