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


def stale_flags(guarded, units, seed):
    """The forward's flags of units (whether their values are all finite), written by the checking warp, read by the warps of two
    query tiles; units may have no second tile, and pass its warps by.  How many flags are read that another unit's has
    overwritten: four slots for all, or (guarded) four for each tile's outputs, with a barrier that frees them."""
    rng = random.Random(seed)
    has = [(True, rng.random() < 0.3) for _ in range(units)]
    flag = [[None] * 4, [None] * 4]
    free = [[Barrier(1) for _ in range(4)] for _ in range(2)]
    done, outputs, written = [0, 0], [0, 0], [0, 0]    # units and outputs behind each tile's warps; flags written for each
    at = wrong = steps = 0
    while min(done) < units:
        steps += 1
        assert steps < 1000 * units, "the flags stand still"
        who = rng.choice([0] * 4 + [1] + [2] * 4)
        if who == 2:
            if at == units or at > done[0] + 2:        # the ring lets the check run two units ahead of the first tile
                continue
            for i in range(2):
                n = written[i] if guarded else at
                if guarded and has[at][i] and not free[i][n % 4].passes(n // 4 & 1 ^ 1):
                    break
            else:
                for i in range(2):
                    if has[at][i]:
                        flag[i if guarded else 0][(written[i] if guarded else at) % 4] = at
                        written[i] += 1
                at += 1
        elif done[who] < units:
            k, n = done[who], outputs[who]
            if has[k][who]:
                if k >= at:
                    continue                           # its output waits for the check
                wrong += flag[who if guarded else 0][(n if guarded else k) % 4] != k
                free[who][n % 4].arrive()
                outputs[who] += 1
            done[who] += 1
    return wrong


def test_the_flags_of_units_wait_for_their_readers():
    with open(os.path.join(CSRC, "packed_tc_fwd.cu")) as f:
        text = f.read()
    guarded = "mbar_init(flag_free(n >> 2, n), 8)" in text and "mbar_wait_w(flag_free(1, n1)" in text
    assert sum(stale_flags(guarded, 300, seed) for seed in range(20)) == 0
    assert sum(stale_flags(False, 300, seed) for seed in range(20)) > 0
