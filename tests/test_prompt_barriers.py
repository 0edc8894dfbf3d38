"""The barriers of the bf16 whole-prompt kernel as a model on the CPU: the thread that issues the
copies, the warp that watches them (the gate), the thread that issues the MMAs and the softmax warps
of both tiles, scheduled at random, with any of them as late as the others allow.  A wait is the
hardware's: it tells phases apart by their parity alone, so a role that looks two phases late waits
for ever.  An item is (blocks of tile 0, blocks of tile 1), tile 1 empty or at least as long."""
import random

import pytest

STEPS = 4  # barriers of the MMA thread's steps


def stuck(items, ring, slow, seed, gate_looks_at_all=False):
    """What each role waits for when none can go on; None when all end.  Roles in ``slow`` run only
    when no other can."""
    rnd = random.Random(seed)
    count = {("p", 0, 0): 2, ("p", 0, 1): 1, ("p", 1, 0): 1, ("p", 1, 1): 1, ("s", 0): 1, ("s", 1): 1}
    count.update({("full", i): 1 for i in range(ring)})
    count.update({("step", i): 1 for i in range(STEPS)})
    phase, here = dict.fromkeys(count, 0), dict.fromkeys(count, 0)

    def arrive(bar):
        here[bar] += 1
        if here[bar] == count[bar]:
            phase[bar], here[bar] = phase[bar] + 1, 0

    def copies():
        issued = steps = 0
        for it in items:
            for _ in range(2 * max(it)):
                while issued >= ring and 2 * steps < issued - ring + 2:
                    yield ("step", steps % STEPS), steps // STEPS & 1
                    steps += 1
                yield None
                arrive(("full", issued % ring))
                issued += 1

    def gate():
        n = blocks = 0
        for it in items:
            looks = [gate_looks_at_all]                      # K of block 0
            for j in range(max(it)):
                seen = j < it[0]
                looks += [seen or gate_looks_at_all] * (1 + (j + 1 < max(it)))
                for look in looks:
                    if look:
                        yield ("full", n % ring), n // ring & 1
                    n += 1
                looks = []
                if seen:
                    if blocks:
                        yield ("p", 0, 0), (blocks - 1) & 1
                    blocks += 1
                    arrive(("p", 0, 0))

    def mma():
        scored, step, i, j, k, v = [0, 0], 0, 0, -1, 0, None
        while True:
            it, last = items[i], j + 1 == max(items[i])
            after = (items[i + 1] if i + 1 < len(items) else (0, 0)) if last else it
            nj = 0 if last else j + 1
            for t in (0, 1):
                if 0 <= j < it[t]:
                    if j >= it[0]:
                        yield ("full", v % ring), v // ring & 1
                    for part in (0, 1):
                        yield ("p", t, part), (scored[t] - 1) & 1
                if nj < after[t]:
                    if nj == 0 if t == 0 else nj >= after[0]:
                        yield ("full", k % ring), k // ring & 1
                    scored[t] += 1
                    arrive(("s", t))
            if last and i + 1 == len(items):
                return
            arrive(("step", step % STEPS))
            step, i, j, k, v = step + 1, i + last, 0 if last else j + 1, k + 2, k + 1

    def softmax(t):
        n = 0
        for it in items:
            for _ in range(it[t]):
                yield ("s", t), n & 1
                for part in (0, 1):
                    yield None
                    arrive(("p", t, part))
                n += 1

    roles = {"copies": copies(), "gate": gate(), "mma": mma(), "s0": softmax(0), "s1": softmax(1)}
    waits = dict.fromkeys(roles)
    while roles:
        ready = [r for r in roles if waits[r] is None or phase[waits[r][0]] & 1 != waits[r][1]]
        if not ready:
            return {r: waits[r] for r in roles}
        r = rnd.choice([r for r in ready if r not in slow] or ready)
        try:
            waits[r] = next(roles[r])
        except StopIteration:
            del roles[r]
    return None


def batches(n):
    rnd = random.Random(1)
    for _ in range(n):
        items = []
        for _ in range(rnd.randint(1, 12)):
            a = rnd.randint(1, 9)
            items.append((a, rnd.choice([0, a, a, a + 1])))
        yield items


SLOW = [(), ("gate",), ("copies",), ("mma",), ("s0",), ("s1",), ("gate", "s1"), ("copies", "gate")]


@pytest.mark.parametrize("slow", SLOW)
@pytest.mark.parametrize("ring", [5, 8])
def test_every_role_may_be_late(ring, slow):
    for seed, items in enumerate(batches(120)):
        assert stuck(items, ring, slow, seed) is None, items


def test_the_model_tells_waits_that_come_too_late():
    # A gate that also looks at the loads that the MMA thread waits for by itself can be passed by.
    assert all(stuck([(9, 9)], ring, ("gate",), 0, gate_looks_at_all=True) for ring in (5, 8))
