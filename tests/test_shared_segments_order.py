"""The order of accesses to the segment statistics of the shared-prefix attention (csrc/shared.cu), on a model of
its synchronisation: what the kernel's barriers order has to include every pair of accesses that must not swap.

With at most 128 readers the two softmax groups A and B take every other key tile of a segment. A thread of either
group, per segment: brings its part of the queries (an arrival), and for each of its tiles waits for the scores,
which are issued when all threads of both groups have arrived; then writes its statistics; meets the others at a
barrier; and reads both groups' statistics. Vector clocks say which accesses are ordered."""
import itertools

import pytest


def conflicts(segments, b_writes_without_scores):
    """Unordered (write, read) or (write, write) pairs of accesses to a group's statistics, for two threads a group
    and segments of the given numbers of key tiles."""
    threads = [(g, i) for g in "AB" for i in range(2)]
    clock = {t: {u: 0 for u in threads} for t in threads}
    seen = []  # (group whose statistics, kind, thread, time, clock)

    def tick(t, group=None, kind=None):
        clock[t][t] += 1
        if group is not None:
            seen.append((group, kind, t, clock[t][t], dict(clock[t])))

    def join(into, others):
        for u in threads:
            into[u] = max([into[u]] + [c[u] for c in others])

    for tiles in segments:
        for t in threads:
            tick(t)  # the queries
        arrived = [dict(clock[t]) for t in threads]
        for t in threads:
            mine = len(range(0 if t[0] == "A" else 1, tiles, 2))
            if mine:
                join(clock[t], arrived)  # its scores come after all arrivals
            if mine or b_writes_without_scores:
                tick(t, t[0], "w")
        met = [dict(clock[t]) for t in threads]
        for t in threads:
            join(clock[t], met)
            for g in "AB" if tiles > 1 else "A":
                tick(t, g, "r")
    pairs = []
    for (g1, k1, t1, at1, c1), (g2, k2, t2, at2, c2) in itertools.combinations(seen, 2):
        if g1 == g2 and t1 != t2 and "w" in (k1, k2) and t1[1] == t2[1] and not (c2[t1] >= at1 or c1[t2] >= at2):
            pairs.append(((g1, k1, t1, at1), (g2, k2, t2, at2)))
    return pairs


@pytest.mark.parametrize("segments", [[2, 1], [3, 1, 2], [1, 1, 1], [5, 2, 1, 1, 4], [1, 3, 1, 3]])
def test_accesses_are_ordered(segments):
    assert conflicts(segments, False) == []


@pytest.mark.parametrize("segments", [[2, 1], [3, 1, 2], [5, 2, 1, 1, 4]])
def test_an_unconditional_write_would_not_be(segments):
    # the model tells: group B's write in a segment of one tile, against group A's read in the one before
    found = conflicts(segments, True)
    assert found and any({p[0][1], p[1][1]} == {"r", "w"} and p[0][0] == "B" and {p[0][2][0], p[1][2][0]} == {"A", "B"}
                         for p in found)
