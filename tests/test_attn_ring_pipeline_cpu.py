"""The ring of the attention kernel for few rows (csrc/gdn_attn_decode.cu), restated as a model and run
under randomised schedules on the host.

Three loading warps fill every third slot of a share, whatever place of the ring that is; NG groups of
computing warps take every NG-th slot. A place's barrier completes one phase a turn, and an mbarrier wait
with parity P passes when the number of completed phases has the other parity. Releases are counted. The
copy engine lands a copy at some later time.

Checked for every schedule: no deadlock, no slot filled before its readers are done with it or read before
its copy has landed, every slot read once by its group. With one wait giving up at a random moment: every
role leaves, nothing is in flight when the last one has left, and no last wait asks for a phase that has
passed by (a bounded wait would run for its whole limit). Last waits that go by the parity alone, that look at
a loader's last turn only, or that are made only after an abort is seen must be caught."""
import collections
import random

import pytest

LOADERS = 3


class Deadlock(Exception):
    pass


class CTA:
    def __init__(self, slots, places, groups, mistake=None):
        self.slots, self.places, self.groups, self.mistake = slots, places, groups, mistake
        self.phases, self.freed = collections.Counter(), collections.Counter()
        self.ring, self.tma, self.read = [None] * places, [], []
        self.abort = False

    def full(self, st, parity):
        return lambda: (self.phases[st] & 1) != parity

    def count(self, st, n):
        return lambda: self.freed[st] >= n

    def loader(self, w):
        sent = -1
        for i in range(w, self.slots, LOADERS):
            st, turn = i % self.places, i // self.places
            if not (yield ("w", self.count(st, turn))):
                break
            assert turn == 0 or (turn - 1) * self.places + st in self.read, "a slot filled before it was read"
            self.ring[st] = None
            self.tma.append((st, i))
            sent = i
        if self.mistake == "after_an_abort_only" and not self.abort:
            return
        if self.mistake == "the_last_turn_only":
            for i in range(sent, max(-1, sent - self.places), -LOADERS):
                st, turn = i % self.places, i // self.places
                landed, was_read = self.full(st, turn & 1), self.count(st, turn + 1)
                yield ("b", lambda landed=landed, was_read=was_read: landed() or was_read())
            return
        for st in range(self.places):
            turn = self.freed[st]
            i = turn * self.places + st
            if i <= sent and i % LOADERS == w:
                landed, was_read = self.full(st, turn & 1), self.count(st, turn + 1)
                if self.mistake == "without_counts":
                    yield ("b", landed)
                else:
                    yield ("b", lambda landed=landed, was_read=was_read: landed() or was_read())

    def group(self, g):
        for i in range(g, self.slots, self.groups):
            st, turn = i % self.places, i // self.places
            if not (yield ("w", self.count(st, turn))) or not (yield ("w", self.full(st, turn & 1))):
                return
            assert self.ring[st] == i, "a slot read before its copy landed"
            self.read.append(i)
            yield ("b", lambda: True)  # it works on the slot for some time
            self.freed[st] += 1

    def run(self, rng, policy, rate=0.0):
        agents = {("L", w): self.loader(w) for w in range(LOADERS)}
        agents.update({("G", g): self.group(g) for g in range(self.groups)})
        waits, results, timed_out = {}, {}, False

        def step(a):
            try:
                waits[a] = agents[a].send(results.pop(a, None))
            except StopIteration:
                del agents[a]
                waits.pop(a, None)

        for a in list(agents):
            step(a)
        while agents:
            ready = [a for a in agents if waits[a][1]() or (waits[a][0] == "w" and self.abort)]
            stuck = [a for a in agents if waits[a][0] == "w" and not waits[a][1]()]
            if rate and not timed_out and stuck and rng.random() < rate:
                a, timed_out, self.abort = rng.choice(stuck), True, True
                results[a] = False
                step(a)
                continue
            pool = [("agent", a) for a in ready] + [("tma", k) for k in range(len(self.tma))]
            if policy == "copies_late" and ready:
                pool = [e for e in pool if e[0] == "agent"]
            elif policy == "copies_first" and self.tma:
                pool = [e for e in pool if e[0] == "tma"]
            if not pool:
                raise Deadlock(list(waits))
            kind, which = rng.choice(pool)
            if kind == "agent":
                results[which] = waits[which][1]()
                step(which)
            else:
                st, i = self.tma.pop(which)
                self.ring[st] = i
                self.phases[st] += 1
        assert not self.tma, "a copy in flight when the block leaves"
        if not self.abort:
            assert sorted(self.read) == list(range(self.slots))


def runs(count, mistake=None, rate=0.0):
    failed = aborted = total = 0
    for places in (8, 9, 10, 12):
        for groups in (1, 2, 4, 8):
            for policy in ("random", "copies_late", "copies_first"):
                for seed in range(count):
                    rng = random.Random(seed)
                    m = CTA(rng.choice([1, 2, 3, 7, rng.randint(1, 60)]), places, groups, mistake)
                    total += 1
                    try:
                        m.run(rng, policy, rate)
                    except (AssertionError, Deadlock):
                        if mistake is None:
                            raise
                        failed += 1
                    aborted += m.abort
    return total, failed, aborted


def test_ring_under_random_schedules():
    runs(12)


@pytest.mark.parametrize("rate", [0.01, 0.2])
def test_nothing_is_in_flight_after_an_abort(rate):
    total, _, aborted = runs(20, rate=rate)
    assert aborted > total // 8


@pytest.mark.parametrize("mistake,rate", [("after_an_abort_only", 0.2), ("without_counts", 0.0), ("the_last_turn_only", 0.01)])
def test_mistakes_are_caught(mistake, rate):
    assert runs(40, mistake, rate)[1] > 0
