"""The barrier protocol of the attention kernel for many rows (csrc/gdn_attn_rows.cu), restated as a
model and run under randomised schedules on the host.

One CTA walks the tiles of its share of units (a unit: the query rows of one sequence and head). Five
agents share its buffers: a loader of keys and one of values (rings of SLOTS tiles), one of queries, the
thread that issues the products, and the softmax warps (one agent: they arrive together). The copy engine
lands a copy at some later time; the tensor core runs the products and commits in order, at some later
time. An mbarrier wait with parity P passes when the barrier's completed-phase count has the other
parity, as the hardware decides it.

Checked for every schedule: no deadlock; no tile, query, score, probability or output rewritten before
its reader is done with it, asynchronous readers included; every read sees the tile meant for it; each
unit's output read once, complete.

The abort paths too: at a random moment one blocked wait gives up, every other one does from then on, each
role leaves by the kernel's own path, and nothing may be in flight when the CTA frees its tensor memory
and leaves. Without the products' last wait that must fail, and so must each planted protocol mistake."""
import collections
import random

import pytest

MISTAKES = ["no_pvdone_wait", "kempty_parity", "no_vempty_wait", "no_qfree_wait", "values_zeroed_late", "output_not_awaited"]


class Deadlock(Exception):
    pass


class CTA:
    def __init__(self, units, slots, mistake=None):
        self.units, self.slots, self.mistake = units, slots, mistake  # units: tiles and whether the last one is cut, each
        self.tiles = [(u, i) for u, (count, _) in enumerate(units) for i in range(count)]
        self.phases = collections.Counter()
        self.fifo, self.tma = collections.deque(), []
        self.k, self.v = [None] * slots, [None] * slots
        self.k_out, self.v_out, self.q_out, self.p_out, self.o_out = [0] * slots, [0] * slots, 0, 0, 0
        self.q, self.s, self.p, self.o = None, [None, None], None, None
        self.s_read, self.o_read = [True, True], []
        self.abort = False

    # ---- loads
    def load(self, ring, at, tile, bar):
        out = (self.k_out if ring is self.k else self.v_out)[at]
        assert out == 0, "a tile copied over one that a product still reads"
        ring[at] = None
        self.tma.append((ring, at, tile, bar))

    def land(self, k):
        ring, at, tile, bar = self.tma.pop(k)
        if ring is None:
            self.q = tile
        else:
            ring[at] = tile
        self.phases[bar] += 1

    def loader(self, ring, name):
        n = 0
        for n_ in range(len(self.tiles)):
            st, turn = n_ % self.slots, n_ // self.slots
            skip = name == "v" and self.mistake == "no_vempty_wait"
            if turn > 0 and not skip:
                flip = 1 if name == "k" and self.mistake == "kempty_parity" else 0
                if not (yield ("w", f"{name}empty{st}", ((turn - 1) & 1) ^ flip)):
                    break
            self.load(ring, st, n_, f"{name}full{st}")
            n = n_ + 1
        for i in range(max(0, n - self.slots), n):
            yield ("b", f"{name}full{i % self.slots}", (i // self.slots) & 1)

    def queries(self):
        sent = 0
        for u in range(len(self.units)):
            if u > 0 and self.mistake != "no_qfree_wait":
                if not (yield ("w", "qfree", (u - 1) & 1)):
                    break
            assert self.q_out == 0, "queries copied over ones that a product still reads"
            self.q = None
            self.tma.append((None, 0, u, "qfull"))
            sent = u + 1
        if sent:
            yield ("b", "qfull", (sent - 1) & 1)

    # ---- products
    def issue_scores(self, n, u):
        assert self.q == u and self.k[n % self.slots] == n, "scores of a tile or of queries that are not there"
        assert self.s_read[n & 1], "scores overwritten before the softmax read them"
        self.s_read[n & 1] = False
        self.s[n & 1] = None
        self.q_out += 1
        self.k_out[n % self.slots] += 1
        self.fifo.append(("qk", n, u))

    def issue_output(self, n):
        assert self.p == n and self.v[n % self.slots] in (n, ("zeroed", n)), "an output of probabilities or values that are not there"
        self.v_out[n % self.slots] += 1
        self.p_out += 1
        self.o_out += 1
        self.fifo.append(("pv", n))

    def commit(self, bar):
        self.fifo.append(("commit", bar))

    def products(self):
        def accumulate(n):
            if not (yield ("w", "pready", n & 1)) or not (yield ("w", f"vfull{n % self.slots}", (n // self.slots) & 1)):
                return False
            self.issue_output(n)
            self.commit(f"vempty{n % self.slots}")
            self.commit("pvdone")
            return True

        n, ok = 0, True
        for u, (count, _) in enumerate(self.units):
            ok = yield ("w", "qfull", u & 1)
            if not ok:
                break
            for i in range(count):
                ok = yield ("w", f"kfull{n % self.slots}", (n // self.slots) & 1)
                if ok and n >= 2:
                    ok = yield ("w", f"sfree{n & 1}", ((n >> 1) - 1) & 1)
                if not ok:
                    break
                self.issue_scores(n, u)
                self.commit(f"kempty{n % self.slots}")
                self.commit(f"sfull{n & 1}")
                if i == count - 1:
                    self.commit("qfree")
                if i > 0:
                    ok = yield from accumulate(n - 1)
                    if not ok:
                        break
                n += 1
            if ok:
                ok = yield from accumulate(n - 1)
            if not ok:
                break
        if self.mistake != "no_drain":  # whatever this thread issued is complete before the tensor memory goes back
            self.commit("drain")
            yield ("b", "drain", 0)

    def complete(self, op):
        if op[0] == "commit":
            self.phases[op[1]] += 1
        elif op[0] == "qk":
            _, n, u = op
            assert self.q == u and self.k[n % self.slots] == n, "operands of a score product changed while it ran"
            self.q_out -= 1
            self.k_out[n % self.slots] -= 1
            self.s[n & 1] = n
        else:
            n = op[1]
            u, i = self.tiles[n]
            assert self.p == n and self.v[n % self.slots] in (n, ("zeroed", n)), "operands of an output product changed while it ran"
            cut = self.units[u][1] and i == self.units[u][0] - 1
            assert (self.v[n % self.slots] != n) == cut, "values past the sequence's end were used"
            assert self.o == (u, i - 1) or i == 0, "an output product skipped a tile"
            self.v_out[n % self.slots] -= 1
            self.p_out -= 1
            self.o_out -= 1
            self.o = (u, i)

    # ---- softmax
    def softmax(self):
        n = 0
        for u, (count, cut) in enumerate(self.units):
            for i in range(count):
                if not (yield ("w", f"sfull{n & 1}", (n >> 1) & 1)):
                    return
                assert self.s[n & 1] == n, "the softmax read scores of another tile"
                self.s_read[n & 1] = True
                self.phases[f"sfree{n & 1}"] += 1
                if i > 0 and self.mistake != "no_pvdone_wait":
                    if not (yield ("w", "pvdone", (n - 1) & 1)):
                        return
                assert self.p_out == 0, "probabilities overwritten under a running product"
                assert self.o_out == 0 and (i == 0 or self.o == (u, i - 1)), "the output rescaled under a running product"
                self.p = n
                if cut and i == count - 1:
                    if self.mistake != "values_zeroed_late":
                        if not (yield ("w", f"vfull{n % self.slots}", (n // self.slots) & 1)):
                            return
                        assert self.v[n % self.slots] == n, "values of another tile zeroed"
                        self.v[n % self.slots] = ("zeroed", n)
                self.phases["pready"] += 1
                n += 1
            if self.mistake != "output_not_awaited":
                if not (yield ("w", "pvdone", (n - 1) & 1)):
                    return
            assert self.o == (u, count - 1) and self.o_out == 0 and self.p_out == 0, "an output read before it was complete"
            self.p = None  # (its memory serves the rows on their way out)
            self.o_read.append(u)

    # ---- the scheduler
    def run(self, rng, policy, timeout_rate=0.0):
        agents = dict(K=self.loader(self.k, "k"), V=self.loader(self.v, "v"), Q=self.queries(), P=self.products(), S=self.softmax())
        waits, results, timed_out = {}, {}, False

        def step(a):
            try:
                waits[a] = agents[a].send(results.pop(a, None))
            except StopIteration:
                del agents[a]
                waits.pop(a, None)

        for a in list(agents):
            step(a)

        def passes(a):
            return (self.phases[waits[a][1]] & 1) != waits[a][2]

        for _ in range(200_000):
            if not agents:
                break
            ready = [a for a in agents if passes(a) or (waits[a][0] == "w" and self.abort)]
            pending = ([("fifo", 0)] if self.fifo else []) + [("tma", k) for k in range(len(self.tma))]
            stuck = [a for a in agents if waits[a][0] == "w" and not passes(a)]
            if timeout_rate and not timed_out and stuck and rng.random() < timeout_rate:
                a, timed_out = rng.choice(stuck), True
                self.abort = True
                results[a] = False
                step(a)
                continue
            if not ready and not pending:
                raise Deadlock({a: waits[a] for a in agents})
            pool = [("agent", a) for a in ready] + pending
            if policy == "agents_first" and ready:
                pool = [("agent", a) for a in ready]
            elif policy == "async_first" and pending:
                pool = pending
            elif policy == "products_late":
                pool = [e for e in pool if e[0] != "fifo"] or pending
            kind, which = rng.choice(pool)
            if kind == "agent":
                results[which] = passes(which)
                step(which)
            elif kind == "fifo":
                self.complete(self.fifo.popleft())
            else:
                self.land(which)
        else:
            raise AssertionError("the model did not finish")
        assert not self.tma and not self.fifo, "work in flight when the CTA frees its tensor memory and leaves"
        if not self.abort:
            assert self.o_read == list(range(len(self.units)))


POLICIES = ["random", "agents_first", "async_first", "products_late"]


def shares(seed):
    rng = random.Random(seed)
    return [(rng.choice([1, 1, 2, 3, rng.randint(1, 20)]), rng.random() < 0.6) for _ in range(rng.randint(1, 8))]


def runs(count, mistake=None, rate=0.0):
    """(runs, those that failed, those that left by the abort paths)"""
    failed = aborted = total = 0
    for slots in (2, 5, 8):
        for policy in POLICIES:
            for seed in range(count):
                m = CTA(shares(seed), slots, mistake)
                total += 1
                try:
                    m.run(random.Random(seed), policy, rate)
                except (AssertionError, Deadlock):
                    if mistake is None:
                        raise
                    failed += 1
                aborted += m.abort
    return total, failed, aborted


def test_protocol_under_random_schedules():
    runs(30)


def test_abort_paths_leave_nothing_in_flight():
    for rate in (0.02, 0.3):
        total, _, aborted = runs(30, rate=rate)
        assert aborted > total // 3


@pytest.mark.parametrize("mistake", MISTAKES)
def test_planted_mistakes_are_caught(mistake):
    assert runs(12, mistake)[1] > 0


def test_an_abort_without_the_last_wait_of_the_products_is_caught():
    assert runs(12, "no_drain", 0.3)[1] > 0
