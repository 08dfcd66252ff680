"""Exhaustive checks, on the CPU, of how the kernels of layernorm_backward and matmul_int8 stop when a
bounded wait runs out.

The roles of a CTA: one issues asynchronous work into a ring of slots (copies into shared memory, or
MMAs that read operand stages), another waits for each slot and hands it back. Any wait that is not
satisfied may run out, which ends its role. The search runs every interleaving of the roles' steps, of
the work's completions and of waits that run out, and checks that none of the work is in flight when
the CTA ends. Where the issuer waits for its work only after a wait of its own ran out, the search finds
a CTA that ends too early: everything was issued when the other role stopped.

The sums of a cluster's CTAs (layernorm_backward): in iteration i a CTA arrives on its barrier i mod 2,
expecting a message from every CTA, sends one to every CTA, and waits for the barrier's phase. Messages
land in any order. The search checks that no CTA arrives on a phase that already has its arrival (the
count would fall below zero), that a wait that succeeds has every CTA's message of its own iteration,
and that at the end only CTAs whose wait ran out have messages under way, which is why those stay a
moment longer. Where a CTA goes on sending after a wait that ran out, the search finds the arrival."""
import functools
import random

import pytest


def _ends_with_work_in_flight(work, slots, drain_always):
    """True if some interleaving ends both roles with work in flight."""

    @functools.lru_cache(maxsize=None)
    def search(issuer, issued, done, user, used):
        # issuer, user: "run", "drain" (issuer), "stopped" or "end"; done: the issued work that is complete
        if issuer in ("end", "stopped") and user in ("end", "stopped"):
            return len(done) < issued
        nxt = []
        for j in range(issued):
            if j not in done:
                nxt.append((issuer, issued, done | {j}, user, used))
        if issuer == "run":
            if issued == work:
                nxt.append(("drain" if drain_always else "end", issued, done, user, used))
            elif issued - used < slots:
                nxt.append((issuer, issued + 1, done, user, used))
            else:
                nxt.append(("drain", issued, done, user, used))               # its wait for a slot runs out
        elif issuer == "drain" and len(done) == issued:
            nxt.append(("stopped", issued, done, user, used))
        if user == "run":
            if used == work:
                nxt.append((issuer, issued, done, "end", used))
            elif used in done:
                nxt.append((issuer, issued, done, user, used + 1))
            else:
                nxt.append((issuer, issued, done, "stopped", used))           # its wait for the work runs out
        return any(search(*s) for s in nxt)

    return search("run", 0, frozenset(), "run", 0)


@pytest.mark.parametrize("work", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("slots", [1, 2, 3])
def test_no_work_in_flight_when_a_cta_ends(work, slots):
    assert not _ends_with_work_in_flight(work, slots, drain_always=True)


def test_the_search_finds_a_cta_that_ends_too_early():
    assert _ends_with_work_in_flight(2, 2, drain_always=False)


class _Cluster:
    """The exchange as states and their successors. Lane r of a CTA's sending warp sends to CTA r, lane 0
    arrives as well, and each lane's wait runs out by itself.

    A state: steps each lane has taken (2 i: sends next, 2 i + 1: waits next); which lanes' waits ran out;
    bars[c][flip] = (phases done, arrived, messages expected, those of this phase as a sorted tuple of
    iterations, those of the last phase); and what is under way, as (to, iteration) pairs."""

    def __init__(self, ctas, rows, stop_sending):
        self.ctas, self.rows, self.stop_sending = ctas, rows, stop_sending
        self.lanes = [(c, r) for c in range(ctas) for r in range(ctas)]
        bar = (0, 0, 0, (), ())
        self.start = ((0,) * len(self.lanes), (False,) * len(self.lanes), ((bar, bar),) * ctas, ())

    @staticmethod
    def _settle(bars, c, flip, arrive, expect, message):
        phases, arrived, count, got, last = bars[c][flip]
        arrived, count = arrived + arrive, count + expect
        if message is not None:
            got = tuple(sorted(got + (message,)))
        if arrived == 1 and count == 0:
            phases, arrived, got, last = phases + 1, 0, (), got
        pair = list(bars[c])
        pair[flip] = (phases, arrived, count, got, last)
        return bars[:c] + (tuple(pair),) + bars[c + 1:]

    def successors(self, state):
        """A list of states, or the fault that is met."""
        pcs, dead, bars, flying = state
        end = 2 * self.rows
        if all(pc == end for pc in pcs):
            stay = {c for n, (c, _) in enumerate(self.lanes) if dead[n]}
            return "a message under way to a CTA that leaves" if any(to not in stay for to, _ in flying) else []
        out = []
        for n, (to, it) in enumerate(flying):                          # a message lands
            if n == 0 or flying[n - 1] != flying[n]:
                out.append((pcs, dead, self._settle(bars, to, it % 2, 0, -1, it), flying[:n] + flying[n + 1:]))
        for n, (c, r) in enumerate(self.lanes):
            i, waits = divmod(pcs[n], 2)
            # the lanes of a warp send together, after all have waited
            if pcs[n] == end or not waits and any(pcs[m] < pcs[n] for m, (d, _) in enumerate(self.lanes) if d == c):
                continue
            step = pcs[:n] + (pcs[n] + 1,) + pcs[n + 1:]
            if waits:
                phases, _, _, _, last = bars[c][i % 2]
                if phases > i // 2:
                    if not dead[n] and last != (i,) * self.ctas:
                        return "sums of another iteration"
                    out.append((step, dead, bars, flying))
                else:                                                  # runs out
                    out.append((step, dead[:n] + (True,) + dead[n + 1:], bars, flying))
            elif dead[n] and self.stop_sending:
                out.append((step, dead, bars, flying))
            else:
                if r == 0 and bars[c][i % 2][1]:
                    return "an arrival on a phase that has it already"
                after = self._settle(bars, c, i % 2, 1, self.ctas, None) if r == 0 else bars
                out.append((step, dead, after, tuple(sorted(flying + ((r, i),)))))
        return out

    def search(self):
        """The first fault that some interleaving meets, or None."""
        seen, todo = {self.start}, [self.start]
        while todo:
            nxt = self.successors(todo.pop())
            if isinstance(nxt, str):
                return nxt
            for state in nxt:
                if state not in seen:
                    seen.add(state)
                    todo.append(state)
        return None

    def walk(self, rng):
        """The fault of one random interleaving, or None. Waits that could run out seldom do."""
        state = self.start
        while True:
            nxt = self.successors(state)
            if isinstance(nxt, str) or not nxt:
                return nxt or None
            patient = [s for s in nxt if s[1] == state[1]]
            state = rng.choice(patient if patient and rng.random() < 0.9 else nxt)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
def test_cluster_sums_stop_together(rows):
    assert _Cluster(2, rows, stop_sending=True).search() is None


@pytest.mark.parametrize("ctas,rows", [(3, 3), (3, 6), (4, 4)])
def test_cluster_sums_stop_together_in_random_orders(ctas, rows):
    rng = random.Random(ctas * 100 + rows)
    model = _Cluster(ctas, rows, stop_sending=True)
    assert all(model.walk(rng) is None for _ in range(1000))


def test_the_search_finds_the_arrival_of_a_cta_that_goes_on():
    assert _Cluster(2, 3, stop_sending=False).search() == "an arrival on a phase that has it already"
