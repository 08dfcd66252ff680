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


def _cluster_fault(ctas, rows, stop_sending):
    """The first fault some interleaving meets, or None."""

    @functools.lru_cache(maxsize=None)
    def search(pcs, dead, bars, flying):
        # pcs: steps taken (2 i: sends next, 2 i + 1: waits next); bars[c][flip] = (phases done, arrived, tx,
        # messages of this phase as a sorted tuple of iterations); flying: (to, iteration) pairs
        if all(pc == 2 * rows for pc in pcs):
            return "a message under way to a CTA that leaves" if any(not dead[to] for to, _ in flying) else None
        for n, (to, it) in enumerate(flying):                          # a message lands
            if n > 0 and flying[n - 1] == flying[n]:
                continue
            found = search(pcs, dead, _settle(bars, to, it % 2, 0, -1, it), flying[:n] + flying[n + 1:])
            if found:
                return found
        for c in range(ctas):
            if pcs[c] == 2 * rows:
                continue
            i, waits = divmod(pcs[c], 2)
            step = pcs[:c] + (pcs[c] + 1,) + pcs[c + 1:]
            if not waits:
                if dead[c] and stop_sending:
                    found = search(step, dead, bars, flying)
                elif bars[c][i % 2][1]:
                    return "an arrival on a phase that has it already"
                else:
                    sent = tuple(sorted(flying + tuple((to, i) for to in range(ctas))))
                    found = search(step, dead, _settle(bars, c, i % 2, 1, ctas, None), sent)
            else:
                phases, _, _, _, last = bars[c][i % 2]
                if phases > i // 2:
                    if not dead[c] and last != (i,) * ctas:
                        return "sums of another iteration"
                    found = search(step, dead, bars, flying)
                else:
                    found = search(step, dead[:c] + (True,) + dead[c + 1:], bars, flying)      # runs out
            if found:
                return found
        return None

    def _settle(bars, c, flip, arrive, tx, message):
        phases, arrived, count, got, last = bars[c][flip]
        arrived, count = arrived + arrive, count + tx
        if message is not None:
            got = tuple(sorted(got + (message,)))
        if arrived == 1 and count == 0:
            phases, arrived, got, last = phases + 1, 0, (), got
        pair = list(bars[c])
        pair[flip] = (phases, arrived, count, got, last)
        return bars[:c] + (tuple(pair),) + bars[c + 1:]

    start = (0, 0, 0, (), ())
    return search((0,) * ctas, (False,) * ctas, ((start, start),) * ctas, ())


@pytest.mark.parametrize("ctas,rows", [(2, 1), (2, 2), (2, 3), (2, 4), (3, 2)])
def test_cluster_sums_stop_together(ctas, rows):
    assert _cluster_fault(ctas, rows, stop_sending=True) is None


def test_the_search_finds_the_arrival_of_a_cta_that_goes_on():
    assert _cluster_fault(2, 3, stop_sending=False) == "an arrival on a phase that has it already"
