"""Exhaustive checks, on the CPU, of how the kernels of layernorm_backward and matmul_int8 stop when a
bounded wait runs out.

The roles of a CTA: one issues asynchronous work into a ring of slots (copies into shared memory, or
MMAs that read operand stages), another waits for each slot and hands it back. Any wait that is not
satisfied may run out, which ends its role. The search runs every interleaving of the roles' steps, of
the work's completions and of waits that run out, and checks that none of the work is in flight when
the CTA ends. Where the issuer waits for its work only after a wait of its own ran out, the search finds
a CTA that ends too early: everything was issued when the other role stopped."""
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
