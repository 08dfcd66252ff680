"""The slots of the 4-bit product's CTA pairs, as a model on the CPU: two loading warps that know one barrier per slot, and a
leader whose copies of scales, commits and MMAs run in the order of their issue. Whatever the order in which loads land and
each side goes on, nothing is overwritten before it has been read, every stage is there when it is used, and nobody waits
for ever. The numbers of slots are the kernel's."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_precision_activation_gb300", "csrc")
with open(os.path.join(CSRC, "rmsq_fp4_pair.cuh")) as f:
    SLOTS, LESS = (int(v) for v in re.search(r"SLOTS = (\d+), SCALE_SLOTS = SLOTS - (\d+);", f.read()).groups())


def run(stages, rng, slots, scale_slots):
    empty, full = [0] * slots, [0] * slots                   # phases that are over
    codes, scales = ([[None] * n, [None] * n] for n in (slots, scale_slots))
    loaded, landed, flying, issued, pipe, copied, multiplied = [0, 0], {}, [], 0, [], set(), set()
    while len(multiplied) < stages:
        can = []
        for cta in (0, 1):
            j = loaded[cta]
            # a wait for a parity passes when the phase of that parity is over; the last slot's first word is of scales
            slot, parity = j % slots, (j // slots) & 1 if j % slots == slots - 1 else ((j // slots) & 1) ^ 1
            if j < stages and (empty[slot] & 1) != parity:
                can.append(("load", cta))
        if flying:
            can.append(("land", 0))
        if issued < stages and full[issued % slots] > issued // slots:
            can.append(("issue", 0))
        if pipe:
            can.append(("execute", 0))
        assert can, "everybody waits"
        what, cta = rng.choice(can)
        if what == "load":
            j = loaded[cta]
            loaded[cta] += 1
            assert codes[cta][j % slots] is None or codes[cta][j % slots] in multiplied, "codes still needed"
            assert scales[cta][j % scale_slots] is None or scales[cta][j % scale_slots] in copied, "scales still needed"
            codes[cta][j % slots] = scales[cta][j % scale_slots] = j
            flying.append(j)
        elif what == "land":
            j = flying.pop(rng.randrange(len(flying)))
            landed[j] = landed.get(j, 0) + 1
            if landed[j] == 2:
                assert full[j % slots] == j // slots, "counted in another phase"
                full[j % slots] += 1
        elif what == "issue":
            pipe += [("copy", issued), ("commit", (issued - 1) % slots), ("multiply", issued)]
            issued += 1
        else:
            kind, at = pipe.pop(0)
            if kind == "copy":
                assert all(s[at % scale_slots] == at for s in scales)
                copied.add(at)
            elif kind == "multiply":
                assert all(c[at % slots] == at for c in codes)
                multiplied.add(at)
            else:
                empty[at] += 1


@pytest.mark.parametrize("seed", range(8))
def test_the_kernels_slots(seed):
    rng = random.Random(seed)
    for _ in range(150):
        run(rng.randint(1, 5 * SLOTS), rng, SLOTS, SLOTS - LESS)


def test_fewer_slots_of_scales_would_not_do():
    # the commit behind a stage's scales frees those, and the codes of the stage before: one slot less, no more
    with pytest.raises(AssertionError):
        for seed in range(200):
            run(40, random.Random(seed), SLOTS, SLOTS - LESS - 1)
