"""The hand-offs of the paged attention's tile kernels at tile granularity: each
role of a CTA is a program of actions that wait for the actions which its
barriers stand for (as in test_loader_protocol.py), under random schedules.

* loader: at a unit's head its q into the one of two buffers that the unit
  before the last used (its score products done, every softmax warp past its
  head), distance tiles -2 and -1, then per step K, r and, `lag` steps behind, V
  together (each stage free);
* score and distance issuers: a unit behind its q, and behind the reads of step
  g0 - 2, for u and v overwrite what the unit before the last used;
* P.V issuer and softmax: D = 64 alternate steps of two parities with an
  accumulator each and four ring slots; D = 128 two halves that take every step,
  three slots."""

import random

import pytest

from test_loader_protocol import _run


def programs(D, nks, lag):
    N = len(nks)
    first = [sum(nks[:u]) for u in range(N)]
    unit = [u for u in range(N) for _ in range(nks[u])]
    tile0 = [first[u] + 2 * u for u in range(N)]
    stages, slots = (4, 4) if D == 64 else (2, 3)

    def owner(g):
        return g & 1

    def read(g):  # the scores and the window of step g have been read
        return [("RD", owner(g), g)] if D == 64 else [("RD", 0, g), ("RD", 1, g)]

    # ---- loader
    loader, held, nv, nr = [], [], 0, 0
    for u, n in enumerate(nks):
        deps = []
        if u >= 2:
            deps = [("S", first[u - 1] - 1), ("G", tile0[u - 1] - 1), ("SEEN", 0, u - 2), ("SEEN", 1, u - 2)]
        loader.append((("LQ", u), deps))
        for _ in range(2):
            loader.append((("LR", nr), [("G", nr - stages)] if nr >= stages else []))
            nr += 1
        for t in range(n):
            g = first[u] + t
            deps = ([("S", g - stages)] if g >= stages else []) + ([("G", nr - stages)] if nr >= stages else [])
            held.append(g)
            has_v = len(held) > lag
            if has_v and nv >= stages:
                deps.append(("PV", nv - stages))
            loader.append((("LK", g), deps))
            loader.append((("LR", nr), []))
            nr += 1
            if has_v:
                loader.append((("LV", held.pop(0)), []))
                nv += 1
    for g in held:
        loader.append((("LV", g), [("PV", nv - stages)] if nv >= stages else []))
        nv += 1
    progs = {"loader": loader}
    # ---- issuers
    progs["S"] = [(("S", g), [("LK", g), ("LQ", unit[g])] + (read(g - 2) if g >= 2 else [])) for g in range(len(unit))]
    prog, slot_of, begun = [], {}, 0
    for u in range(N):
        for e in range(nks[u] + 2):
            x = tile0[u] + e
            deps = [("LR", x), ("LQ", u)]
            if e == 0 and first[u] >= 2:
                deps += read(first[u] - 2)
            slot = (begun + e) % 4 if D == 64 else e % 3
            for g in slot_of.get(slot, []):
                deps += read(g)
            # who reads the tile: steps max(0, e - 2) .. e of the unit; D = 128 frees a unit's last two at its end
            slot_of[slot] = [first[u] + t for t in range(max(0, e - 2), min(e, nks[u] - 1) + 1)]
            prog.append((("G", x), deps))
        begun += nks[u] + 2
    progs["G"] = prog
    progs["PV"] = []
    for g, u in enumerate(unit):
        t = g - first[u]
        deps = [("LV", g)] + ([("P", owner(g), g)] if D == 64 else [("P", 0, g), ("P", 1, g)])
        if u > 0 and t < (2 if D == 64 else 1):
            deps.append(("EP", u - 1))
        progs["PV"].append((("PV", g), deps))
    # ---- softmax
    for w in (0, 1):
        prog = []
        for u in range(N):
            prog.append((("SEEN", w, u), [("LQ", u)]))
            for t in range(nks[u]):
                g = first[u] + t
                if D == 64 and owner(g) != w:
                    continue
                seen = [("S", g)] + [("G", tile0[u] + t + k) for k in range(3)]
                if D == 64:  # the scores lie in tensor memory until the weights are made, into the buffer of step g - 2
                    prog.append((("RD", w, g), seen + ([("PV", g - 2)] if g >= 2 else [])))
                    prog.append((("P", w, g), []))
                    continue
                prog.append((("RD", w, g), seen))
                prog.append((("X", w, g), []))  # the halves exchange their maxima; a rescaling waits for the P.V before
                prog.append((("P", w, g), [("X", 0, g), ("X", 1, g)] + ([("PV", g - 1)] if w == 0 and t else []) +
                             ([("PV", g - 2)] if g >= 2 else [])))
            last = first[u] + nks[u] - 1
            if w == (owner(last) if D == 64 else 0):
                prog.append((("EP", u), [("L", u)] + [("PV", first[u] + t) for t in range(nks[u])]))
            else:
                prog.append((("L", u), [("EP", u - 1)] if D == 64 and u > 0 else []))
        progs["sm%d" % w] = prog
    return progs


MIXES = [[1] * 9, [2] * 8, [1, 2, 1, 1, 3, 1, 1], [5, 1, 4, 1, 1], [16, 14, 2, 1, 3], [1], [7]]


@pytest.mark.parametrize("D,lag", [(64, 0), (128, 1)])
def test_no_schedule_stops(D, lag):
    for seed in range(200):
        rng = random.Random(seed)
        nks = MIXES[seed] if seed < len(MIXES) else [rng.choice([1, 1, 2, 3, 6]) for _ in range(rng.randint(1, 9))]
        ok, pc = _run(programs(D, nks, lag), rng)
        assert ok, (D, nks, seed, pc)


@pytest.mark.parametrize("D,lag", [(64, 3), (128, 2)])
def test_values_that_trail_too_far_are_caught(D, lag):
    assert not _run(programs(D, [1] * 9, lag), random.Random(0))[0]
