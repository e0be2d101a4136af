"""The decode kernel's ring of key tiles on a model of mbarrier phases under
random schedules.

A barrier's wait for a parity returns as soon as the barrier's current phase
has the other parity, whichever phase that is.  The producer fills stage
g % NS with tile g once the stage's last tile has been given back, loads land
some time later; tile g goes to warp g % warps.  A warp that takes a tile must
find that tile, landed, in the stage."""

import random

import pytest

from test_loader_protocol import _programs, _run


class Bar:
    def __init__(self):
        self.phase = 0  # phases completed

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(NS, warps, tiles, rng):
    """None, or what went wrong."""
    full, empty = [Bar() for _ in range(NS)], [Bar() for _ in range(NS)]
    held = [None] * NS       # tile landed in the stage
    flying = []              # loads in flight
    made = 0
    at = list(range(warps))  # next tile of each warp
    taken = [False] * warps
    while made < tiles or flying or any(x < tiles for x in at):
        moves = []
        if made < tiles and empty[made % NS].passes(((made // NS) & 1) ^ 1):
            moves.append(("load", made))
        moves += [("land", g) for g in flying]
        for w in range(warps):
            if taken[w]:
                moves.append(("give", w))
            elif at[w] < tiles and full[at[w] % NS].passes((at[w] // NS) & 1):
                moves.append(("take", w))
        if not moves:
            return "deadlock"
        what, x = rng.choice(moves)
        if what == "load":
            if any(at[w] % NS == x % NS and taken[w] for w in range(warps)):
                return "overwritten while read"
            flying.append(x)
            made += 1
        elif what == "land":
            flying.remove(x)
            held[x % NS] = x
            full[x % NS].phase += 1
        elif what == "take":
            if held[at[x] % NS] != at[x]:
                return "another tile"
            taken[x] = True
        else:
            empty[at[x] % NS].phase += 1
            taken[x] = False
            at[x] += warps
    return None


@pytest.mark.parametrize("n", [3, 4])
def test_ring(n):
    """As many warps as stages (3 at D = 128, 4 at D = 64)."""
    for seed in range(300):
        rng = random.Random(seed)
        assert run(n, n, rng.randint(1, 40), rng) is None


def test_a_stage_shared_by_warps_is_caught():
    """Three stages and four warps: a warp does not see every phase of a stage."""
    assert any(run(3, 4, 40, random.Random(seed)) for seed in range(300))


# ---------------------------------------------------------------------------
# the loader of the kernels of longer entries, the other roles as programs of
# actions that wait for actions (test_loader_protocol.py)
# ---------------------------------------------------------------------------
def loader_program(nks, lag, NS, ahead, flush=True):
    """K, r and V tiles of a step are issued together, V `lag` tiles behind; a unit's queries are loaded behind the first
    step of the unit before (ahead) or at its head, behind (flush) that unit's last V tile."""
    prog, queued, g, nr, nv, tiles = [], [], 0, 0, 0, []  # tiles: of r, so far

    def v_wait():
        return [("PV", nv - NS)] if nv >= NS else []

    def issue_v():
        nonlocal nv
        prog.append((("LV", queued[0][0]), v_wait()))
        queued.pop(0)
        nv += 1

    def issue_r():
        nonlocal nr
        prog.append((("LR", nr), [("G", nr - NS)] if nr >= NS else []))
        nr += 1

    def built(u):  # the operands of unit u
        return [("B", p, u) for p in (0, 1)] if u > 0 else [("B0",)]

    if ahead:
        prog.append((("LQ", 0), []))
    for u, n in enumerate(nks):
        if not ahead:
            while flush and queued:
                issue_v()
            prog.append((("LQ", u), built(u - 1) if u > 0 else []))
        issue_r()
        issue_r()
        for t in range(n):
            # one wait for the three stages
            both = ([("S", g - NS)] if g >= NS else []) + ([("G", nr - NS)] if nr >= NS else [])
            queued.append((g, u))
            has_v = len(queued) > lag
            if has_v:
                both += v_wait()
            prog.append((("LK", g), both))
            prog.append((("LR", nr), []))
            nr += 1
            if has_v:
                prog.append((("LV", queued.pop(0)[0]), []))
                nv += 1
            g += 1
            if t == 0 and ahead and u + 1 < len(nks):
                prog.append((("LQ", u + 1), built(u)))
    while queued:
        issue_v()
    return prog


def programs64(nks, lag, flush=True):
    progs = _programs(nks, lag, True)
    progs["loader"] = loader_program(nks, lag, 4, True)
    progs["PV"] = [(act, [("LV", act[1])] + deps) for act, deps in progs["PV"]]
    return progs


def programs128(nks, lag, flush=True):
    """Two stages, three ring slots; both halves of the softmax take every step: one builds the next unit's operands
    behind a unit's last weights, the other writes the unit out."""
    N = len(nks)
    first = [sum(nks[:u]) for u in range(N)]
    unit = [u for u in range(N) for _ in range(nks[u])]
    tile0 = [first[u] + 2 * u for u in range(N)]
    last_read = {}  # r tile -> step behind whose reads (or the unit's end) its slot is free
    for u in range(N):
        for e in range(nks[u] + 2):
            last_read[tile0[u] + e] = first[u] + min(e, nks[u] - 1)

    def built(u):
        return [("B", p, u) for p in (0, 1)] if u > 0 else [("B0",)]

    progs = {"loader": loader_program(nks, lag, 2, False, flush)}
    progs["S"] = [(("S", g), [("LK", g)] + ([("RD0", g - 2), ("RD1", g - 2)] if g >= 2 else []) + built(unit[g]))
                  for g in range(len(unit))]
    prog, slot_of = [], {}
    for u in range(N):
        for e in range(nks[u] + 2):
            x, deps = tile0[u] + e, [("LR", tile0[u] + e)] + built(u)
            back = slot_of.get(e % 3)
            if back is not None:
                deps += [("RD0", last_read[back]), ("RD1", last_read[back])]
            slot_of[e % 3] = x
            prog.append((("G", x), deps))
    progs["G"] = prog
    progs["PV"] = [(("PV", g), [("LV", g), ("P0", g), ("P1", g)] + ([("EP", unit[g] - 1)] if unit[g] > 0 and
                    g == first[unit[g]] else [])) for g in range(len(unit))]
    for half in (0, 1):
        prog = [(("B0",), [("LQ", 0)])] if half else []
        for u in range(N):
            for t in range(nks[u]):
                g = first[u] + t
                prog.append((("RD%d" % half, g), [("S", g)] + [("G", tile0[u] + t + k) for k in range(3)]))
                # the two halves exchange their maxima; a rescaling waits for the P.V before
                prog.append((("X%d" % half, g), []))
                prog.append((("P%d" % half, g), [("X0", g), ("X1", g)] +
                             ([("PV", g - 1 if half == 0 and t else g - 2)] if g >= 2 or (half == 0 and t) else [])))
            if half == 0:
                prog.append((("EP", u), [("L", u)] + [("PV", first[u] + t) for t in range(nks[u])]))
            else:
                prog.append((("L", u), []))
                if u + 1 < N:
                    prog.append((("B", 0, u + 1), [("LQ", u + 1)]))
                    prog.append((("B", 1, u + 1), []))
        progs["sm%d" % half] = prog
    return progs


MIXES = [[1] * 9, [2] * 8, [1, 2, 1, 1, 3, 1, 1], [5, 1, 4, 1, 1], [16, 14, 2, 1, 3]]


@pytest.mark.parametrize("nks", MIXES)
@pytest.mark.parametrize("lag", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_the_loader_does_not_deadlock(D, lag, nks):
    for seed in range(40):
        ok, pc = _run((programs64 if D == 64 else programs128)(nks, lag), random.Random(seed))
        assert ok, (D, lag, nks, seed, pc)


@pytest.mark.parametrize("D,lag", [(64, 3), (128, 2)])
def test_values_held_back_are_caught(D, lag):
    """V tiles that trail too far."""
    ok, _ = _run((programs64 if D == 64 else programs128)([1] * 9, lag, flush=False), random.Random(0))
    assert not ok
