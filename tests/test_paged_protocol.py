"""The decode kernel's ring of key tiles on a model of mbarrier phases under
random schedules.

A barrier's wait for a parity returns as soon as the barrier's current phase
has the other parity, whichever phase that is.  The producer fills stage
g % NS with tile g once the stage's last tile has been given back, loads land
some time later; tile g goes to warp g % warps.  A warp that takes a tile must
find that tile, landed, in the stage."""

import random

import pytest


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
# the D = 64 kernel of longer entries: softmax warps that wait for a value tile
# ---------------------------------------------------------------------------
def with_dead_rows(progs, dead, build_first):
    """The roles of test_loader_protocol.py, where the softmax of the steps in `dead` needs its value tile landed before
    it hands over its weights, and builds the next unit's operands before that (build_first) or after."""
    progs = dict(progs)
    # the loader waits for the stages of K(t), R(t+1) and V(t-2) before it issues any of the three
    loader = progs["loader"]
    progs["loader"] = [(act, deps + ([d for a, more in loader[i + 1:i + 3] if a[0] in ("LR", "LV") for d in more]
                                     if act[0] == "LK" else [])) for i, (act, deps) in enumerate(loader)]
    for name in ("sm0", "sm1"):
        prog, out, i = progs[name], [], 0
        while i < len(prog):
            act, deps = prog[i]
            if act[0] == "P" and act[1] in dead:
                handed = (act, deps + [("LV", act[1])])
                if build_first and i + 1 < len(prog) and prog[i + 1][0][0] == "B":
                    out.append(prog[i + 1])
                    i += 1
                out.append(handed)
            else:
                out.append((act, deps))
            i += 1
        progs[name] = out
    return progs


MIXES = [[1] * 9, [2] * 8, [1, 2, 1, 1, 3, 1, 1], [5, 1, 4, 1, 1], [16, 14, 2, 1, 3]]


@pytest.mark.parametrize("nks", MIXES)
def test_value_waits_do_not_deadlock(nks):
    from test_loader_protocol import _programs, _run

    for seed in range(60):
        rng = random.Random(seed)
        dead = {g for g in range(sum(nks)) if rng.random() < 0.5} if seed else set(range(sum(nks)))
        ok, pc = _run(with_dead_rows(_programs(nks, 2, flush=True), dead, True), rng)
        assert ok, (nks, seed, pc)


def test_waiting_before_the_build_is_caught():
    from test_loader_protocol import _programs, _run

    ok, _ = _run(with_dead_rows(_programs([1] * 9, 2, flush=True), set(range(9)), False), random.Random(0))
    assert not ok
