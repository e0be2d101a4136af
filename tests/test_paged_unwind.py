"""The decode kernel's producer and consumers when a wait runs out: a model of
units published two deep and tiles in a ring of stages, in which the producer
gives up a stage that a slow consumer holds.  Whatever the schedule, a consumer
finds the tile that belongs to the place in its unit, or none.

What the producer does behind the tile that it gave up is read from the kernel's
source."""

import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_xl_relative_txl_gb300",
                    "csrc")


def block_end(text, at):
    """Behind the block that opens at or after `at`."""
    depth = 0
    for i in range(text.index("{", at), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise ValueError("no end")


def leaves_at_once():
    """Whether the producer's loop over units ends where its loop over a unit's tiles gave up."""
    with open(os.path.join(CSRC, "paged_decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("for (int t = w.p.t0; t < w.p.t0 + w.p.nks")
    return re.match(r"\s*if \(!ok( \|\| \w+)?\) break;", text[block_end(text, start):]) is not None


def run(NS, nks, gives_up, leaves, rng):
    """Units of nks[u] key tiles.  The producer's wait for the stage of tile number `gives_up` runs out.  None, or what
    went wrong."""
    first = [sum(nks[:u]) for u in range(len(nks))]
    loaded = {}              # tile number -> (unit, tile) as loaded
    published = []           # units that the consumers may read
    # The producer's program: the actions it takes, given that the wait for tile `gives_up` fails.
    program, g = [], 0
    for u, n in enumerate(nks):
        program.append(("publish", u))
        for t in range(n):
            if g == gives_up:
                gives_up = -1
                program.append(("gave up",))
                break
            program.append(("load", g, (u, t)))
            g += 1
        if program[-1] == ("gave up",) and leaves:
            break
    # Consumer w takes the tiles with number % NS == w of each published unit, in order.
    takes = [[(u, t, first[u] + t) for u, n in enumerate(nks) for t in range(n) if (first[u] + t) % NS == w]
             for w in range(NS)]
    at, given, pc = [0] * NS, [0] * NS, 0
    while True:
        moves = []
        if pc < len(program):
            step = program[pc]
            if step[0] == "publish":  # two units deep: every warp has read the one before the last
                if len(published) < 2 or all(at[w] == len(takes[w]) or takes[w][at[w]][0] >= published[-1]
                                             for w in range(NS)):
                    moves.append("produce")
            elif step[0] == "load":
                if given[step[1] % NS] >= step[1] // NS:
                    moves.append("produce")
            else:
                moves.append("produce")
        for w in range(NS):
            if at[w] < len(takes[w]) and takes[w][at[w]][0] in published and takes[w][at[w]][2] in loaded:
                moves.append(w)
        if not moves:
            return None  # finished, or waits that run out
        m = rng.choice(moves)
        if m == "produce":
            step = program[pc]
            if step[0] == "publish":
                published.append(step[1])
            elif step[0] == "load":
                loaded[step[1]] = step[2]
            pc += 1
        else:
            u, t, number = takes[m][at[m]]
            if loaded[number] != (u, t):
                return "tile %r taken as %r" % (loaded[number], (u, t))
            at[m] += 1
            given[m] += 1


def wrong(leaves, NS):
    for seed in range(400):
        rng = random.Random(seed)
        nks = [rng.randint(1, 9) for _ in range(rng.randint(1, 5))]
        bad = run(NS, nks, rng.randrange(sum(nks)), leaves, rng)
        if bad:
            return bad
    return None


@pytest.mark.parametrize("NS", [3, 4])
def test_no_tile_is_taken_for_another(NS):
    assert wrong(leaves_at_once(), NS) is None


@pytest.mark.parametrize("NS", [3, 4])
def test_going_on_with_the_next_unit_is_caught(NS):
    assert "taken as" in wrong(False, NS)
