"""CPU pins of the paged memory's oracle, and the C entry points' argument
checks (none of which reaches a device)."""

import ctypes

import numpy as np
import pytest

from oracle import txl_oracle as O
from oracle.pages_oracle import Book, attend, spread, tolerance

INVALID, UNSUPPORTED, ALIAS = 1, 2, 3


def check(book):
    """Every live page is counted once per table entry, no entry is free, and
    entries past a slot's pages are -1."""
    count = [0] * len(book.refs)
    for s, row in enumerate(book.table):
        n = book.pages(s)
        assert all(p >= 0 for p in row[:n]) and all(p == -1 for p in row[n:])
        for p in row[:n]:
            count[p] += 1
    assert count == book.refs


def test_random_steps_keep_rows_and_counts():
    """Reserve, append, fork, free and compact in random order against a
    plain list of rows per slot."""
    rng = np.random.default_rng(0)
    book = Book(6, 5, 18, 16)
    pool = np.full((18, 1, 16, 1), np.nan)
    model = [[] for _ in range(6)]
    stamp = 0
    refused_some = shared_some = moved_some = False
    for _ in range(400):
        what = rng.integers(4)
        if what == 0:
            slots = [int(s) for s in rng.permutation(6)[:rng.integers(1, 6)]]
            counts = [int(c) for c in rng.integers(0, 20, len(slots))]
            cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
            new = np.arange(stamp, stamp + cu[-1], dtype=np.float64).reshape(-1, 1, 1)
            stamp += cu[-1]
            granted, src, dst, refused = book.reserve(slots, cu)
            refused_some |= refused
            shared_some |= any(a >= 0 for a in src)
            book.append(pool, slots, cu, granted, src, dst, new)
            for i, s in enumerate(slots):
                assert granted[i] in (0, counts[i])
                model[s] += new[cu[i]:cu[i] + granted[i], 0, 0].tolist()
        elif what == 1:
            a, d = int(rng.integers(6)), int(rng.integers(6))
            if book.fork([a], [d])[0]:
                model[d] = list(model[a])
        elif what == 2:
            s, keep = int(rng.integers(6)), int(rng.integers(-2, 40))
            book.free([s], [keep])
            model[s] = model[s][max(0, len(model[s]) - max(0, keep)):]
        else:
            _, src, dst = book.compact()
            moved_some |= bool(src)
            pool[dst] = pool[src]
        check(book)
        for s in range(6):
            assert book.gather(pool, s)[:, 0, 0].tolist() == model[s]
    assert refused_some and shared_some and moved_some


def test_attend_is_the_segment_attention():
    """With the memory in front the paged attention is relattn_forward."""
    rng = np.random.default_rng(1)
    n, m, H, D = 5, 7, 2, 6
    q, k, v = rng.normal(size=(n, H, D)), rng.normal(size=(n + m, H, D)), rng.normal(size=(n + m, H, D))
    r, u, vb = rng.normal(size=(n + m, H, D)), rng.normal(size=(H, D)), rng.normal(size=(H, D))
    o, lse, _ = attend(q, k, v, r, u, vb, D ** -0.5)
    eo, el = O.relattn_forward(q[None], k[None], v[None], r, u, vb, m)
    np.testing.assert_allclose(o, eo[0], rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse, el[0], rtol=0, atol=1e-12)


def test_attend_without_a_row():
    """Queries at negative positions see nothing."""
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(4, 1, 3)), rng.normal(size=(2, 1, 3))
    o, lse, _ = attend(q, k, k, k, np.zeros((1, 3)), np.zeros((1, 3)), 1.0)
    assert (o[:2] == 0).all() and np.isneginf(lse[0, :2]).all()
    np.testing.assert_allclose(o[2], k[0], atol=1e-15)
    assert np.isfinite(lse[0, 2:]).all()


def test_tolerance_covers_rounded_operands():
    """Rounding q + u, q + v, the distance term and the weights to bf16 stays
    within the first-order bound."""
    import torch

    rng = np.random.default_rng(3)
    bf = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731
    n, L, D = 3, 40, 64
    q, k, v, r = (bf(rng.normal(size=(x, 1, D))) for x in (n, L, L, L))
    u, vb = rng.normal(size=(1, D)), rng.normal(size=(1, D))
    o, lse, do, dl = tolerance(q, k, v, r, u, vb, 0.125, 2.0 ** -8, 2, 2.0 ** -8)

    def rounded(shift):
        got = np.zeros_like(o)
        for t in range(n):
            m = L - n + t
            z = bf(q[t, 0] + u[0]) @ k[:m + 1, 0].T + bf(bf(q[t, 0] + vb[0]) @ np.roll(r, shift, 0)[m::-1, 0].T)
            w = np.exp(0.125 * z - (0.125 * z).max())
            got[t, 0] = bf(bf(w) @ v[:m + 1, 0] / w.sum())
            if shift == 0:
                assert abs((0.125 * z).max() + np.log(w.sum()) - lse[0, t]) <= dl[0, t]
        return got

    assert (np.abs(rounded(0) - o) <= do).all()
    # The elements' worst case is wide; what independent roundings leave of
    # the whole is not, and that bound tells a distance that is off by one.
    room = spread(q, k, v, r, u, vb, 0.125, 2.0 ** -8, 2.0 ** -8)
    assert ((rounded(0) - o) ** 2).sum() <= room < ((rounded(1) - o) ** 2).sum() / 100


@pytest.mark.parametrize("scale", [0.0, 0.125, -0.2, 1.0])
def test_spread_is_what_roundings_leave(scale):
    """Over many draws the squared error is below the bound, and not far below."""
    import torch

    rng = np.random.default_rng(4)
    bf = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731
    n, L, D = 1, 60, 64
    got = room = 0.0
    for _ in range(40):
        q, k, v, r = (bf(rng.normal(size=(x, 1, D))) for x in (n, L, L, L))
        r = 0.5 * r
        u, vb = 0.3 * rng.normal(size=(1, D)), 0.3 * rng.normal(size=(1, D))
        o, _, _ = attend(q, k, v, r, u, vb, scale)
        z = scale * (bf(q[0, 0] + u[0]) @ k[:, 0].T + bf(bf(q[0, 0] + vb[0]) @ r[::-1, 0].T))
        w = np.exp(z - z.max())
        got += ((bf(bf(w) @ v[:, 0] / w.sum()) - o[0, 0]) ** 2).sum()
        room += spread(q, k, v, r, u, vb, scale, 2.0 ** -8, 2.0 ** -8)
    assert 0.1 * room <= got <= room


@pytest.fixture(scope="module")
def lib():
    import test_library_cpu

    test_library_cpu._build_if_missing()
    import transformer_xl_relative_txl_gb300 as txl

    return txl


def book_struct(txl, **change):
    f = dict(table=0x10000, start=0x20000, rows=0x30000, refs=0x40000, n_slots=4, max_pages=8, n_pages=64, page_rows=16)
    f.update(change)
    return ctypes.byref(txl._PageBook(*[f[n] for n, _ in txl._PageBook._fields_]))


# Made-up addresses, 256 MiB apart: no check reads what they point to.
A = {x: 0x10000000 * (i + 1) for i, x in enumerate("slots cu granted src dst ok kp vp kn vn q r u vb o lse ws keep".split())}


def calls(txl, **c):
    """Every entry point on the made-up addresses; only refused or empty calls are made of them."""
    g = lambda x: c.get(x, A.get(x))  # noqa: E731
    book = c.get("book", book_struct(txl, **c.get("book_change", {})))
    n, T, H, D, dt = c.get("n", 2), c.get("T", 10), c.get("H", 2), c.get("D", 64), c.get("dtype", 1)
    L = txl.lib
    return {
        "reserve": lambda: L.txl_pages_reserve(book, g("slots"), g("cu"), n, g("granted"), g("src"), g("dst"), None),
        "append": lambda: L.txl_pages_append(book, g("kp"), g("vp"), H, D, g("slots"), g("cu"), n, g("granted"),
                                             g("src"), g("dst"), g("kn"), g("vn"), T, dt, None),
        "copy": lambda: L.txl_pages_copy(g("kp"), g("vp"), c.get("n_pages", 64), c.get("page_elems", 2048), g("src"),
                                         g("dst"), n, dt, None),
        "fork": lambda: L.txl_pages_fork(book, g("src"), g("dst"), n, g("ok"), None),
        "free": lambda: L.txl_pages_free(book, g("slots"), g("keep"), n, None),
        "compact": lambda: L.txl_pages_compact(book, g("granted"), g("src"), g("dst"), g("ok"), None),
        "attend": lambda: L.txl_relattn_forward_paged(
            g("q"), g("kp"), g("vp"), book, g("slots"), g("cu"), n, T, c.get("max_new", 4), g("r"), g("u"), g("vb"),
            g("o"), g("lse"), H, D, c.get("n_r", 20), c.get("scale", 0.125), dt, c.get("o_dtype", 1), g("ws"),
            c.get("ws_bytes", 200 << 20), None),
    }


BOOKED = ("reserve", "append", "fork", "free", "compact", "attend")
REFUSED = [
    (BOOKED, dict(book=None), INVALID),
    (BOOKED, dict(book_change=dict(table=None)), INVALID),
    (BOOKED, dict(book_change=dict(start=0x20002)), INVALID),
    (("reserve", "fork", "free", "compact"), dict(book_change=dict(refs=None)), INVALID),
    (BOOKED, dict(book_change=dict(n_slots=0)), INVALID),
    (BOOKED, dict(book_change=dict(page_rows=-16)), INVALID),
    (BOOKED, dict(book_change=dict(page_rows=24)), UNSUPPORTED),
    (BOOKED, dict(book_change=dict(page_rows=8)), UNSUPPORTED),
    (BOOKED, dict(book_change=dict(page_rows=2048)), UNSUPPORTED),
    (BOOKED, dict(book_change=dict(n_slots=16385)), UNSUPPORTED),
    (BOOKED, dict(book_change=dict(max_pages=1 << 27)), UNSUPPORTED),
    (BOOKED, dict(book_change=dict(rows=0x20004)), ALIAS),
    (("reserve", "append", "copy", "fork", "free", "attend"), dict(n=-1), INVALID),
    (("reserve", "append", "fork", "free", "attend"), dict(n=16385), UNSUPPORTED),
    (("reserve", "append", "free", "attend"), dict(slots=None), INVALID),
    (("reserve", "append", "attend"), dict(cu=None), INVALID),
    (("reserve", "append", "attend"), dict(cu=A["cu"] + 2), INVALID),
    (("reserve", "append", "compact"), dict(granted=None), INVALID),
    (("reserve", "append", "copy", "fork", "compact"), dict(src=None), INVALID),
    (("reserve",), dict(granted=A["slots"] + 4), ALIAS),
    (("reserve", "fork", "compact"), dict(dst=0x30000), ALIAS),
    (("free",), dict(keep=0x20004), ALIAS),
    (("fork",), dict(ok=A["src"]), ALIAS),
    (("append", "copy", "attend"), dict(dtype=2), INVALID),
    (("append",), dict(T=-1), INVALID),
    (("append",), dict(D=257), UNSUPPORTED),
    (("append", "copy", "attend"), dict(kp=None), INVALID),
    (("append", "copy"), dict(kp=A["kp"] + 1), INVALID),
    (("append", "copy"), dict(vp=A["kp"] + 64), ALIAS),
    (("append",), dict(kn=A["kp"] + 64), ALIAS),
    (("append",), dict(src=A["src"], dst=None), INVALID),
    (("copy",), dict(page_elems=0), INVALID),
    (("copy",), dict(n_pages=0), INVALID),
    (("attend",), dict(T=-1), INVALID),
    (("attend",), dict(max_new=-1), INVALID),
    (("attend",), dict(n_r=0), INVALID),
    (("attend",), dict(scale=float("nan")), INVALID),
    (("attend",), dict(D=40), UNSUPPORTED),
    (("attend",), dict(dtype=0, o_dtype=1), UNSUPPORTED),
    (("attend",), dict(dtype=0, o_dtype=0, D=257), UNSUPPORTED),
    (("attend",), dict(kp=A["kp"] + 2), INVALID),
    (("attend",), dict(o=A["o"] + 8), INVALID),
    (("attend",), dict(ws=None), INVALID),
    (("attend",), dict(ws=A["ws"] + 16), INVALID),
    (("attend",), dict(ws_bytes=16), INVALID),
    (("attend",), dict(o=A["q"]), ALIAS),
    (("attend",), dict(lse=A["o"]), ALIAS),
    (("attend",), dict(ws=A["q"] - 0x200), ALIAS),
    (("attend",), dict(lse=0x30000), ALIAS),
]


@pytest.mark.parametrize("names,change,want", REFUSED, ids=[f"{i}" for i in range(len(REFUSED))])
def test_refusals(lib, names, change, want):
    for name in names:
        assert calls(lib, **change)[name]() == want, name


def test_empty_calls(lib):
    for name in ("reserve", "append", "copy", "fork", "free", "attend"):
        assert calls(lib, n=0)[name]() == 0, name
    assert calls(lib, T=0)["append"]() == 0
    assert calls(lib, T=0)["attend"]() == 0
    assert calls(lib, max_new=0)["attend"]() == 0
    assert lib.lib.txl_relattn_paged_workspace_bytes(-1, 1, 1, 64, 1) == 0
    assert lib.txl_status_string(6) == "TXL_ERR_PAGES"


def test_binding_refuses(lib):
    import torch

    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    book = dict(table=z(2, 3), start=z(2), rows=z(2), refs=z(8))
    with pytest.raises(ValueError):  # host memory
        lib.txl_pages_reserve(book, 16, z(1), z(2), z(1), z(1), z(1))
    with pytest.raises(ValueError):
        lib.txl_pages_free(dict(book, start=z(3)), 16, z(1))
    with pytest.raises(ValueError):
        lib.txl_pages_copy(torch.zeros(8, 1, 16, 4), torch.zeros(8, 1, 16, 5), z(1), z(1))
    with pytest.raises(TypeError):  # no tensor
        lib.txl_pages_reserve(book, 16, [0], z(2), z(1), z(1), z(1))
    with pytest.raises(TypeError):
        lib.txl_pages_compact(book, 16, None, z(8), z(8), z(1))
    with pytest.raises(TypeError):
        lib.txl_relattn_forward_paged(z(1), z(1), z(1), book, 0, z(2), z(1), z(1), z(1), z(1), z(1))


def steps(start, rows, n, first, count, BK):
    """Key steps that queries first .. first + count - 1 of n can see."""
    x = start + rows - n + min(first + count, n) - 1
    return [start // BK] if x < start else list(range(start // BK, x // BK + 1))


@pytest.mark.parametrize("kind,D", [(0, 64), (0, 128), (1, 64), (2, 40)])
def test_every_step_has_one_cta(lib, kind, D):
    """The division of the paged attention: every key step of every unit on one CTA, the pieces of a unit numbered in
    key order on consecutive CTAs, their places distinct, and no CTA with much more than its share."""
    rng = np.random.default_rng(kind + D)
    BK = 32 if kind == 2 or (kind == 0 and D == 128) else 64
    tile = (0, 128, 16)[kind]
    unit = (4, 7, 3)[kind]  # cost of a unit besides its steps, in half steps
    for trial in range(120):
        n = int(rng.integers(1, [2, 5, 60][trial % 3] + 1))
        H = int(rng.integers(1, 9))
        start = rng.integers(0, [1, 16, 1024][trial % 3], n)
        rows = (10 ** rng.uniform(0, 4.5, n)).astype(int) * (rng.random(n) > 0.1)
        new = rng.integers(1, 5, n) if kind == 0 else rng.integers(5 if kind == 1 else 1, 700, n)
        ctas = int(rng.choice([1, 7, 152, 304]))
        got = lib.txl_debug_paged_pieces(kind, D, H, start, rows, new, ctas)
        assert (np.diff(got[:, 0]) >= 0).all() and got[:, 0].max() < ctas
        units, places, load = {}, set(), np.zeros(ctas)
        for c, i, h, qt, t0, nks, first, index, pieces, place in got.tolist():
            assert nks > 0 and first + index == c and 0 <= index < pieces
            units.setdefault((i, h, qt), []).append((index, t0, nks, pieces))
            if pieces > 1:
                assert place not in places and place // 2 == c
                places.add(place)
            load[c] += 2 * nks + unit
        count = {}
        for (i, h, qt), p in units.items():
            want = steps(start[i], rows[i], new[i], tile * qt, tile or 4, BK)
            assert [x[0] for x in p] == list(range(p[0][3]))
            assert [t for _, t0, nks, _ in p for t in range(t0, t0 + nks)] == want
            count[i] = count.get(i, 0) + 1
            first_pieces = [c for c, *r in got.tolist() if tuple(r[:3]) == (i, h, qt)] if n < 4 else []
            assert first_pieces == sorted(set(first_pieces))
        for i in range(n):
            assert count[i] == H * (-(-int(new[i]) // tile) if kind else 1)
        # a CTA's range, a step more at its end, and what a unit costs besides its steps at each end
        whole = sum(2 * x[2] for p in units.values() for x in p) + unit * len(units)
        assert load.max() <= whole / min(ctas, max(1, whole // 4)) + 2 + 2 * unit


def test_one_split_unit_starts_per_cta(lib):
    """The merge counters: no CTA has the first piece of two split units."""
    got = lib.txl_debug_paged_pieces(0, 64, 16, [3] * 40, list(range(100, 4100, 100)), [1] * 40, 304)
    firsts = [c for c, i, h, qt, t0, nks, first, index, pieces, place in got.tolist() if pieces > 1 and index == 0]
    assert len(firsts) == len(set(firsts)) and len(firsts) > 100
