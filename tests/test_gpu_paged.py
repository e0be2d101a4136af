"""The paged memory on the GPU: every step of the book and of the pools
against the list-and-loop oracle, the attention against float64, and the
calls run together as a server would."""

import numpy as np
import pytest
import torch

from gpu_util import BF16_REL_L2
from oracle.pages_oracle import Book, spread, tolerance

pytestmark = pytest.mark.gpu

NAMES = ("table", "start", "rows", "refs")


@pytest.fixture(scope="module")
def txl():
    import transformer_xl_relative_txl_gb300 as m

    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def to_gpu(book):
    return {x: ints(getattr(book, x)) for x in NAMES}


def same(dev, book):
    for x in NAMES:
        assert dev[x].tolist() == getattr(book, x), x


def cu_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(int).tolist()


def filled(rng, spans, P, H, D, dtype, spare=5, n_slots=None, leftover=float("nan")):
    """A book and pools whose slot i holds rows live rows after start dead ones (spans: start, rows), pages in random
    order; what is not live holds `leftover`."""
    n_slots = n_slots or len(spans)
    need = [-(-(a + m) // P) if m else 0 for a, m in spans]
    max_pages = max(need + [1]) + 3
    book = Book(n_slots, max_pages, sum(need) + spare, P)
    ids = rng.permutation(len(book.refs)).tolist()
    pools = [torch.full((len(book.refs), H, P, D), leftover) for _ in range(2)]
    for s, (a, m) in enumerate(spans):
        for j in range(need[s]):
            p = ids.pop()
            book.table[s][j] = p
            book.refs[p] = 1
            lo, hi = max(a - j * P, 0), min(a + m - j * P, P)
            for pool in pools:
                pool[p, :, lo:hi] = torch.from_numpy(rng.normal(size=(H, hi - lo, D))).float()
        book.start[s], book.rows[s] = (a, m) if m else (0, 0)
    return book, [x.to(dtype) for x in pools]


def workspace(txl, n, T, H, D, dtype):
    return torch.full((txl.txl_relattn_paged_workspace_bytes(n, T, H, D, dtype),), 255, dtype=torch.uint8, device="cuda")


def attend_case(txl, rng, spans, counts, P, H, D, dtype, o_dtype=None, slots=None, scale=None, leftover=float("nan"),
                tail=0, max_new=None, n_r_extra=0):
    """Runs txl_relattn_forward_paged and holds o, lse to the oracle; returns the call's arguments."""
    book, pools = filled(rng, spans, P, H, D, dtype, leftover=leftover)
    slots = list(range(len(spans))) if slots is None else slots
    cu = cu_of(counts)
    T = cu[-1] + tail
    n_r = max([m for _, m in spans] + [1]) + n_r_extra
    q, r = (torch.from_numpy(rng.normal(size=(x, H, D))).float().to(dtype) for x in (T, n_r))
    r = r * 0.5
    u, vb = (torch.from_numpy(0.3 * rng.normal(size=(H, D))).float() for _ in range(2))
    scale = D ** -0.5 if scale is None else scale
    dev = to_gpu(book)
    o = torch.full((T, H, D), 7.0, device="cuda", dtype=o_dtype or dtype)
    lse = torch.full((H, T), 7.0, device="cuda")
    k, v = (x.cuda() for x in pools)
    args = (q.cuda(), k, v, dev, ints(slots), ints(cu), r.cuda(), u.cuda(), vb.cuda(), o,
            workspace(txl, len(slots), T, H, D, dtype))
    kw = dict(lse=lse, max_new=max_new or max(counts + [1]), scale=scale)
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == 0
    same(dev, book)
    got, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    # Operands: q + u, q + v, the distance term and the weights are each rounded once at most in bf16; in fp32 a
    # product chain of D terms and one of all rows carry one rounding per term.
    longest = max([m for _, m in spans] + [1])
    if dtype == torch.bfloat16:
        step, terms = 2.0 ** -8, 2
    else:
        step, terms = 2.0 ** -24, 2 * D + longest
    out = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[o.dtype]
    off = room = 0.0
    for i, s in enumerate(slots):
        rows = slice(cu[i], cu[i + 1])
        kk, vv = (book.gather(x.float().numpy(), s) for x in pools)
        want, want_l, do, dl = tolerance(q[rows].float().numpy(), kk, vv, r.float().numpy(), u.numpy(), vb.numpy(),
                                         scale, step, terms, out)
        e = np.abs(got[rows] - want)
        assert np.isfinite(got[rows]).all()
        assert (e <= do + 1e-7).all(), (i, (e - do).max())
        none = np.isneginf(want_l)
        assert (np.isneginf(got_l[:, rows]) == none).all()
        assert (np.abs(got_l[:, rows][~none] - want_l[~none]) <= dl[~none] + 1e-6).all()
        if dtype == torch.bfloat16:  # the elements' worst case is wide: the whole is held to what roundings leave
            off += (e ** 2).sum()
            room += spread(q[rows].float().numpy(), kk, vv, r.float().numpy(), u.numpy(), vb.numpy(), scale, step, out)
    # 1e-9: fp32 sums where nothing is rounded to bf16 (an output of fp32 that is one value row)
    assert off <= room + 1e-9 * T * H * D
    assert (got[cu[-1]:] == 7.0).all() and (got_l[:, cu[-1]:] == 7.0).all()
    return args, kw


BF, F32 = torch.bfloat16, torch.float32

ONE_TOKEN = [
    # page rows, H, D, (start, rows) of each slot
    (16, 1, 64, [(0, 1)]),
    (16, 2, 64, [(0, 16), (15, 1), (15, 2), (3, 64)]),
    (64, 3, 64, [(63, 1), (0, 64), (1, 63), (1, 64), (17, 300), (0, 513)]),
    (128, 2, 128, [(100, 29), (5, 200), (0, 130), (127, 258)]),
    (32, 8, 128, [(a, 1 + 37 * a) for a in range(12)]),
    (1024, 2, 64, [(1000, 400), (0, 1024), (512, 1)]),
    (16, 16, 64, [(i % 16, 40 + 3 * i) for i in range(33)]),
    # many key tiles per CTA: each stage of the ring is filled over and over
    (32, 16, 128, [(i % 32, 2000 + 31 * i) for i in range(16)]),
    (64, 16, 64, [(i % 64, 4000 + 61 * i) for i in range(16)]),
    (16, 1, 128, [(7, 5000)]),
]


@pytest.mark.parametrize("P,H,D,spans", ONE_TOKEN, ids=[f"P{c[0]}H{c[1]}D{c[2]}n{len(c[3])}" for c in ONE_TOKEN])
def test_one_token_each(txl, P, H, D, spans):
    attend_case(txl, np.random.default_rng(P + D), spans, [1] * len(spans), P, H, D, BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 4, 5, 8])
def test_few_tokens(txl, n, D):
    """Several new tokens a sequence, with rows that see nothing (more tokens than rows) and unlike counts."""
    spans = [(0, n), (3, 70), (15, 1), (0, 257), (9, 0), (2, n - 1)]
    counts = [n, n - 1, n, n, 1, n]
    attend_case(txl, np.random.default_rng(n), spans, counts, 16, 2, D, BF)


CHUNKS = [
    # page rows, H, D, spans, counts
    (64, 2, 64, [(0, 128), (0, 127), (0, 129), (63, 130)], [128, 127, 129, 130]),
    (16, 1, 64, [(5, 300), (0, 64), (15, 700), (1, 9)], [200, 64, 1, 9]),
    (32, 2, 128, [(31, 290), (0, 33), (4, 65)], [131, 33, 1]),
    (128, 3, 64, [(77, 450), (0, 1), (0, 20)], [256, 1, 30]),
    (256, 1, 128, [(200, 600), (0, 600)], [600, 10]),
    (64, 2, 64, [(0, 0), (0, 40), (60, 70)], [0, 40, 0]),
    (16, 2, 64, [(3, 100), (0, 0), (15, 30)], [150, 40, 200]),
    (16, 2, 128, [(3, 100), (0, 0), (15, 30)], [150, 40, 200]),
    # many tiles a head, cut in the middle of one
    (64, 1, 64, [(9, 3500), (0, 50)], [2401, 50]),
    (32, 1, 128, [(9, 3300), (0, 50)], [2111, 2]),
]


@pytest.mark.parametrize("P,H,D,spans,counts", CHUNKS, ids=[f"P{c[0]}H{c[1]}D{c[2]}n{max(c[4])}" for c in CHUNKS])
@pytest.mark.parametrize("o_dtype", [BF, F32])
def test_chunks(txl, P, H, D, spans, counts, o_dtype):
    attend_case(txl, np.random.default_rng(P + D), spans, counts, P, H, D, BF, o_dtype=o_dtype, tail=3, n_r_extra=5)


@pytest.mark.parametrize("D", [1, 7, 40, 64, 128, 200, 256])
def test_float32(txl, D):
    spans, counts = [(3, 60), (0, 1), (15, 90), (0, 5), (0, 0)], [20, 1, 33, 9, 2]
    attend_case(txl, np.random.default_rng(D), spans, counts, 16, 2, D, F32, tail=2)


MANY = {  # more than 32 units a block, more entries than threads, entries of the other kernel and empty ones between
    "decode": (BF, 64, 16, 700, lambda rng: rng.choice([0, 1, 1, 1, 2, 7])),
    "decode128": (BF, 128, 16, 700, lambda rng: rng.choice([0, 1, 1, 1, 4])),
    "tiles": (BF, 64, 16, 450, lambda rng: rng.choice([0, 1, 5, 6, 9, 130], p=[.1, .1, .3, .3, .19, .01])),
    "tiles128": (BF, 128, 16, 450, lambda rng: rng.choice([0, 3, 5, 8], p=[.05, .05, .5, .4])),
    "float32": (F32, 8, 32, 560, lambda rng: rng.choice([0, 1, 3, 20])),
}


@pytest.mark.parametrize("case", MANY)
def test_many_units(txl, case):
    dtype, D, H, n, draw = MANY[case]
    rng = np.random.default_rng(n + D)
    counts = [int(draw(rng)) for _ in range(n)]
    counts[40:120] = [0] * 80  # the lists that a warp reads are empty for a while
    spans = [(int(rng.integers(16)), c + int(rng.integers(0, 60))) for c in counts]
    attend_case(txl, rng, spans, counts, 16, H, D, dtype, tail=3)


@pytest.mark.parametrize("dtype,D,counts", [(BF, 64, [1, 1]), (BF, 128, [3, 2]), (BF, 64, [90, 20]), (BF, 128, [70, 9]),
                                            (F32, 24, [5, 1])])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scale(txl, dtype, D, counts, scale):
    attend_case(txl, np.random.default_rng(7), [(2, 100), (0, 130)], counts, 32, 2, D, dtype, scale=scale)


@pytest.mark.parametrize("dtype,D,counts", [(BF, 64, [1, 1, 1]), (BF, 64, [80, 20, 1]), (BF, 128, [80, 20, 1]),
                                            (F32, 8, [6, 1, 3])])
@pytest.mark.parametrize("leftover", [float("inf"), -float("inf"), 3e38])
def test_leftovers(txl, dtype, D, counts, leftover):
    """What pages hold outside the live rows is never used (NaN in every other test)."""
    attend_case(txl, np.random.default_rng(8), [(5, 100), (0, 30), (15, 1)], counts, 16, 2, D, dtype, leftover=leftover)


@pytest.mark.parametrize("counts,max_new", [([1, 1, 1], 4), ([2, 1, 3], 600), ([70, 70, 1], 128)])
def test_slots_in_any_order(txl, counts, max_new):
    """Entries name slots out of order, one of them twice; max_new above what comes."""
    attend_case(txl, np.random.default_rng(9), [(1, 90), (2, 200), (3, 80), (0, 77)], counts, 32, 2, 64, BF,
                slots=[2, 0, 2], max_new=max_new)


@pytest.mark.parametrize("dtype,D,new", [(BF, 64, 1), (BF, 64, 300), (BF, 128, 1), (BF, 128, 200), (F32, 16, 40)])
def test_refused_entries_stay(txl, dtype, D, new):
    """Entries out of range leave their rows as they were; the others are served, and the status says so."""
    rng = np.random.default_rng(11)
    args, kw = attend_case(txl, rng, [(0, new + 20)] * 6, [new] * 6, 16, 2, D, dtype)
    good = args[9].clone()
    q, k, v, dev, slots, cu, r, u, vb, o, ws = args
    bad = slots.clone()
    bad[0], bad[2] = -1, 6
    dev["rows"][3] = len(r) + 1
    dev["start"][4] = 16
    o.fill_(7.0)
    txl.txl_relattn_forward_paged(q, k, v, dev, bad, cu, r, u, vb, o, ws, **kw)
    assert txl.txl_get_device_status() == 6
    assert txl.txl_get_device_status() == 0
    rows = [slice(i * new, (i + 1) * new) for i in range(6)]
    for i in (0, 2, 3, 4):
        assert (o[rows[i]] == 7.0).all()
    # Which CTA has which key steps goes by the whole batch: the others' results may round elsewhere, and two results
    # that are each within the tolerance of the exact one are within twice that of each other.
    near = lambda a, b: ((a.double() - b.double()).norm() / b.double().norm()).item() <= 2 * BF16_REL_L2  # noqa: E731
    for i in (1, 5):
        assert near(o[rows[i]], good[rows[i]])
    # an entry with more rows than max_new is refused, as is one past q's end
    dev["rows"].fill_(new + 20)
    dev["start"].fill_(0)
    o.fill_(7.0)
    far = cu.clone()
    far[6] = len(q) + 1
    txl.txl_relattn_forward_paged(q, k, v, dev, slots, far, r, u, vb, o, ws, **kw)
    assert txl.txl_get_device_status() == 6
    assert (o[rows[5]] == 7.0).all() and near(o[:5 * new], good[:5 * new])


@pytest.mark.parametrize("dtype,D,new", [(BF, 64, 1), (BF, 128, 90), (BF, 64, 90), (F32, 16, 5)])
def test_bad_page_is_not_followed(txl, dtype, D, new):
    rng = np.random.default_rng(12)
    args, kw = attend_case(txl, rng, [(0, 130)] * 3, [new] * 3, 16, 2, D, dtype)
    good = args[9].clone()
    args[3]["table"][1, 2] = 10 ** 8
    args[3]["table"][1, 5] = -7
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == 6
    keep = torch.ones(3 * new, dtype=torch.bool, device="cuda")
    keep[new:2 * new] = False
    assert torch.equal(args[9][keep], good[keep])


@pytest.mark.parametrize("dtype,D,counts", [(BF, 64, [1] * 5), (BF, 128, [1] * 5), (BF, 64, [200, 1, 3, 128, 1]),
                                            (BF, 128, [200, 1, 3, 128, 1]), (F32, 40, [200, 1, 3, 128, 1])])
def test_the_same_bits_every_time(txl, dtype, D, counts):
    args, kw = attend_case(txl, np.random.default_rng(13), [(0, 700), (4, 900), (1, 260), (0, 300), (15, 1200)], counts,
                           16, 4, D, dtype)
    first, lse = args[9].clone(), kw["lse"].clone()
    for _ in range(5):
        args[10].fill_(0x5a)
        args[9].fill_(1.0)
        txl.txl_relattn_forward_paged(*args, **kw)
        assert torch.equal(args[9], first) and torch.equal(kw["lse"], lse)


def test_two_streams_at_once(txl):
    """Two calls in flight, each with a workspace of its own."""
    rng = np.random.default_rng(14)
    cases = [attend_case(txl, rng, [(0, 900), (4, 1500)], [150, 1], 64, 4, 64, BF),
             attend_case(txl, rng, [(0, 2000), (4, 1500)], [1, 1], 64, 4, 64, BF)]
    want = [c[0][9].clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (args, kw), s in zip(cases, streams):
            with torch.cuda.stream(s):
                args[9].fill_(0.0)
                txl.txl_relattn_forward_paged(*args, **kw)
    torch.cuda.synchronize()
    for (args, _), w in zip(cases, want):
        assert torch.equal(args[9], w)


def test_the_segment_forward(txl):
    """Memory in front, one length: the paged call and txl_relattn_forward give the same attention up to the roundings
    each allows itself."""
    rng = np.random.default_rng(15)
    B, W, M, H, D, P = 3, 130, 70, 2, 64, 64
    book, pools = filled(rng, [(0, M + W)] * B, P, H, D, BF)
    q, r = (torch.from_numpy(rng.normal(size=(x, H, D))).to(BF).cuda() for x in (B * W, M + W))
    u, vb = (torch.from_numpy(rng.normal(size=(H, D))).float().cuda() for _ in range(2))
    k, v = (torch.stack([torch.from_numpy(book.gather(x.float().numpy(), s)) for s in range(B)]).to(BF).cuda()
            for x in pools)
    a = torch.empty(B, W, H, D, device="cuda")
    txl.txl_relattn_forward(q.view(B, W, H, D), k, v, r, u, vb, a)
    b = torch.empty(B * W, H, D, device="cuda")
    txl.txl_relattn_forward_paged(q, pools[0].cuda(), pools[1].cuda(), to_gpu(book), ints([0, 1, 2]),
                                  ints([0, W, 2 * W, 3 * W]), r, u, vb, b, workspace(txl, B, B * W, H, D, BF),
                                  max_new=W)
    assert ((a.view_as(b) - b).norm() / a.norm()).item() <= 2 * BF16_REL_L2


# ---------------------------------------------------------------------------
# the book
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,H,D,P", [(BF, 2, 64, 16), (F32, 3, 5, 32), (BF, 1, 3, 16), (BF, 2, 6, 64)])
def test_random_steps(txl, dtype, H, D, P):
    """Every call in random order, valid and not, the whole state compared after each."""
    rng = np.random.default_rng(D)
    n_slots, n_pages = 9, 40
    book = Book(n_slots, 7, n_pages, P)
    pools = [torch.full((n_pages, H, P, D), float("nan")).to(dtype) for _ in range(2)]
    dev, gpu = to_gpu(book), [p.cuda() for p in pools]
    host = [p.float().numpy() for p in pools]
    seen = set()
    for step in range(400):
        what = ["append", "append", "fork", "free", "compact"][rng.integers(5)]
        refused = False
        if what == "append":
            slots = rng.integers(-1, n_slots + 1, rng.integers(1, 8)).tolist() if step % 7 == 0 else \
                rng.permutation(n_slots)[:rng.integers(1, 8)].tolist()
            counts = rng.integers(0, [3, 2 * P][rng.integers(2)] + 1, len(slots)).tolist()
            cu = cu_of(counts)
            new = [torch.from_numpy(rng.normal(size=(cu[-1] + 1, H, D))).to(dtype) for _ in range(2)]
            g, a, z, refused = book.reserve(slots, cu)
            out = [ints([9] * len(slots)) for _ in range(3)]
            txl.txl_pages_reserve(dev, P, ints(slots), ints(cu), *out)
            assert [x.tolist() for x in out] == [g, a, z]
            for h, x in zip(host, new):
                book.append(h, slots, cu, g, a, z, x.float().numpy())
            txl.txl_pages_append(dev, *gpu, ints(slots), ints(cu), *out, *[x.cuda() for x in new])
            seen |= {"copied"} if any(x >= 0 for x in a) else set()
            seen |= {"full"} if refused and step % 7 else set()
        elif what == "fork":
            a, d = (rng.permutation(n_slots)[:3].tolist() for _ in range(2))
            if step % 5 == 0:
                a[0], d[1] = -3, n_slots
            elif step % 2:  # a held slot into an empty one, where there are such
                held = [x for x in range(n_slots) if book.rows[x]]
                a[0], d[0] = (held or a)[0], ([x for x in range(n_slots) if not book.rows[x]] or d)[0]
            want = book.fork(a, d)
            ok = ints([9] * 3)
            txl.txl_pages_fork(dev, P, ints(a), ints(d), ok)
            assert ok.tolist() == want
            refused = 0 in want
            seen |= {"forked"} if 1 in want else set()
        elif what == "free":
            slots = rng.integers(0, n_slots, 3).tolist()
            keep = (rng.integers(-2, 4 * P, 3) * rng.integers(0, 2, 3)).tolist()
            refused = book.free(slots, keep)
            txl.txl_pages_free(dev, P, ints(slots), ints(keep))
        else:
            new_id, a, z = book.compact()
            out = [ints([9] * n_pages) for _ in range(3)] + [ints([9])]
            txl.txl_pages_compact(dev, P, *out)
            pad = [-1] * (n_pages - len(a))
            assert [x.tolist() for x in out] == [new_id, a + pad, z + pad, [len(a)]]
            for h in host:
                h[z] = h[a]
            txl.txl_pages_copy(*gpu, out[1], out[2])
            seen |= {"moved"} if a else set()
        assert txl.txl_get_device_status() == (6 if refused else 0), what
        same(dev, book)
        for x, h in zip(gpu, host):
            np.testing.assert_array_equal(x.float().cpu().numpy(), h)
    assert seen == {"copied", "full", "forked", "moved"}


def test_large_book(txl):
    """A reserve whose free pages lie scattered over several steps of the scan, many slots, long table rows; then all
    freed."""
    rng = np.random.default_rng(21)
    n_slots, n_pages, P, max_pages = 3000, 50001, 16, 40
    book = Book(n_slots, max_pages, n_pages, P)
    held = sorted(rng.choice(n_pages, 30000, replace=False).tolist())
    for s in range(1000):
        for j in range(30):
            book.table[s][j] = held[s * 30 + j]
            book.refs[held[s * 30 + j]] = 1
        book.start[s], book.rows[s] = s % P, 30 * P - s % P
    dev = to_gpu(book)
    slots = rng.permutation(n_slots)[:2500].tolist()
    counts = rng.integers(0, 9 * P, 2500).tolist()
    cu = cu_of(counts)
    out = [ints([9] * 2500) for _ in range(3)]
    g, a, z, refused = book.reserve(slots, cu)
    txl.txl_pages_reserve(dev, P, ints(slots), ints(cu), *out)
    assert [x.tolist() for x in out] == [g, a, z] and not refused
    same(dev, book)
    keep = rng.integers(0, 30 * P, 2500).tolist()
    book.free(slots, keep)
    txl.txl_pages_free(dev, P, ints(slots), ints(keep))
    same(dev, book)
    new_id, src, dst = book.compact()
    out = [ints([9] * n_pages) for _ in range(3)] + [ints([9])]
    txl.txl_pages_compact(dev, P, *out)
    assert out[0].tolist() == new_id and out[3].item() == len(src) and out[1].tolist()[:len(src)] == src
    assert out[2].tolist()[:len(src)] == dst and len(src) > 1000
    same(dev, book)
    txl.txl_pages_free(dev, P, ints(list(range(n_slots))))
    assert (dev["table"] == -1).all() and not dev["refs"].any() and not dev["rows"].any() and not dev["start"].any()
    assert txl.txl_get_device_status() == 0


@pytest.mark.parametrize("n_slots,n", [(7000, 1024), (7000, 1025), (9000, 1), (16384, 1000), (1100, 1024)])
def test_reserve_sizes(txl, n_slots, n):
    """More pages than are placed at a time; either side of one entry a thread; shared last pages; too few pages left."""
    rng = np.random.default_rng(n_slots + n)
    assert txl.txl_get_device_status() == 0
    P, n_pages, max_pages = 16, 17000, 12
    book = Book(n_slots, max_pages, n_pages, P)
    for page in rng.choice(n_pages, 5000, replace=False).tolist():  # held elsewhere
        book.refs[page] = 1
    dev = to_gpu(book)

    def reserve(slots, counts):
        cu = cu_of(counts)
        out = [ints([9] * len(slots)) for _ in range(3)]
        g, a, z, refused = book.reserve(slots, cu)
        txl.txl_pages_reserve(dev, P, ints(slots), ints(cu), *out)
        assert [x.tolist() for x in out] == [g, a, z]
        same(dev, book)
        assert (txl.txl_get_device_status() == 0) == (not refused)
        return refused

    order = rng.permutation(n_slots).tolist()
    slots, others = order[:n], order[n:2 * n]
    assert not reserve(slots, rng.integers(1, 9 * P, n).tolist())
    pairs = min(len(others), n)
    if pairs:
        ok = book.fork(slots[:pairs], others[:pairs])
        out = ints([9] * pairs)
        txl.txl_pages_fork(dev, P, ints(slots[:pairs]), ints(others[:pairs]), out)
        assert out.tolist() == ok
    assert not reserve(slots, [1] * n)  # copies of shared last pages
    reserve(slots + others[:pairs], rng.integers(0, 9 * P, n + pairs).tolist())  # some ask for too much
    reserve(slots[::-1], [P] * n)  # until the pages are gone


def test_pools_off_the_wide_path(txl):
    """Pools and rows on a 2-byte boundary go by the narrow copies."""
    rng = np.random.default_rng(22)
    P, H, D, N = 16, 2, 10, 12
    book = Book(3, 4, N, P)
    dev = to_gpu(book)
    raw = [torch.zeros(N * H * P * D + 1, dtype=BF, device="cuda")[1:].view(N, H, P, D) for _ in range(2)]
    new = [torch.from_numpy(rng.normal(size=(50, H, D))).to(BF) for _ in range(2)]
    slots, cu = [0, 1, 2], [0, 17, 20, 50]
    g, a, z, _ = book.reserve(slots, cu)
    out = [ints([0] * 3) for _ in range(3)]
    txl.txl_pages_reserve(dev, P, ints(slots), ints(cu), *out)
    txl.txl_pages_append(dev, *raw, ints(slots), ints(cu), *out, *[x.cuda() for x in new])
    txl.txl_pages_copy(*raw, ints([0, -1, 2]), ints([9, 4, 10]))
    for pool, x in zip(raw, new):
        want = np.zeros((N, H, P, D), np.float32)
        book.append(want, slots, cu, g, a, z, x.float().numpy())
        want[9], want[10] = want[0], want[2]
        np.testing.assert_array_equal(pool.float().cpu().numpy(), want)
    assert txl.txl_get_device_status() == 0


def test_copy_refuses_pages_past_the_pool(txl):
    pools = [torch.arange(4, device="cuda", dtype=F32).view(4, 1, 1, 1).expand(4, 1, 16, 4).contiguous()
             for _ in range(2)]
    txl.txl_pages_copy(*pools, ints([4, 1, 0]), ints([0, 3, 1 << 27]))
    assert txl.txl_get_device_status() == 6
    for p in pools:
        assert p[:, 0, 0, 0].tolist() == [0, 1, 2, 1]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def serve(txl, dev, pools, slots, cu, new, q, r, u, vb, out, ws, keep, max_new):
    P = pools[0].shape[2]
    lists = [torch.empty_like(slots) for _ in range(3)]
    txl.txl_pages_reserve(dev, P, slots, cu, *lists)
    txl.txl_pages_append(dev, *pools, slots, cu, *lists, *new)
    txl.txl_relattn_forward_paged(q, *pools, dev, slots, cu, r, u, vb, out, ws, max_new=max_new)
    txl.txl_pages_free(dev, P, slots, keep)


@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (64, 140), (128, 70)])
def test_a_server(txl, D, n):
    """Steps of a ragged batch: rows written, attended, the oldest freed; a fork in between, and a compaction; each
    step's output against the oracle on the rows each sequence should hold."""
    rng = np.random.default_rng(D + n)
    H, P, M, slots = 2, 16, 100, 5
    pools = [torch.full((120, H, P, D), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
    dev = to_gpu(Book(slots, (M + n) // P + 3, 120, P))
    model = [[], [], []]  # per sequence: (k, v) rows
    where = [0, 1, 2]
    r = (0.5 * torch.from_numpy(rng.normal(size=(M + n, H, D)))).to(BF).cuda()
    u, vb = (0.3 * torch.from_numpy(rng.normal(size=(H, D))).float().cuda() for _ in range(2))
    off = room = 0.0
    for step in range(12 if n > 1 else 130):
        counts = [n] * len(where) if n == 1 else rng.integers(1, n + 1, len(where)).tolist()
        cu = cu_of(counts)
        q, *new = [torch.from_numpy(rng.normal(size=(cu[-1], H, D))).to(BF).cuda() for _ in range(3)]
        out = torch.empty_like(q)
        serve(txl, dev, pools, ints(where), ints(cu), new, q, r, u, vb, out,
              workspace(txl, len(where), cu[-1], H, D, BF), ints([M] * len(where)), n)
        host = [x.float().cpu().numpy() for x in (q, *new, out)]
        for i in range(len(where)):
            rows = slice(cu[i], cu[i + 1])
            model[i] = model[i] + list(zip(host[1][rows], host[2][rows]))
            if step % 10 == 3 or n > 1 or step > 125:
                kk, vv = (np.stack([x[y] for x in model[i]]) for y in range(2))
                want, _, do, _ = tolerance(host[0][rows], kk, vv, r.float().cpu().numpy(), u.cpu().numpy(),
                                           vb.cpu().numpy(), D ** -0.5, 2.0 ** -8, 2, 2.0 ** -8)
                e = np.abs(host[3][rows] - want)
                assert (e <= do).all()
                off += (e ** 2).sum()
                room += spread(host[0][rows], kk, vv, r.float().cpu().numpy(), u.cpu().numpy(), vb.cpu().numpy(),
                               D ** -0.5, 2.0 ** -8, 2.0 ** -8)
            model[i] = model[i][-M:]
        if step == 5:  # sequence 1 forks into slots 3 and 4
            ok = ints([0, 0])
            txl.txl_pages_fork(dev, P, ints([1, 1]), ints([3, 4]), ok)
            assert ok.tolist() == [1, 1]
            where, model = [0, 1, 2, 3, 4], model + [list(model[1]), list(model[1])]
        if step == 8:  # sequence 0 ends; the pool is put in order
            txl.txl_pages_free(dev, P, ints([0]))
            moves = [torch.empty(len(pools[0]), dtype=torch.int32, device="cuda") for _ in range(3)]
            txl.txl_pages_compact(dev, P, *moves, ints([0]))
            txl.txl_pages_copy(*pools, moves[1], moves[2])
            live = int((dev["refs"] > 0).sum())
            assert not dev["refs"][live:].any()
            where, model = where[1:], model[1:]
    assert txl.txl_get_device_status() == 0
    assert off <= room


@pytest.mark.parametrize("n,max_new", [(1, 1), (30, 40)])
def test_captured_and_replayed(txl, n, max_new):
    """A step captured into a graph: its replays find the lengths that the replay before left, and a second graph with
    its own workspace runs beside it."""
    rng = np.random.default_rng(n)
    H, D, P, M, seqs = 2, 64, 16, 90, 4
    T = seqs * n

    def world(seed):
        g = np.random.default_rng(seed)
        draw = lambda *s: torch.from_numpy(g.normal(size=s)).to(BF).cuda()  # noqa: E731
        pools = [torch.full((120, H, P, D), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
        return dict(dev=to_gpu(Book(seqs, 20, 120, P)), pools=pools, slots=ints(list(range(seqs))),
                    cu=ints([n * i for i in range(seqs + 1)]), new=[draw(T, H, D), draw(T, H, D)], q=draw(T, H, D),
                    r=draw(M + n, H, D), u=draw(H, D).float(), vb=draw(H, D).float(),
                    out=torch.empty(T, H, D, dtype=BF, device="cuda"), ws=workspace(txl, seqs, T, H, D, BF),
                    keep=ints([M] * seqs), max_new=max_new)

    eager, graphed, other = world(1), world(1), world(2)
    graphs = []
    for w in (graphed, other):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            serve(txl, **w)  # warm-up
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            serve(txl, **w)
        graphs.append((gr, side))
    serve(txl, **eager)
    for step in range(110 if n == 1 else 25):
        x = torch.from_numpy(rng.normal(size=(T, H, D))).to(BF).cuda()
        for w in (eager, graphed, other):
            w["q"].copy_(x)
            w["new"][0].copy_(x.flip(0))
        torch.cuda.synchronize()
        for gr, side in graphs:
            with torch.cuda.stream(side):
                gr.replay()
        serve(txl, **eager)
        torch.cuda.synchronize()
        assert torch.equal(eager["out"], graphed["out"])
        for name in NAMES:
            assert torch.equal(eager["dev"][name], graphed["dev"][name]), name
    assert int(eager["dev"]["rows"][0]) == M
    assert txl.txl_get_device_status() == 0


def test_a_stream_of_its_own(txl):
    """The calls run on the stream that is named, not on the current one."""
    rng = np.random.default_rng(33)
    args, kw = attend_case(txl, rng, [(0, 300), (5, 40)], [1, 1], 16, 2, 64, BF)
    want = args[9].clone()
    s = torch.cuda.Stream()
    args[9].fill_(0.0)
    torch.cuda.synchronize()
    txl.txl_relattn_forward_paged(*args, **kw, stream=s)
    s.synchronize()
    assert torch.equal(args[9], want)


def test_refused_arguments(txl):
    """What the binding turns away before any launch."""
    rng = np.random.default_rng(5)
    args, kw = attend_case(txl, rng, [(3, 40), (0, 9)], [2, 1], 16, 2, 64, BF)
    q, k, v, book, slots, cu, r, u, vb, o, ws = args

    def attend(**change):
        names = "q k_pages v_pages book slots cu r bias_u bias_v o workspace".split()
        full = dict(zip(names, args))
        full.update(kw)
        full.update(change)
        return txl.txl_relattn_forward_paged(**full)

    before = o.clone()
    for change in (dict(slots=slots.long()), dict(slots=slots.cpu()), dict(cu=cu[:-1]), dict(cu=slots), dict(q=q[:, :1]),
                   dict(q=q.float()), dict(r=r.float()), dict(bias_u=u.to(BF)), dict(bias_v=vb[:1]), dict(o=o[:-1]),
                   dict(lse=torch.zeros(2, 2, device="cuda")), dict(k_pages=k[:-1], v_pages=v[:-1]), dict(v_pages=v[:-1]),
                   dict(k_pages=k.transpose(1, 2)), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                   dict(slots=torch.stack([slots, slots], 1)[:, 0]), dict(book=dict(book, rows=book["rows"].long())),
                   dict(book=dict(book, table=book["table"][0])), dict(book=dict(book, refs=book["refs"][:-1])),
                   dict(max_new=2 ** 31), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            attend(**change)
    with pytest.raises(TypeError):
        attend(book=list(book.values()))
    with pytest.raises(KeyError):
        attend(book={x: book[x] for x in ("table", "start", "rows")})
    with pytest.raises(TypeError):
        attend(scale="1")
    with pytest.raises(txl.TxlError):
        attend(workspace=ws[:16])
    with pytest.raises(txl.TxlError):
        txl.txl_pages_free(book, 24, slots)  # page rows: no power of two
    with pytest.raises(ValueError):
        txl.txl_pages_append(book, k, v, slots, cu, slots.clone(), slots.clone(), None, k[0], v[0])
    torch.cuda.synchronize()
    assert torch.equal(o, before) and txl.txl_get_device_status() == 0
    attend()
    assert torch.equal(o, before)


def test_offsets_past_32_bits(txl):
    """A pool of more than 2^31 elements whose live pages are its last ones."""
    H, D, P, N = 8, 128, 1024, 2100
    if torch.cuda.mem_get_info()[0] < 14e9:
        pytest.skip("needs 14 GB")
    assert N * H * D * P > 2 ** 31
    rng = np.random.default_rng(34)
    pools = [torch.zeros(N, H, P, D, dtype=BF, device="cuda") for _ in range(2)]
    book = Book(2, 2, N, P)
    book.refs = [1] * (N - 2) + [0, 0]
    dev = to_gpu(book)
    n = 60
    q, k, v = (torch.from_numpy(rng.normal(size=(2 * n, H, D))).to(BF) for _ in range(3))
    r = torch.from_numpy(rng.normal(size=(n, H, D))).to(BF)
    u = torch.zeros(H, D)
    out = [ints([0, 0]) for _ in range(3)]
    txl.txl_pages_reserve(dev, P, ints([0, 1]), ints([0, n, 2 * n]), *out)
    assert dev["table"].tolist() == [[N - 2, -1], [N - 1, -1]]
    txl.txl_pages_append(dev, *pools, ints([0, 1]), ints([0, n, 2 * n]), *out, k.cuda(), v.cuda())
    for new in (n, 1):
        o = torch.empty(2 * new, H, D, dtype=BF, device="cuda")
        qq = torch.cat([q[n - new:n], q[2 * n - new:]])
        txl.txl_relattn_forward_paged(qq.cuda(), *pools, dev, ints([0, 1]), ints([0, new, 2 * new]), r.cuda(),
                                      u.cuda(), u.cuda(), o, workspace(txl, 2, 2 * new, H, D, BF), max_new=new)
        for i in range(2):
            rows = slice(i * n, (i + 1) * n)
            want, _, do, _ = tolerance(qq[i * new:(i + 1) * new].float().numpy(), k[rows].float().numpy(),
                                       v[rows].float().numpy(), r.float().numpy(), u.numpy(), u.numpy(), D ** -0.5,
                                       2.0 ** -8, 2, 2.0 ** -8)
            assert (np.abs(o[i * new:(i + 1) * new].float().cpu().numpy() - want) <= do).all()
    txl.txl_pages_copy(*pools, ints([N - 1]), ints([N - 3]))
    assert torch.equal(pools[0][N - 3], pools[0][N - 1])
    assert txl.txl_get_device_status() == 0
