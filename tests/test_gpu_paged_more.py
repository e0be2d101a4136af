"""The paged attention held closer: the decode kernel's two-part operands, fp32
entries beside refused ones, slots that share pages inside one call, and fp32
over more blocks than fit the GPU at once."""

import numpy as np
import pytest
import torch

from oracle.pages_oracle import Book, tolerance
from test_gpu_paged import BF, F32, attend_case, cu_of, ints, to_gpu, workspace
from test_paged_precision import bounds, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def txl():
    import transformer_xl_relative_txl_gb300 as m

    assert m.txl_get_device_status() == 0
    return m


def paged(rng, k, v, P, start):
    """One slot that holds the rows k, v behind `start` dead ones, and its pools on the GPU."""
    m, H, D = k.shape
    need = -(-(start + m) // P)
    book = Book(1, need, need, P)
    book.table[0] = rng.permutation(need).tolist()
    book.refs = [1] * need
    book.start, book.rows = [start], [m]
    pools = []
    for x in (k, v):
        pool = torch.full((need, H, P, D), float("nan"))
        for j in range(m):
            p, at = book.place(0, j)
            pool[p][:, at] = torch.from_numpy(x[j]).float()
        pools.append(pool.to(BF).cuda())
    return book, pools


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(1, 30), (2, 60), (4, 90), (4, 130)])
def test_low_parts(txl, D, n, L):
    """Up to four tokens, output in fp32: q + u, q + v and the weights keep both their parts."""
    rng = np.random.default_rng(D)
    H = 2
    q, k, v, r, u, vb = case(rng, n, L, H, D)
    book, pools = paged(rng, k, v, 16, 5)
    f = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().cuda()  # noqa: E731
    o = torch.empty(n, H, D, device="cuda")
    txl.txl_relattn_forward_paged(f(q).to(BF), *pools, to_gpu(book), ints([0]), ints([0, n]), f(r).to(BF), f(u), f(vb), o,
                                  workspace(txl, 1, n, H, D, BF), max_new=n)
    assert txl.txl_get_device_status() == 0
    want, each, room = bounds(q, k, v, r, u, vb, D ** -0.5)
    off = np.abs(o.double().cpu().numpy() - want)
    assert (off <= each).all() and (off ** 2).sum() <= room


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(9, 60), (20, 40), (70, 90), (130, 131)])
def test_low_parts_of_tiles(txl, D, n, L):
    """More tokens: q + u, q + v and the weights keep both their parts, the distance part its 32 bits."""
    rng = np.random.default_rng(D)
    H = 2
    q, k, v, r, u, vb = case(rng, n, L, H, D)
    book, pools = paged(rng, k, v, 16, 5)
    f = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().cuda()  # noqa: E731
    o = torch.empty(n, H, D, device="cuda")
    txl.txl_relattn_forward_paged(f(q).to(BF), *pools, to_gpu(book), ints([0]), ints([0, n]), f(r).to(BF), f(u), f(vb), o,
                                  workspace(txl, 1, n, H, D, BF), max_new=n)
    assert txl.txl_get_device_status() == 0
    want, each, room = bounds(q, k, v, r, u, vb, D ** -0.5)
    off = np.abs(o.double().cpu().numpy() - want)
    assert (off <= each).all() and (off ** 2).sum() <= room


@pytest.mark.parametrize("D,new", [(16, 5), (64, 1), (128, 40)])
def test_float32_beside_refused_entries(txl, D, new):
    """The entries that are served, against the oracle at fp32's own tolerance."""
    rng = np.random.default_rng(D + new)
    args, kw = attend_case(txl, rng, [(0, new + 20)] * 5, [new] * 5, 16, 2, D, F32)
    q, k, v, dev, slots, cu, r, u, vb, o, ws = args
    bad = slots.clone()
    bad[0] = -1
    dev["rows"][3] = len(r) + 1
    o.fill_(7.0)
    txl.txl_relattn_forward_paged(q, k, v, dev, bad, cu, r, u, vb, o, ws, **kw)
    assert txl.txl_get_device_status() == 6
    book = Book(5, dev["table"].shape[1], len(k), 16)
    book.table, book.start, book.rows = (dev[x].tolist() for x in ("table", "start", "rows"))
    host = [x.cpu().numpy() for x in (q, k, v, r, u, vb, o)]
    for i in range(5):
        rows = slice(i * new, (i + 1) * new)
        if i in (0, 3):
            assert (host[6][rows] == 7.0).all()
            continue
        want, _, do, _ = tolerance(host[0][rows], book.gather(host[1], i), book.gather(host[2], i), host[3], host[4],
                                   host[5], kw["scale"], 2.0 ** -24, 2 * D + new + 20, 2.0 ** -24)
        assert (np.abs(host[6][rows] - want) <= do).all()


@pytest.mark.parametrize("dtype,D,counts", [(BF, 64, [200, 131, 3, 70]), (BF, 128, [150, 1, 129, 20]),
                                            (BF, 64, [1, 4, 2, 1]), (F32, 24, [30, 1, 17, 50])])
def test_shared_pages_in_one_call(txl, dtype, D, counts):
    """A slot and its forks extended by rows of their own (copies of the shared last page), then attended together, the
    rows before it in pages that all of them share."""
    rng = np.random.default_rng(D)
    H, P, old = 2, 16, 147
    book = Book(4, 30, 120, P)
    dev = to_gpu(book)
    pools = [torch.full((120, H, P, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    host = [np.full((120, H, P, D), np.nan, np.float32) for _ in range(2)]

    def extend(slots, counts):
        cu = cu_of(counts)
        new = [torch.from_numpy(rng.normal(size=(cu[-1], H, D))).to(dtype) for _ in range(2)]
        out = [ints([9] * len(slots)) for _ in range(3)]
        g, a, z, refused = book.reserve(slots, cu)
        assert not refused
        for h, x in zip(host, new):
            book.append(h, slots, cu, g, a, z, x.float().numpy())
        txl.txl_pages_reserve(dev, P, ints(slots), ints(cu), *out)
        txl.txl_pages_append(dev, *pools, ints(slots), ints(cu), *out, *[x.cuda() for x in new])
        return cu

    extend([0], [old])
    assert book.fork([0, 0, 0], [1, 2, 3]) == [1, 1, 1]
    txl.txl_pages_fork(dev, P, ints([0, 0, 0]), ints([1, 2, 3]), ints([0, 0, 0]))
    cu = extend([0, 1, 2, 3], counts)
    assert dev["refs"].max().item() == 4
    n_r = old + max(counts)
    q, r = (torch.from_numpy(rng.normal(size=(x, H, D))).to(dtype) for x in (cu[-1], n_r))
    u, vb = (torch.from_numpy(0.3 * rng.normal(size=(H, D))).float() for _ in range(2))
    o = torch.empty(cu[-1], H, D, device="cuda", dtype=dtype)
    txl.txl_relattn_forward_paged(q.cuda(), *pools, dev, ints([0, 1, 2, 3]), ints(cu), r.cuda(), u.cuda(), vb.cuda(), o,
                                  workspace(txl, 4, cu[-1], H, D, dtype), max_new=max(counts))
    assert txl.txl_get_device_status() == 0
    got = o.double().cpu().numpy()
    step, terms, out = (2.0 ** -8, 2, 2.0 ** -8) if dtype == BF else (2.0 ** -24, 2 * D + n_r, 2.0 ** -24)
    for s in range(4):
        rows = slice(cu[s], cu[s + 1])
        want, _, do, _ = tolerance(q[rows].float().numpy(), book.gather(host[0], s), book.gather(host[1], s),
                                   r.float().numpy(), u.numpy(), vb.numpy(), D ** -0.5, step, terms, out)
        assert (np.abs(got[rows] - want) <= do).all(), s


@pytest.mark.parametrize("D", [100, 128, 200, 256])
def test_float32_over_many_blocks(txl, D):
    """More units than blocks, and more blocks than the shared memory of their rows lets the GPU hold."""
    rng = np.random.default_rng(D)
    counts = [int(x) for x in rng.integers(1, 35, 90)]
    spans = [(int(rng.integers(16)), c + int(rng.integers(0, 70))) for c in counts]
    attend_case(txl, rng, spans, counts, 16, 8, D, F32)
