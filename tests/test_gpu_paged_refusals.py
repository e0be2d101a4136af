"""Entries that the paged calls refuse change nothing; a page out of range is
never followed, and the attention takes its rows as zeros."""

import numpy as np
import pytest
import torch

from test_gpu_paged import BF, F32, attend_case, cu_of, filled, ints, same, to_gpu

pytestmark = pytest.mark.gpu

PAGES = 6


@pytest.fixture(scope="module")
def txl():
    import transformer_xl_relative_txl_gb300 as m

    assert m.txl_get_device_status() == 0
    return m


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 6), (F32, 5)])
@pytest.mark.parametrize("bad", [10 ** 8, -7])
def test_append_refuses_a_page(txl, dtype, D, bad):
    """A page out of range among those of an entry's new rows: none of the entry's rows is written, first or last page."""
    rng = np.random.default_rng(D)
    P, H, new = 16, 2, [40, 40, 70, 9]
    book, pools = filled(rng, [(3, 50), (0, 50), (5, 90), (0, 30)], P, H, D, dtype)
    book.table[1][3], book.table[2][1], book.table[3][1] = bad, bad, bad  # new rows from row 10; 25; 21
    dev = to_gpu(book)
    cu = cu_of(new)
    rows = [torch.from_numpy(rng.normal(size=(cu[-1], H, D))).to(dtype) for _ in range(2)]
    k, v = (x.cuda() for x in pools)
    txl.txl_pages_append(dev, k, v, ints([0, 1, 2, 3]), ints(cu), ints(new), None, None, *[x.cuda() for x in rows])
    assert txl.txl_get_device_status() == PAGES
    same(dev, book)
    for pool, before, x in zip((k, v), pools, rows):
        want = before.float().numpy()
        book.append(want, [0], [0, new[0]], [new[0]], [-1], [-1], x.float().numpy())  # entry 0 alone
        np.testing.assert_array_equal(pool.float().cpu().numpy(), want)


@pytest.mark.parametrize("bad", [10 ** 8, -7])
@pytest.mark.parametrize("keep", [0, 20])
def test_free_refuses_a_page(txl, bad, keep):
    """A page out of range in a row that the call reads: the slot stays as it is."""
    rng = np.random.default_rng(3)
    book, _ = filled(rng, [(3, 60), (0, 100), (5, 90)], 16, 1, 4, BF)
    dead, kept = (1, 6), (2, 5)  # of the pages that leave, and of those that stay
    book.table[dead[0]][0], book.table[kept[0]][kept[1]] = bad, bad
    dev = to_gpu(book)
    txl.txl_pages_free(dev, 16, ints([0, 1, 2]), ints([keep] * 3))
    assert txl.txl_get_device_status() == PAGES
    assert not book.free([0], [keep])  # the first alone
    same(dev, book)


@pytest.mark.parametrize("dtype,D,counts", [(BF, 64, [1, 2, 4]), (BF, 128, [1, 4, 1]), (BF, 64, [90, 20, 200]),
                                            (BF, 128, [130, 7, 20]), (F32, 16, [5, 1, 40])])
@pytest.mark.parametrize("bad", [10 ** 8, -7])
def test_a_bad_page_counts_as_zeros(txl, dtype, D, counts, bad):
    """The same bits as with a page of zeros in its place."""
    rng = np.random.default_rng(12)
    args, kw = attend_case(txl, rng, [(3, 230)] * 3, counts, 16, 2, D, dtype)
    k, v, dev, o = args[1], args[2], args[3], args[9]
    free = (dev["refs"] == 0).nonzero()[0]
    k[free], v[free] = 0.0, 0.0
    dev["table"][1, 2] = free
    dev["table"][2, 9] = free
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == 0
    want, want_l = o.clone(), kw["lse"].clone()
    assert torch.isfinite(want.float()).all()
    dev["table"][1, 2] = bad
    dev["table"][2, 9] = bad
    o.fill_(7.0)
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == PAGES
    assert torch.equal(o, want) and torch.equal(kw["lse"], want_l)


def test_reserve_refuses_rows_before_the_first(txl):
    """Rows that append would not find: nothing is granted, 1024 entries or fewer and more."""
    for n in (4, 1100):
        book, _ = filled(np.random.default_rng(n), [(0, 5)] * n, 16, 1, 4, BF, spare=2 * n)
        dev = to_gpu(book)
        cu = [-9, -4, -4, 6] + list(range(7, 4 + n))  # entry 1 is empty, entry 2 starts before row 0
        out = [ints([9] * n) for _ in range(3)]
        g, a, z, refused = book.reserve(list(range(n)), cu)
        txl.txl_pages_reserve(dev, 16, ints(list(range(n))), ints(cu), *out)
        assert refused and len(cu) == n + 1 and g[:4] == [0, 0, 0, 1]
        assert [x.tolist() for x in out] == [g, a, z]
        assert txl.txl_get_device_status() == PAGES
        same(dev, book)
