"""The paged attention's bounded waits run out (test hook, 50 ms): the kernels
unwind, the status word says so, and the next call computes as the one before.
Even CTAs' loaders stop; in odd ones a role that gives stages back does, so that
the loader's own wait is the one that runs out."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 5
BF = torch.bfloat16


def call(txl, D, H, P, counts, rows, dead):
    """Arguments of a call over slots of `rows` live rows after `dead` dead ones, several units to a CTA."""
    g = torch.Generator(device="cuda").manual_seed(D + len(counts))
    draw = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    per = -(-(dead + rows) // P)
    n = len(counts)
    book = dict(table=ints(np.random.default_rng(1).permutation(n * per).reshape(n, per).tolist()), start=ints([dead] * n),
                rows=ints([rows] * n), refs=ints([1] * (n * per)))
    k, v = (draw(n * per, H, P, D).to(BF) for _ in range(2))
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    T = cu[-1]
    ws = torch.empty(txl.txl_relattn_paged_workspace_bytes(n, T, H, D, BF), dtype=torch.uint8, device="cuda")
    args = (draw(T, H, D).to(BF), k, v, book, ints(list(range(n))), ints(cu), (0.5 * draw(rows, H, D)).to(BF),
            0.1 * draw(H, D), 0.1 * draw(H, D), torch.empty(T, H, D, dtype=BF, device="cuda"), ws)
    return args, dict(lse=torch.empty(H, T, device="cuda"), max_new=max(counts))


@pytest.mark.parametrize("D,H,counts,rows", [
    (64, 16, [1] * 40, 1500),               # about two units of 24 tiles a CTA
    (128, 16, [1, 4, 2, 3] * 10, 700),      # of 22
    (64, 8, [300] * 24, 900),               # about four tiles of queries a CTA, of 10 to 15 steps each
    (128, 8, [300] * 24, 900),
    (64, 8, [300, 2, 200, 1] * 12, 800),    # both kernels
    (128, 8, [300, 2, 200, 1] * 12, 800),
])
def test_waits_that_run_out(D, H, counts, rows):
    import transformer_xl_relative_txl_gb300 as txl

    args, kw = call(txl, D, H, 32, counts, rows, 5)
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == OK
    want, want_l = args[9].clone(), kw["lse"].clone()
    assert torch.isfinite(want.float()).all()
    assert txl.txl_debug_set_wait_limit_ns(50_000_000) == OK
    try:
        assert txl.txl_debug_inject_stall(True) == OK
        txl.txl_relattn_forward_paged(*args, **kw)
        assert txl.txl_get_device_status() == TIMEOUT
        assert txl.txl_get_device_status() == OK  # the word was cleared
    finally:
        txl.txl_debug_inject_stall(False)
        txl.txl_debug_set_wait_limit_ns(2_000_000_000)
    args[9].fill_(0.0)
    txl.txl_relattn_forward_paged(*args, **kw)
    assert txl.txl_get_device_status() == OK
    assert torch.equal(args[9], want) and torch.equal(kw["lse"], want_l)
