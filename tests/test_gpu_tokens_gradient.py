"""What the header says of the order and the roundings of the embedding's gradient."""

import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_tokens import BF, F32, _at_offset, _ints, _tensor, _zipf, txl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,d,ids", [(1, 5, 3, "z"), (300, 64, 64, "z"), (4999, 1000, 333, "z"), (9000, 3000, 512, "s"), (40000, 700, 72, "z"), (33001, 9, 20, "s")])
def test_the_order_is_the_ids_own(txl, T, V, d, ids):  # noqa: F811
    """The same bits whatever dout's type, the addresses, and whether the table is written or added to (0 and -0 alike)."""
    rng = np.random.default_rng(T + d)
    tokens = _ints(_zipf(rng, T, V) if ids == "z" else np.full(T, V - 1))
    dout = _tensor(rng.standard_normal((T, d)), BF)
    want = txl.txl_embed_backward(tokens, dout, torch.empty(V, d, device=dev()), scale=3.7)
    for rows in (dout.float(), _at_offset(dout, 1), _at_offset(dout.float(), 3)):
        for off in (0, 1):
            for accumulate in (False, True):
                got = _at_offset(torch.full((V, d), 0.0 if accumulate else float("nan"), device=dev()), off)
                txl.txl_embed_backward(_at_offset(tokens, 1), rows, got, scale=3.7, accumulate=accumulate)
                assert torch.equal(got, want)


def test_up_to_4096_ids_are_one_sum(txl):  # noqa: F811
    """Its products with the scale alone would overflow; the sum of all is 0."""
    for d in (8, 333, 512):
        dout = torch.full((4096, d), 2.0 ** 27, device=dev())
        dout[2048:] *= -1
        for accumulate in (False, True):
            got = torch.zeros(7, d, device=dev())
            txl.txl_embed_backward(_ints(np.full(4096, 5)), dout, got, scale=2.0 ** 100, accumulate=accumulate)
            assert not got.any()


@pytest.mark.parametrize("off", [0, 1])
def test_subnormal_sums(txl, off):  # noqa: F811
    """Stored as they are; added, by the call or as a later part of a long sum, as 0."""
    tiny = float(np.float32(1e-42))
    for T, parts in ((1, 1), (4096, 1), (8192, 2)):
        dout = torch.full((T, 8), tiny, device=dev())
        want = float(np.float32(tiny * T))
        for accumulate in (False, True):
            got = _at_offset(torch.zeros(3, 8, device=dev()), off)
            txl.txl_embed_backward(_ints(np.full(T, 1)), dout, got, accumulate=accumulate)
            assert not got[0].any() and not got[2].any()
            assert (got[1] == (want if parts == 1 and not accumulate else 0.0)).all(), (T, accumulate)
