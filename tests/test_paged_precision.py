"""What the bf16 kernels' two-part operands leave: (q + u), (q + v), or u and v
beside an exact q, and the weights as two bf16 numbers each, hi + lo, products
and sums in fp32.  The bounds that the GPU tests hold them to, and on the CPU that
arithmetic of this kind keeps them while leaving out any one of the low parts,
or rounding the distance part, does not."""

import numpy as np
import pytest
import torch

from oracle.pages_oracle import attend, spread, tolerance

# A part rounds to nearest, off by at most 2^-8 of what it rounds; lo rounds what hi left: 2^-8 * 2^-8.
SPLIT = 2.0 ** -16
# fp32 chains: an accumulator of a score takes D/16 products of 16 terms for each of q + u and q + v, in each part; one
# of the output rows/16; a step is off by 2^-23 at most (the tensor core may cut off), the exponential by 2^-22.  For D
# up to 128 and 1024 rows that is under 2 * 2^-18 of the sum of the terms' absolute values.
CHAIN = 2.0 ** -18


def bounds(q, k, v, r, u, vb, scale):
    """o, what each element may be off, and what the sum of the squared errors may be: of errors a + b, (a + b)^2 <= 2 a^2
    + 2 b^2, a the parts' independent roundings, b the chains at their worst."""
    o, _, split, _ = tolerance(q, k, v, r, u, vb, scale, SPLIT, 1, 2.0 ** -24)
    _, _, chain, _ = tolerance(q, k, v, r, u, vb, scale, CHAIN, 2, 2.0 ** -24)
    return o, split + chain, 2 * (spread(q, k, v, r, u, vb, scale, SPLIT, 2.0 ** -24) + (chain ** 2).sum())


def bf(x):
    return torch.tensor(x).to(torch.bfloat16).double().numpy()


def parts(x, low):
    hi = bf(x)
    return hi + (bf(x - hi) if low else 0.0)


def case(rng, n, L, H, D):
    q, k, v, r = (bf(rng.normal(size=(x, H, D))) for x in (n, L, L, L))
    u, vb = (rng.normal(size=(H, D)) * 0.3 for _ in range(2))
    return q, k, v, r, u.astype(np.float32).astype(float), vb.astype(np.float32).astype(float)


def computed(q, k, v, r, u, vb, scale, without=""):
    o = np.zeros_like(q)
    n, H, _ = q.shape
    for h in range(H):
        for t in range(n):
            m = len(k) - n + t
            a = parts(scale * (q[t, h] + u[h]), without != "u")
            b = parts(scale * (q[t, h] + vb[h]), without != "v")
            far = r[m::-1, h] @ b
            z = k[:m + 1, h] @ a + (bf(far) if without == "distance" else far)
            w = np.exp(z - z.max())
            o[t, h] = parts(w, without != "weights") @ v[:m + 1, h] / w.sum()
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("without", ["", "u", "v", "weights", "distance"])
def test_each_low_part_shows(D, without):
    rng = np.random.default_rng(D)
    for n, L in ((1, 30), (2, 60), (4, 90), (9, 60), (20, 40)):
        c = case(rng, n, L, 2, D)
        want, each, room = bounds(*c, D ** -0.5)
        off = (computed(*c, D ** -0.5, without=without) - want) ** 2
        if without:
            assert off.sum() > room
        else:
            assert (off <= each ** 2).all() and off.sum() <= room
            assert np.array_equal(want, attend(*c, D ** -0.5)[0])
