"""Values of the operators around the layers at the ends of what their settings may be, against the oracle in 64 bits."""

import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_tokens import BF, F32, _check_sample, _host, _tensor, txl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3000, 20000])
def test_sample_hot_rows(txl, V, dtype):  # noqa: F811
    """Logits further apart than the largest float, which temperatures of their size bring near each other."""
    rng = np.random.default_rng(V)
    z = 3.3e38 * rng.uniform(-1, 1, (6, V))
    z[:, 3], z[:, 5] = 3.3e38, -3.3e38
    z[1, ::4], z[2, 7] = np.inf, -np.inf
    inf = _tensor(z, dtype)
    z = inf.clamp(max=torch.finfo(dtype).max)  # what +inf counts as: the oracle knows fp32's alone
    hot = [1e38, 3e38, 2e38, 5e37, 1.5e38, 3.4e38]
    u = rng.random(6)
    for s in ({}, dict(top_k=[2, 7, 30, V // 2, V - 1, V]), dict(top_p=[0.1, 0.5, 0.9, 0.99, 0.999, 0.7]),
              dict(top_k=[3, 20, 35, V // 3, V - 1, 0], top_p=[0.3, 0.5, 0.7, 0.9, 0.99, 0.5]), dict(min_p=[0.5, 0.1, 0.01, 0.9, 1e-4, 0.05])):
        _check_sample(txl, z, u, temperature=hot, **s)
    _check_sample(txl, z, u, temperature=[1e30, 1e36, 1e37, 2e37, 8e36, 3e36])
    same = []
    for x in (inf, z):
        same.append((torch.empty(6, device=dev(), dtype=torch.int32), torch.empty(6, device=dev())))
        txl.txl_sample(x, _tensor(u, F32), same[-1][0], temperature=_tensor(hot, F32), prob=same[-1][1])
    assert all(torch.equal(a, b) for a, b in zip(*same))


@pytest.mark.parametrize("V", [40, 3000, 20000])
def test_sample_cold_rows(txl, V):  # noqa: F811
    """Subnormal temperatures, whose reciprocals no float holds, and logits as close together; such a temperature among
    logits of any size leaves the largest."""
    rng = np.random.default_rng(V + 1)
    cold = [1e-45, 1e-44, 1e-42, 1e-40, 4e-39, 1e-39]
    z = np.float32(cold)[:, None].astype(np.float64) * rng.integers(-30, 1, (6, V))
    u = rng.random(6)
    for s in ({}, dict(top_k=[2, 7, 30, V // 2, V - 1, V]), dict(top_p=[0.1, 0.5, 0.9, 0.99, 0.999, 0.7]), dict(min_p=[0.5, 0.1, 0.01, 0.9, 1e-4, 0.05])):
        _check_sample(txl, _tensor(z, F32), u, temperature=cold, **s)
    wide = np.sign(rng.standard_normal((6, V))) * 10.0 ** rng.uniform(-38, 38, (6, V))
    for s in ({}, dict(top_p=[0.1, 0.5, 0.9, 0.99, 0.999, 0.7])):
        _check_sample(txl, _tensor(wide, F32), u, temperature=cold, **s)
        _check_sample(txl, _tensor(wide, BF), u, temperature=[1e-30] * 6, **s)


def _ledge(rng, V):
    """A row of twenty tokens with three quarters of the weight and, far lower, the others, of which the largest comes
    last, and shares of top-p next to that of the twenty: the nearest floats but one to three."""
    z = np.log(60 / V) + 6 + 0.1 * rng.standard_normal(V)
    z[-1] = np.log(60 / V) + 6.7
    z[rng.choice(V - 1, 20, replace=False)] = rng.uniform(7, 9, 20)
    z = np.float32(z)
    w = np.exp(z.astype(np.float64) - z.max())
    share = w[z >= 7].sum() / w.sum()
    return z, [float(np.float32(share) + np.float32(j * 2.0 ** -24)) for j in (-3, -2, -1, 1, 2, 3)]


@pytest.mark.parametrize("V", [3000, 50021, 131072])
def test_sample_by_the_edge_of_a_gap(txl, V):  # noqa: F811
    """The share of top-p ends just before or just behind a wide gap of logits, so that a guess from counts in bins puts
    the border on its other side, and the row is searched again.  A uniform number of 1 names the last kept token."""
    rng = np.random.default_rng(V)
    for _ in range(4):
        z, p = _ledge(rng, V)
        _check_sample(txl, _tensor(np.tile(z, (6, 1)), F32), [1.0] * 6, top_p=p)
        _check_sample(txl, _tensor(np.tile(z, (6, 1)), F32), [1.0] * 6, top_p=p, min_p=[1e-9] * 6)


@pytest.mark.parametrize("V", [5000, 131072, 1 << 18])
@pytest.mark.parametrize("low", [14.3, 20.8, 27.9, 30.1])
def test_sample_far_tails(txl, low, V):  # noqa: F811
    """Many tokens of little weight, of which a weight is cut to whole multiples of 2^-44 of the largest: the token's
    stretch of running shares holds the uniform number but for V of these, and what the weights leave (2^-39), both
    in the sum and in the whole."""
    rng = np.random.default_rng(V + int(low))
    z = -low + 0.01 * rng.standard_normal((5, V))
    z[:, -1] = 0.0
    z = _tensor(z, F32)
    w = np.exp(_host(z))
    upto = w.cumsum(1) / w.sum(1, keepdims=True)
    u = np.float32(upto[:, -2] * [0.1, 0.3, 0.5, 0.9, 0.999])  # among the tail
    tokens, prob = torch.empty(5, device=dev(), dtype=torch.int32), torch.empty(5, device=dev())
    txl.txl_sample(z, _tensor(u, F32), tokens, prob=prob)
    off = 2 * (V * 2.0 ** -44 + 2.0 ** -39)
    for b, t in enumerate(tokens.tolist()):
        assert (upto[b, t - 1] if t else 0.0) - off <= u[b] <= upto[b, t] + off, (b, t)
        assert abs(float(prob[b]) - w[b, t] / w[b].sum()) <= 2.0 ** -22 * float(prob[b]) + off
