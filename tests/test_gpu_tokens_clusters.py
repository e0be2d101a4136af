"""Sizes at which it goes by the number of clusters that run at a time how many CTAs share a product's k or a row's
logits, and sizes beside them."""

import numpy as np
import pytest

import test_gpu_tokens as base
from test_gpu_tokens import BF, F32, _check_sample, _tensor, txl  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,k,n,group", [(1, 8192, 720, 32), (8, 4096, 5792, 128), (8, 8192, 5792, 32), (16, 8192, 4096, 128), (32, 8192, 11584, 128), (32, 8192, 11528, 32)])
def test_products(txl, m, k, n, group):  # noqa: F811
    base.test_dense_w4_exact(txl, m, k, n, group)
    base.test_dense_w4(txl, m, k, n, group, "bf16")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(15, 185364), (16, 185364), (36, 92682), (37, 92682), (37, 131072), (37, 185364)])
def test_rows(txl, B, V, dtype):  # noqa: F811
    rng = np.random.default_rng(V + B)
    z = _tensor(2.0 * rng.standard_normal((B, V)) + 6 * (rng.random((B, V)) < 30 / V), dtype)
    _check_sample(txl, z, rng.random(B), top_k=rng.integers(0, 600, B), top_p=rng.uniform(0.5, 1.1, B), min_p=rng.uniform(0, 0.01, B))
