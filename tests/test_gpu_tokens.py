"""The operators around the layers on the GPU against the oracle in 64 bits, each
element within a bound that counts its roundings: half a step of the output's
type (2^-8 of the value in bf16, 2^-24 in fp32), 2^-24 of the terms' sizes for
each fp32 addition, 2^-23 for those of the tensor cores, which may cut off."""

import math
import threading

import numpy as np
import pytest
import torch

from gpu_util import dev
from oracle import tokens_oracle as O

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
NAMES = {"bf16": BF, "f32": F32}


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import transformer_xl_relative_txl_gb300 as lib

    torch.cuda.set_device(0)
    lib.txl_get_device_status()
    return lib


def _host(t):
    return t.detach().double().cpu().numpy()


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())


def _tensor(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dev()).to(dtype)


def _at_offset(t, elements):
    """The same values, starting `elements` behind an aligned address."""
    flat = torch.zeros(t.numel() + elements, device=t.device, dtype=t.dtype)
    flat[elements:] = t.reshape(-1)
    return flat[elements:].view(t.shape)


def _zipf(rng, T, V):
    return np.minimum(V - 1, np.floor((V + 1.0) ** rng.random(T)).astype(np.int64) - 1)


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,V,d,off", [
    (1, 1, 1, 0), (3, 2, 7, 0), (5, 9, 8, 0), (33, 100, 64, 0), (70, 50, 333, 0), (17, 40, 1024, 0), (9, 12, 64, 1),
    (2100, 300, 2056, 0), (6000, 1000, 40, 0), (300, 64, 300, 0),
])
def test_embed_forward(txl, T, V, d, off, table, out):
    rng = np.random.default_rng(T * 31 + d)
    tokens = _zipf(rng, T, V)
    tokens[rng.random(T) < 0.2] = rng.choice([-1, V, -2 ** 31, 2 ** 31 - 1])
    tab = _at_offset(_tensor(rng.standard_normal((V, d)), NAMES[table]), off)
    got = _at_offset(torch.full((T, d), float("nan"), device=dev(), dtype=NAMES[out]), off)
    scale = float(np.float32(math.sqrt(d)))
    assert txl.txl_embed_forward(_ints(tokens), tab, got, scale=scale) is got
    want = O.embed(tokens, _host(tab), scale)
    err = np.abs(_host(got) - want)
    assert (err <= (HALF[NAMES[out]] + 2.0 ** -24) * np.abs(want)).all()


def test_embed_forward_values(txl):
    """Rows with infinities and NaN reach only their own tokens; ids of any shape; guards around the output."""
    tab = torch.randn(6, 24, device=dev())
    tab[2, 3], tab[4] = float("inf"), float("nan")
    tokens = _ints([[0, 2, -1], [4, 5, 7]])
    buf = torch.full((8, 24), 7.0, device=dev())
    out = buf[1:7].view(2, 3, 24)
    txl.txl_embed_forward(tokens, tab, out, scale=2.0)
    assert torch.equal(out[0, 0], 2 * tab[0]) and torch.equal(out[0, 1], 2 * tab[2]) and torch.equal(out[1, 1], 2 * tab[5])
    assert not out[0, 2].any() and not out[1, 2].any() and out[1, 0].isnan().all()
    assert (buf[0] == 7).all() and (buf[7] == 7).all()
    txl.txl_embed_forward(tokens[:, :0], tab, out[:, :0])  # no tokens


GRADS = [  # T, V, d, padding, ids: z by frequency, s all the same, u evenly, l a row of the last class only
    (1, 1, 1, 0.0, "z"), (40, 3, 5, 0.3, "u"), (300, 64, 64, 0.0, "z"), (513, 1000, 333, 0.1, "z"), (700, 90, 128, 0.0, "s"),
    (1000, 5000, 130, 0.0, "u"), (2000, 17, 512, 0.0, "z"), (8193, 300, 36, 0.1, "z"), (20000, 40, 24, 0.0, "z"),
    (200, 40000, 8, 0.0, "u"), (64, 1300000, 4, 0.0, "u"), (90, 70, 2304, 0.5, "l"), (50, 20, 16, 1.0, "z"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d,pad,ids", GRADS)
def test_embed_backward(txl, T, V, d, pad, ids, accumulate, dtype):
    rng = np.random.default_rng(T * 7 + V + d)
    tokens = dict(z=lambda: _zipf(rng, T, V), s=lambda: np.full(T, V // 2), u=lambda: rng.integers(0, V, T), l=lambda: np.full(T, V - 1))[ids]()
    tokens[rng.random(T) < pad] = rng.choice([-1, V, 2 ** 31 - 1])
    dout = _tensor(rng.standard_normal((T, d)), NAMES[dtype])
    dout[torch.from_numpy((tokens < 0) | (tokens >= V)).to(dev())] = float("nan")  # padding is not read
    old = np.float32(rng.standard_normal((V, d)))
    named = np.zeros(V, bool)
    named[tokens[(tokens >= 0) & (tokens < V)]] = True
    if accumulate:
        old[~named] = np.nan  # such rows are not touched
    got = torch.from_numpy(old).to(dev())
    scale = float(np.float32(math.sqrt(d)))
    assert txl.txl_embed_backward(_ints(tokens), dout, got, scale=scale, accumulate=accumulate) is got
    grad, size, terms = O.embed_backward(tokens, _host(dout), V, scale)
    have = _host(got)
    if accumulate:
        assert np.isnan(have[~named]).all()
        have, grad, size, terms, kept = have[named], grad[named], size[named], terms[named], old[named].astype(np.float64)
    else:
        assert not have[~named].any()
        kept = np.zeros_like(grad)
    bound = 1.01 * 2.0 ** -24 * ((terms + 1) * size + np.abs(kept + grad))
    assert (np.abs(have - (kept + grad)) <= bound).all()
    again = torch.from_numpy(old).to(dev())
    txl.txl_embed_backward(_ints(tokens), dout, again, scale=scale, accumulate=accumulate)
    assert torch.equal(got.view(torch.int32), again.view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,V,d,pad,ids", [
    (70000, 500, 40, 0.1, "z"), (33001, 9, 20, 0.0, "s"), (40000, 70000, 8, 0.0, "u"), (33000, 5000, 130, 0.2, "z"),
    (2000, 300, 701, 0.0, "z"), (1500, 200, 1201, 0.1, "z"), (9000, 2, 1100, 0.0, "u"),
])
def test_embed_backward_long(txl, T, V, d, pad, ids, accumulate, dtype):
    """More ids than one pass takes, more of one row than a warp lists, and wide rows that start anywhere."""
    test_embed_backward(txl, T, V, d, pad, ids, accumulate, dtype)


def test_embed_backward_unaligned(txl):
    rng = np.random.default_rng(3)
    tokens, V, d = _zipf(rng, 400, 60), 60, 64
    for dtype in (BF, F32):
        dout = _at_offset(_tensor(rng.standard_normal((400, d)), dtype), 1)
        got = _at_offset(torch.full((V, d), float("nan"), device=dev()), 1)
        txl.txl_embed_backward(_at_offset(_ints(tokens), 3), dout, got, scale=0.5)
        grad, size, terms = O.embed_backward(tokens, _host(dout), V, 0.5)
        assert (np.abs(_host(got) - grad) <= 1.01 * 2.0 ** -24 * ((terms + 1) * size + np.abs(grad))).all()


def test_embed_backward_without_tokens(txl):
    tokens, dout = _ints([]), torch.empty(0, 40, device=dev())
    table = torch.ones(2000, 40, device=dev())
    txl.txl_embed_backward(tokens, dout, table, accumulate=True)
    assert (table == 1).all()
    txl.txl_embed_backward(tokens, dout, table)
    assert not table.any()


def test_embed_gradient_is_the_forward_difference(txl):
    """<dout, embed(table)> is linear in the table: a difference of powers of two has no error but its sums' own."""
    rng = np.random.default_rng(4)
    V, d, T = 30, 16, 200
    tokens = _ints(_zipf(rng, T, V))
    dout = _tensor(rng.integers(-8, 9, (T, d)), F32)
    grad = txl.txl_embed_backward(tokens, dout, torch.empty(V, d, device=dev()), scale=4.0)
    for v, c in ((0, 0), (1, 7), (5, 15), (29, 3)):
        table = torch.zeros(V, d, device=dev())
        table[v, c] = 1.0
        out = txl.txl_embed_forward(tokens, table, torch.empty(T, d, device=dev()), scale=4.0)
        assert float((out.double() * dout.double()).sum()) == float(grad[v, c])


# ---------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------
PRODUCTS = [  # m, k, n, group
    (1, 32, 8, 32), (1, 512, 512, 32), (3, 96, 24, 32), (8, 224, 40, 32), (9, 192, 136, 64), (16, 128, 520, 128),
    (17, 640, 72, 128), (32, 2080, 48, 32), (33, 256, 16, 64), (70, 384, 264, 128), (5, 1024, 4096, 64), (4, 4096, 1024, 128),
    (2, 8320, 56, 64), (12, 2304, 2440, 128), (1, 256, 20000, 32), (20, 1152, 5000, 128),
]


def _product(rng, m, k, n, group, integers=False):
    code = rng.integers(0, 16, (n, k))
    codes = torch.from_numpy((code[:, ::2] + 16 * code[:, 1::2]).astype(np.uint8)).to(dev())
    if integers:
        x, scales = rng.integers(-4, 5, (m, k)), 2.0 ** rng.integers(-2, 3, (k // group, n))
    else:
        x, scales = rng.standard_normal((m, k)), (0.5 + rng.random((k // group, n))) * k ** -0.5
    return _tensor(x, BF), codes, _tensor(scales, BF)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,group", PRODUCTS)
def test_dense_w4(txl, m, k, n, group, out):
    rng = np.random.default_rng(m + k + n)
    x, codes, scales = _product(rng, m, k, n, group)
    bias = _tensor(rng.standard_normal(n), F32) if (m + n) % 2 else None
    relu = n % 16 == 8
    buf = torch.full((m + 2, n), 9.0, device=dev(), dtype=NAMES[out])
    y = buf[1:m + 1]
    assert txl.txl_dense_w4(x, codes, scales, y, bias=bias, relu=relu) is y
    W = O.unpack_w4(codes.cpu().numpy(), _host(scales))
    want, size = _host(x) @ W, np.abs(_host(x)) @ np.abs(W)
    if bias is not None:
        want, size = want + _host(bias), size + np.abs(_host(bias))
    if relu:
        want = np.maximum(want, 0)
    # a group's sum, the scaled groups' sum, the warps' sums and the bias
    bound = HALF[NAMES[out]] * np.abs(want) + 1.01 * 2.0 ** -23 * (group + k // group + 16) * size
    assert (np.abs(_host(y) - want) <= bound).all()
    assert (buf[0] == 9).all() and (buf[-1] == 9).all()
    again = torch.empty_like(y)
    txl.txl_dense_w4(x, codes, scales, again, bias=bias, relu=relu)
    assert torch.equal(again, y)


@pytest.mark.parametrize("m,k,n,group", PRODUCTS)
def test_dense_w4_exact(txl, m, k, n, group):
    """Whole numbers and scales of powers of two: no rounding, so every code counts."""
    rng = np.random.default_rng(k)
    x, codes, scales = _product(rng, m, k, n, group, integers=True)
    y = torch.empty(m, n, device=dev())
    txl.txl_dense_w4(x, codes, scales, y)
    assert np.array_equal(_host(y), _host(x) @ O.unpack_w4(codes.cpu().numpy(), _host(scales)))


@pytest.mark.parametrize("m,k,n,group", [
    (32, 4096, 1024, 128), (32, 4096, 4096, 64), (8, 4096, 1024, 32), (70, 4096, 256, 128), (32, 4096, 64, 64), (9, 8320, 264, 64),
    (1, 8192, 40, 32), (16, 4096, 512, 32),
])
def test_dense_w4_shared_k(txl, m, k, n, group):
    """Sizes at which clusters of CTAs share k, x in one stretch and in several."""
    test_dense_w4_exact(txl, m, k, n, group)
    test_dense_w4(txl, m, k, n, group, "bf16")


def test_dense_w4_rows_do_not_meet(txl):
    """A row of x with infinities or NaN, and a column of scales with one, reach only their own outputs."""
    rng = np.random.default_rng(8)
    x, codes, scales = _product(rng, 11, 320, 72, 64)
    clean = torch.empty(11, 72, device=dev())
    txl.txl_dense_w4(x, codes, scales, clean)
    x[4, 7], x[9, 319], scales[2, 30] = float("nan"), float("inf"), float("inf")
    y = torch.empty_like(clean)
    txl.txl_dense_w4(x, codes, scales, y)
    rows, cols = [r for r in range(11) if r not in (4, 9)], [c for c in range(72) if c != 30]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert y[4].isnan().all() and not y[9].isfinite().any() and not y[:, 30].isfinite().any()
    relu = torch.empty_like(clean)
    txl.txl_dense_w4(x, codes, scales, relu, relu=True)
    assert relu[4].isnan().all()  # as txl_dense's products would
    txl.txl_dense_w4(x[:0], codes, scales, y[:0])  # no rows


def test_dense_w4_is_the_same_in_any_batch(txl):
    """A row's sums do not depend on the rows beside it where they share a tile of tokens."""
    rng = np.random.default_rng(9)
    x, codes, scales = _product(rng, 8, 512, 256, 128)
    y = torch.empty(8, 256, device=dev())
    txl.txl_dense_w4(x, codes, scales, y)
    for m in (1, 3, 7):
        part = torch.empty(m, 256, device=dev())
        txl.txl_dense_w4(x[:m], codes, scales, part)
        assert torch.equal(part, y[:m])


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------
def _check_sample(txl, z, u, **settings):
    """Every row's token and share.  u is drawn, so that it lies within the weights' error (2^-36 of the whole) of a
    border with a chance of 2^-35 for each kept token; such a row would not say anything."""
    B = z.shape[0]
    one = {k: v for k, v in settings.items() if v is not None}
    t = {k: torch.as_tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else F32).to(dev()) for k, v in one.items()}
    tokens = torch.full((B,), -7, device=dev(), dtype=torch.int32)
    prob = torch.full((B,), -7.0, device=dev())
    ud = torch.as_tensor(np.asarray(u), dtype=F32).to(dev())
    assert txl.txl_sample(z, ud, tokens, prob=prob, **t) is tokens
    zs, got, share = _host(z), tokens.cpu().numpy(), prob.cpu().numpy()
    for b in range(B):
        own = {k: (int(v[b]) if k == "top_k" else float(np.float32(v[b]))) for k, v in one.items()}
        want, p, near = O.sample(zs[b], float(np.float32(u[b])), **own)
        assert near > 2.0 ** -36 or len(O.keep(zs[b], **own)[0]) == 1 or float(np.float32(u[b])) in (0.0, 1.0), "a row that says nothing"
        assert got[b] == want, (b, own)
        assert abs(share[b] - p) <= 2.0 ** -22 * p, (b, own)
    only = torch.empty_like(tokens)
    txl.txl_sample(z, ud, only, **t)  # without prob
    assert torch.equal(only, tokens)


SETTINGS = [
    {}, dict(temperature=(0.3, 1.7)), dict(top_k=(1, 40)), dict(top_p=(0.1, 0.999)), dict(min_p=(0.001, 0.3)), dict(top_k=(1, 3000), top_p=(0.3, 1.0)),
    dict(temperature=(0.2, 2.0), top_k=(5, 500), top_p=(0.5, 0.99), min_p=(0.0001, 0.05)), dict(temperature=(0.5, 1.5), top_p=(0.9, 0.9999)),
    dict(top_p=(0.8, 0.999), min_p=(0.0001, 0.2)), dict(temperature=(0.01, 50.0), min_p=(0.0001, 1.0)),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("settings", SETTINGS, ids=[" ".join(s) or "none" for s in SETTINGS])
@pytest.mark.parametrize("B,V", [(3, 1), (4, 2), (9, 33), (6, 1000), (5, 2049), (3, 30011), (2, 131072)])
def test_sample(txl, B, V, settings, dtype):
    rng = np.random.default_rng(V + B + len(settings))
    z = 2.5 * rng.standard_normal((B, V)) + 8 * (rng.random((B, V)) < 10 / V)
    z = _tensor(z, NAMES[dtype])
    s = {k: rng.uniform(*v, B) for k, v in settings.items()}
    if "top_k" in s:
        s["top_k"] = s["top_k"].astype(int)
    _check_sample(txl, z, rng.random(B), **s)


@pytest.mark.parametrize("kind", ["equal", "two values", "wide", "masked", "lowest", "inf", "tiny", "empty", "steps"])
@pytest.mark.parametrize("V", [64, 5000, 40000])
def test_sample_hard_rows(txl, kind, V):
    """Rows that the search's bins do not separate at once: equal logits, logits of all sizes, masks of -inf and of the
    type's lowest value, NaN, denormals, +inf, nothing to keep."""
    rng = np.random.default_rng(V)
    n = 6
    z = rng.standard_normal((n, V))
    if kind == "equal":
        z[:] = 1.25
    elif kind == "two values":
        z = np.where(rng.random((n, V)) < 0.5, 0.5, -0.0)
    elif kind == "wide":
        z = np.sign(z) * 10.0 ** rng.uniform(-38, 38, (n, V))
    elif kind == "masked":
        z[rng.random((n, V)) < 0.7] = -np.inf
        z[rng.random((n, V)) < 0.1] = np.nan
        z[:, 5] = 1.0
    elif kind == "lowest":
        z[rng.random((n, V)) < 0.7] = -3.4028234663852886e38
        z[1] = -3.4028234663852886e38
        z[:, -1] = -1e4
    elif kind == "inf":
        z[:, ::7] = np.inf
    elif kind == "tiny":
        z = 1e-42 * rng.integers(-50, 50, (n, V))
    elif kind == "empty":
        z[0], z[1], z[2, 1:], z[3, :-1] = -np.inf, np.nan, -np.inf, np.nan
    elif kind == "steps":
        z = np.float32(1.0) + np.float32(2.0 ** -23) * rng.integers(0, 3000, (n, V))  # neighbours in fp32
    z = _tensor(z, F32)
    u = rng.random(n)
    for s in ({}, dict(top_k=[1, 2, 7, V // 2, V - 1, V + 5]), dict(top_p=[0.0, 0.1, 0.5, 0.9, 0.999, 1.0]),
              dict(top_k=[3, 30, 60, V // 3, V - 1, 0], top_p=[0.3, 0.5, 0.7, 0.9, 0.99, 0.5]),
              dict(min_p=[1.0, 0.5, 2.0, 0.1, 1e-5, 0.0], temperature=[1.0, 0.5, 3.0, 0.1, 10.0, 1e-3]),
              dict(temperature=[0.0, -1.0, np.nan, 0.0, 0.0, 0.0], top_p=[0.5] * n)):
        _check_sample(txl, z, u, **s)


def test_sample_borders(txl):
    """Uniform numbers at and past the ends; settings past theirs; a warm temperature makes all weights equal."""
    rng = np.random.default_rng(5)
    z = _tensor(rng.integers(-3, 4, (8, 300)), BF)
    _check_sample(txl, z, [0.0, 1.0, 1.0, 0.0, 1.0, 0.0, 1.0, 0.0], top_k=[0, 0, 5, 5, -3, 1 << 30, 2, 2])
    tokens = torch.empty(8, device=dev(), dtype=torch.int32)
    u = torch.tensor([-1.0, 2.0, float("nan"), float("-inf"), float("inf"), 0.0, 1.0, -0.0], device=dev())
    txl.txl_sample(z, u, tokens)
    assert tokens.tolist() == [0, 299, 0, 0, 299, 0, 299, 0]
    nan = torch.full((8,), float("nan"), device=dev())
    plain, off = torch.empty_like(tokens), torch.empty_like(tokens)
    half = torch.full((8,), 0.37, device=dev())
    txl.txl_sample(z, half, plain)
    txl.txl_sample(z, half, off, top_p=nan, min_p=nan, top_k=torch.zeros(8, device=dev(), dtype=torch.int32))
    assert torch.equal(plain, off)
    txl.txl_sample(z, half, off, temperature=torch.full((8,), float("inf"), device=dev()))
    assert off.tolist() == [111] * 8  # the first index over 0.37 of 300 equal weights


def test_sample_rows_apart(txl):
    """Rows with a distance, from an odd element on; every row as if alone."""
    rng = np.random.default_rng(6)
    for dtype, V, stride, off in ((BF, 1000, 1024, 0), (BF, 1000, 1003, 0), (F32, 77, 80, 3), (F32, 4096, 4100, 0)):
        wide = _tensor(rng.standard_normal((7, stride)) * 3, dtype)
        z = _at_offset(wide, off)[:, :V]
        u = rng.random(7)
        _check_sample(txl, z, u, top_k=rng.integers(1, 60, 7), top_p=rng.uniform(0.5, 1, 7))
        both, one = torch.empty(7, device=dev(), dtype=torch.int32), torch.empty(1, device=dev(), dtype=torch.int32)
        ud = _tensor(u, F32)
        txl.txl_sample(z, ud, both)
        for b in range(7):
            txl.txl_sample(z[b:b + 1], ud[b:b + 1], one)
            assert int(one) == int(both[b])


def test_sample_many_rows(txl):
    rng = np.random.default_rng(7)
    z = _tensor(rng.standard_normal((700, 200)) * 2, BF)
    _check_sample(txl, z, rng.random(700), top_k=rng.integers(0, 50, 700), top_p=rng.uniform(0.2, 1.2, 700))


def test_sample_longest_rows(txl):
    """The largest vocabulary; all its weights equal, so that the sum is the largest there is."""
    V = 1 << 18
    z = torch.zeros(2, V, device=dev())
    z[1] = torch.from_numpy(np.random.default_rng(8).standard_normal(V).astype(np.float32)).to(dev())
    tokens = torch.empty(2, device=dev(), dtype=torch.int32)
    u = torch.tensor([0.7, 0.7], device=dev())
    txl.txl_sample(z, u, tokens)
    assert int(tokens[0]) == math.floor(float(u[0]) * V)
    upto = np.exp(_host(z[1]) - _host(z[1]).max()).cumsum()
    assert int(tokens[1]) == int(np.searchsorted(upto, float(u[1]) * upto[-1], side="right"))
    txl.txl_sample(z, u, tokens, top_k=_ints([V - 1, 1000]), top_p=torch.tensor([0.5, 0.5], device=dev()))
    assert int(tokens[0]) == math.floor(float(u[0]) * math.ceil(0.5 * (V - 1)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,V", [(1, 131072), (3, 70000), (20, 90000), (60, 20000), (30, 20000), (160, 20011), (12, 70001), (2, 1 << 18)])
def test_sample_shared_rows(txl, B, V, dtype):
    """Rows that one, two, four or eight CTAs share."""
    rng = np.random.default_rng(V + B)
    z = _tensor(2.0 * rng.standard_normal((B, V)) + 6 * (rng.random((B, V)) < 30 / V), NAMES[dtype])
    _check_sample(txl, z, rng.random(B), top_k=rng.integers(0, 600, B), top_p=rng.uniform(0.5, 1.1, B), min_p=rng.uniform(0, 0.01, B))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [0, 300, 50000, 130800])
def test_sample_largest_together(txl, first, dtype):
    """The largest tokens in one CTA's stretch, more than it can hand over at once."""
    rng = np.random.default_rng(first)
    z = rng.standard_normal((4, 131072))
    z[:, first:first + 240] += 9
    z = _tensor(z, NAMES[dtype])
    for k in (60, 100, 200, 256, 700):
        for s in ({}, dict(top_p=[0.3, 0.8, 0.95, 1.0]), dict(min_p=[0.5, 0.1, 0.01, 0.0])):
            _check_sample(txl, z[:1], rng.random(1), top_k=[k], **{n: v[:1] for n, v in s.items()})
            _check_sample(txl, z, rng.random(4), top_k=[k] * 4, **s)
    wide = rng.standard_normal((3, 131072))
    wide[:, first:first + 480] += 9
    for k in (300, 450, 480, 512, 513):
        _check_sample(txl, _tensor(wide, F32), rng.random(3), top_k=[k] * 3, top_p=[0.6, 0.99, 1.0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 20000, 131072])
def test_sample_few_that_matter(txl, V, dtype):
    """A few tokens with most of the weight: the border of top-p is far from where the bins' middles put it."""
    rng = np.random.default_rng(V)
    for lead in (1, 2, 3, 9):
        z = rng.standard_normal((5, V))
        at = rng.integers(0, V, (5, lead))
        np.put_along_axis(z, at, 18 + rng.random((5, lead)), 1)
        _check_sample(txl, _tensor(z, NAMES[dtype]), rng.random(5), top_p=[0.2, 0.6, 0.9, 0.999, 0.9999999])
        _check_sample(txl, _tensor(40 * z, NAMES[dtype]), rng.random(5), top_p=[0.2, 0.6, 0.9, 0.999, 0.9999999], temperature=[30.0] * 5)


@pytest.mark.parametrize("V", [64, 5000, 40000])
def test_sample_hard_rows_bf16(txl, V):
    """In bf16: equal logits (there are few values), +inf, masks of -inf and of the type's lowest value, NaN."""
    rng = np.random.default_rng(V + 1)
    z = rng.integers(-2, 3, (6, V)).astype(np.float64)
    z[1, rng.random(V) < 0.5] = -np.inf
    z[2, rng.random(V) < 0.5] = -3.3895313892515355e38
    z[3, ::5] = np.inf
    z[4, rng.random(V) < 0.5] = np.nan
    z[5] = -np.inf
    z = _tensor(z, BF)
    u = rng.random(6)
    for s in ({}, dict(top_k=[1, 3, V // 2, V, 9, 4]), dict(top_p=[0.1, 0.5, 0.9, 0.3, 0.99, 0.5]),
              dict(top_k=[200, 20, V // 3, 2, 0, 1], top_p=[0.7] * 6, min_p=[0.2] * 6), dict(temperature=[0.0] * 6)):
        _check_sample(txl, z, u, **s)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _settle():
    torch.cuda.synchronize()


def test_calls_on_streams_and_graphs(txl):
    """Each call on another stream, then captured and replayed on changed inputs; a default-stream call of the same
    shapes runs beside it."""
    rng = np.random.default_rng(10)
    V, d, T = 500, 256, 64
    table = _tensor(rng.standard_normal((V, d)), BF)
    x, codes, scales = _product(rng, T, d, V // 8 * 8, 64)
    tokens, h = _ints(rng.integers(0, V, T)), torch.empty(T, d, device=dev(), dtype=BF)
    logits, grad = torch.empty(T, codes.shape[0], device=dev()), torch.empty(V, d, device=dev())
    u, out = _tensor(rng.random(T), F32), torch.empty(T, device=dev(), dtype=torch.int32)
    k, p = _ints(np.full(T, 20)), torch.full((T,), 0.9, device=dev())

    def step():
        txl.txl_embed_forward(tokens, table, h, scale=0.5)
        txl.txl_dense_w4(h, codes, scales, logits)
        txl.txl_sample(logits, u, out, top_k=k, top_p=p)
        txl.txl_embed_backward(tokens, h, grad, scale=0.5)

    def results():
        _settle()
        return [t.clone() for t in (h, logits, out, grad)]

    step()
    want = results()
    side = torch.cuda.Stream()
    for t in (h, logits, grad):
        t.fill_(float("nan"))
    _settle()
    with torch.cuda.stream(side):
        step()
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12):
        tokens.copy_(_ints(np.random.default_rng(seed).integers(-1, V, T)))
        u.copy_(_tensor(np.random.default_rng(seed).random(T), F32))
        step()
        want = results()
        for t in (h, logits, grad):
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    handle = side.cuda_stream
    txl.txl_embed_forward(tokens, table, h, 0.5, stream=handle)
    txl.txl_dense_w4(h, codes, scales, logits, stream=side)
    txl.txl_sample(logits, u, out, top_k=k, top_p=p, stream=side)
    txl.txl_embed_backward(tokens, h, grad, 0.5, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(results(), want))


def test_calls_of_many_threads(txl):
    """Calls of other sizes from several threads, each on its own stream, at the same time: a call's shared memory is
    its own, whatever the last one of the same kernel needed."""
    lib, ptr = txl.lib, torch.Tensor.data_ptr
    rng = np.random.default_rng(15)
    jobs = []
    for V, k, n in ((64, 128, 64), (30000, 4096, 256), (2000, 512, 64), (20000, 2048, 128)):
        z, u, out = _tensor(rng.standard_normal((2, V)), F32), torch.full((2,), 0.5, device=dev()), torch.empty(2, device=dev(), dtype=torch.int32)
        x, codes, scales = _product(rng, 4, k, n, 32)
        y, tokens = torch.empty(4, n, device=dev(), dtype=BF), _ints(rng.integers(0, V, 100))
        dout, grad = _tensor(rng.standard_normal((100, 16)), F32), torch.empty(V, 16, device=dev())
        jobs.append((V, k, n, z, u, out, x, codes, scales, y, tokens, dout, grad, torch.cuda.Stream()))
    want = []
    for V, k, n, z, u, out, x, codes, scales, y, tokens, dout, grad, _ in jobs:
        txl.txl_sample(z, u, out)
        txl.txl_dense_w4(x, codes, scales, y)
        txl.txl_embed_backward(tokens, dout, grad)
        want.append([t.clone() for t in (out, y, grad)])
    _settle()
    bad, start = [], threading.Barrier(len(jobs))

    def run(V, k, n, z, u, out, x, codes, scales, y, tokens, dout, grad, stream):
        s = stream.cuda_stream
        start.wait()
        for _ in range(300):
            bad.append(lib.txl_sample(ptr(z), V, 2, V, ptr(u), None, None, None, None, ptr(out), None, 0, s))
            bad.append(lib.txl_dense_w4(ptr(x), ptr(codes), ptr(scales), ptr(y), 4, n, k, 32, None, 0, 1, s))
            bad.append(lib.txl_embed_backward(ptr(tokens), ptr(dout), ptr(grad), 100, V, 16, 1.0, 0, 0, s))

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _settle()
    assert sum(bad) == 0, (sum(b != 0 for b in bad), len(bad))
    for (_, _, _, _, _, out, _, _, _, y, _, _, grad, _), w in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip((out, y, grad), w))


def test_decoding_over_pages(txl):
    """A small decoder's steps: ids to rows, their products with 4-bit weights, the paged memory and the attention over
    it, the logits, the next ids.  Each call's result against the oracle on the inputs that it had."""
    rng = np.random.default_rng(13)
    n, H, D, P, V, group, steps = 3, 2, 64, 16, 320, 64, 5
    d = H * D
    table = _tensor(rng.standard_normal((V, d)) * 0.3, BF)
    weights = {w: _product(rng, 1, d, c, group)[1:] for w, c in (("q", d), ("k", d), ("v", d), ("o", d), ("logits", V))}
    W = {w: O.unpack_w4(c.cpu().numpy(), _host(s)) for w, (c, s) in weights.items()}
    r = _tensor(rng.standard_normal((64, H, D)) * 0.3, BF)
    bu, bv = (_tensor(rng.standard_normal((H, D)) * 0.1, F32) for _ in range(2))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev())  # noqa: E731
    book = dict(table=i32(n, 8) - 1, start=i32(n), rows=i32(n), refs=i32(24))
    pools = [torch.full((24, H, P, D), float("nan"), device=dev(), dtype=BF) for _ in range(2)]
    slots, cu, granted, src, dst = _ints(range(n)), _ints(range(n + 1)), i32(n), i32(n), i32(n)
    tokens = _ints(rng.integers(0, V, n))
    bf = lambda: torch.empty(n, d, device=dev(), dtype=BF)  # noqa: E731
    h, q, kn, vn, a, y = (bf() for _ in range(6))
    z, prob = torch.empty(n, V, device=dev()), torch.empty(n, device=dev())
    u = _tensor(rng.random((steps, n)), F32)
    temperature, top_k, top_p = torch.full((n,), 0.8, device=dev()), _ints([0, 40, 5]), torch.tensor([0.9, 1.0, 0.8], device=dev())
    ws = torch.empty(txl.txl_relattn_paged_workspace_bytes(n, n, H, D, BF), dtype=torch.uint8, device=dev())
    keys, values = [], []

    def close(got, x, w, dtype=BF):
        want, size = _host(x) @ W[w], np.abs(_host(x)) @ np.abs(W[w])
        bound = HALF[dtype] * np.abs(want) + 1.01 * 2.0 ** -23 * (group + d // group + 16) * size
        assert (np.abs(_host(got) - want) <= bound).all(), w

    for step in range(steps):
        before = tokens.clone()
        txl.txl_embed_forward(tokens, table, h, scale=d ** 0.5)
        for w, out in (("q", q), ("k", kn), ("v", vn)):
            txl.txl_dense_w4(h, *weights[w], out)
        txl.txl_pages_reserve(book, P, slots, cu, granted, src, dst)
        txl.txl_pages_append(book, *pools, slots, cu, granted, src, dst, kn.view(n, H, D), vn.view(n, H, D))
        txl.txl_relattn_forward_paged(q.view(n, H, D), *pools, book, slots, cu, r, bu, bv, a.view(n, H, D), ws, max_new=1)
        txl.txl_dense_w4(a, *weights["o"], y)
        txl.txl_dense_w4(y, *weights["logits"], z)
        txl.txl_sample(z, u[step], tokens, temperature=temperature, top_k=top_k, top_p=top_p, prob=prob)
        assert txl.txl_get_device_status() == 0
        scale = float(np.float32(d ** 0.5))
        rows = O.embed(before.cpu().numpy(), _host(table), scale)
        assert (np.abs(_host(h) - rows) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(rows)).all()
        for w, got in (("q", q), ("k", kn), ("v", vn)):
            close(got, h, w)
        keys.append(_host(kn).reshape(n, H, D))
        values.append(_host(vn).reshape(n, H, D))
        K, Vv, Q, R = np.stack(keys, 1), np.stack(values, 1), _host(q).reshape(n, H, D), _host(r)[step::-1][:step + 1]
        s = np.einsum("bhd,bjhd->bhj", Q + _host(bu), K) + np.einsum("bhd,jhd->bhj", Q + _host(bv), R)
        p = np.exp((s - s.max(2, keepdims=True)) * D ** -0.5)
        att = np.einsum("bhj,bjhd->bhd", p / p.sum(2, keepdims=True), Vv).reshape(n, d)
        # Half a step of bf16 is 2^-8 of the value, here up to 60: an absolute 2e-2 would be less than that.  Besides,
        # q + u, q + v and the weights keep 16 bits: scores are off by e = 2^-16 of their terms' sizes, a weight by
        # 2^-16 + e of itself, and the quotient of the two sums by twice that of the largest value.
        terms = np.einsum("bhd,bjhd->bhj", np.abs(Q + _host(bu)), np.abs(K)) + np.einsum("bhd,jhd->bhj", np.abs(Q + _host(bv)), np.abs(R))
        off = 2 * (2.0 ** -16 + 2.0 ** -16 * D ** -0.5 * terms.max(2))[:, :, None] * np.abs(Vv).max(1)
        assert (np.abs(_host(a) - att) <= 2.0 ** -8 * np.abs(att) + 1.01 * off.reshape(n, d)).all()
        assert np.linalg.norm(_host(a) - att) <= 5e-3 * np.linalg.norm(att)
        close(y, a, "o")
        close(z, y, "logits", F32)
        for b in range(n):
            want, share, near = O.sample(_host(z)[b], float(u[step, b]), temperature=float(temperature[b]), top_k=int(top_k[b]),
                                         top_p=float(top_p[b]))
            assert near > 2.0 ** -36 and int(tokens[b]) == want and abs(float(prob[b]) - share) <= 2.0 ** -22 * share


def test_training_step_of_the_table(txl):
    """Ids to rows, attention of a segment, its gradient, and the table's: the embedding's gradient on the attention's."""
    rng = np.random.default_rng(14)
    B, W, H, D, V = 2, 40, 2, 64, 50
    d = H * D
    table = _tensor(rng.standard_normal((V, d)) * 0.05, BF)
    tokens = _ints(_zipf(rng, B * W, V).reshape(B, W))
    q = torch.empty(B, W, d, device=dev(), dtype=BF)
    txl.txl_embed_forward(tokens, table, q, scale=2.0)
    qh = q.view(B, W, H, D)
    k, v, r = (_tensor(rng.standard_normal(s), BF) for s in ((B, W, H, D), (B, W, H, D), (W, H, D)))
    u = torch.zeros(H, D, device=dev())
    o, lse = torch.empty_like(qh), torch.empty(B, H, W, device=dev())
    txl.txl_relattn_forward(qh, k, v, r, u, u, o, lse)
    dq = txl.txl_relattn_backward(qh, k, v, r, u, u, o, lse, _tensor(rng.standard_normal((B, W, H, D)), BF))["dq"]
    grad = txl.txl_embed_backward(tokens, dq.view(B, W, d), torch.empty(V, d, device=dev()), scale=2.0)
    want, size, terms = O.embed_backward(tokens.cpu().numpy().ravel(), _host(dq).reshape(-1, d), V, 2.0)
    assert (np.abs(_host(grad) - want) <= 1.01 * 2.0 ** -24 * ((terms + 1) * size + np.abs(want))).all()
    assert txl.txl_get_device_status() == 0


def test_bindings_refuse(txl):
    """Wrong types, shapes and layouts, before any launch."""
    i, f = _ints([0, 1]), torch.zeros(2, device=dev())
    table, out = torch.zeros(4, 32, device=dev()), torch.zeros(2, 32, device=dev())
    x, codes, scales = torch.zeros(2, 64, device=dev(), dtype=BF), torch.zeros(8, 32, device=dev(), dtype=torch.uint8), torch.zeros(2, 8, device=dev(), dtype=BF)
    y = torch.zeros(2, 8, device=dev())
    bad = [
        lambda: txl.txl_embed_forward(i.long(), table, out), lambda: txl.txl_embed_forward(i, table, out[:, :31]),
        lambda: txl.txl_embed_forward(i, table.half(), out), lambda: txl.txl_embed_forward(i, table[:, ::2], out[:, :16]),
        lambda: txl.txl_embed_backward(i, out, table.to(BF)), lambda: txl.txl_embed_backward(i, out[:1], table),
        lambda: txl.txl_dense_w4(x.float(), codes, scales, y), lambda: txl.txl_dense_w4(x, codes.int(), scales, y),
        lambda: txl.txl_dense_w4(x, codes, scales.float(), y), lambda: txl.txl_dense_w4(x, codes[:, :31], scales, y),
        lambda: txl.txl_dense_w4(x, codes, scales[:0], y), lambda: txl.txl_dense_w4(x, codes, scales, y[:1]),
        lambda: txl.txl_dense_w4(x, codes, scales, y, bias=f), lambda: txl.txl_dense_w4(x, codes, scales, y.half()),
        lambda: txl.txl_sample(y, f, i.long()), lambda: txl.txl_sample(y, f[:1], i), lambda: txl.txl_sample(y, None, i),
        lambda: txl.txl_sample(y.t(), torch.zeros(8, device=dev()), _ints(range(8))), lambda: txl.txl_sample(y, f, i, top_k=f),
        lambda: txl.txl_sample(y, f, i, temperature=i), lambda: txl.txl_sample(y, f.cpu(), i), lambda: txl.txl_sample(y.cpu(), f, i),
        lambda: txl.txl_sample(y[:1].expand(2, 8), f, i),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(n)
    for group in (16, 48):
        with pytest.raises(txl.TxlError) as e:
            txl.txl_dense_w4(torch.zeros(1, 96, device=dev(), dtype=BF), torch.zeros(8, 48, device=dev(), dtype=torch.uint8),
                             torch.zeros(96 // group, 8, device=dev(), dtype=BF), torch.zeros(1, 8, device=dev()))
        assert e.value.status == 2
    with pytest.raises(txl.TxlError) as e:
        txl.txl_sample(y, f, f.view(torch.int32))
    assert e.value.status == 3
