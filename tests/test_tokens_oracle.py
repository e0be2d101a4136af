"""The operators around the layers on the CPU: the oracle against what it does not
share its steps with, and the calls' refusals, which come before any launch."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import test_library_cpu as base
from oracle import tokens_oracle as O


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------
def test_embedding_is_a_product_with_the_indicator():
    rng = np.random.default_rng(0)
    table, tokens = rng.standard_normal((7, 5)), np.array([3, 0, 6, 3, -1, 7, 3])
    ones = (tokens[:, None] == np.arange(7)).astype(float)
    assert np.allclose(O.embed(tokens, table, 1.5), 1.5 * ones @ table, rtol=1e-15, atol=0)
    dout = rng.standard_normal((7, 5))
    grad, size, terms = O.embed_backward(tokens, dout, 7, 1.5)
    assert np.allclose(grad, 1.5 * ones.T @ dout, rtol=1e-14, atol=1e-15)
    assert np.allclose(size, 1.5 * ones.T @ np.abs(dout), rtol=1e-14) and terms.ravel().tolist() == [1, 0, 0, 3, 0, 0, 1]
    # the forward is linear in the table: its differences are the gradient
    for v, c in ((3, 1), (6, 4), (1, 0)):
        e = np.zeros_like(table)
        e[v, c] = 0.5
        up, down = (np.sum(dout * O.embed(tokens, table + s * e, 1.5)) for s in (1, -1))
        assert math.isclose(up - down, grad[v, c], rel_tol=1e-12, abs_tol=1e-12)


def test_codes_by_their_digits():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (6, 64))
    scales = rng.standard_normal((2, 6))
    codes = (code[:, ::2] + 16 * code[:, 1::2]).astype(np.uint8)
    W = O.unpack_w4(codes, scales)
    for j, i in ((0, 0), (1, 0), (31, 5), (32, 5), (63, 2)):
        assert W[j, i] == scales[j // 32, i] * (int(code[i, j]) - 8)


@pytest.mark.parametrize("settings", [{}, dict(top_k=4), dict(top_p=0.7), dict(min_p=0.1), dict(temperature=0.0),
                                      dict(temperature=2.0, top_k=6, top_p=0.8, min_p=0.05)])
def test_sample_shares(settings):
    """Uniform numbers over [0, 1) name each kept token as often as its share of the weights says."""
    z = np.array([1.0, 3.0, -2.0, 3.0, 0.5, 2.0, -math.inf, math.nan, 0.0, 2.0])
    n = 4000
    got = np.bincount([O.sample(z, (i + 0.5) / n, **settings)[0] for i in range(n)], minlength=len(z))
    t = settings.get("temperature", 1.0)
    ok = np.isfinite(z)
    w = np.where(ok, np.exp(np.where(ok, z, 0) / (t or 1.0)), 0.0)
    order = np.argsort(-np.where(ok, z, -np.inf), kind="stable")
    mask = np.zeros(len(z), bool)
    if t == 0:
        mask[order[0]] = True
    else:
        k = settings.get("top_k") or len(z)
        top = order[:k]
        share = w[top] / w[top].sum()
        mask[top[np.concatenate([[0.0], share.cumsum()[:-1]]) < settings.get("top_p", 2.0)]] = True
        mask &= w >= settings.get("min_p", 0.0) * w.max()
    want = w * mask / (w * mask).sum()
    assert np.abs(got / n - want).max() <= 1 / n
    assert all(O.sample(z, u, **settings)[1] == pytest.approx(want[O.sample(z, u, **settings)[0]], rel=1e-12)
               for u in (0.0, 0.3, 0.77, 0.999, 1.0))


def test_sample_edges():
    assert O.sample([-math.inf, math.nan], 0.3)[0] == -1
    assert O.sample([1.0, 1.0, 1.0], 0.9, top_k=2)[0] == 1      # equal ones by index
    assert O.sample([1.0, 1.0, 1.0, 1.0], 0.99, top_p=0.5)[0] == 1  # two of four make up a half
    assert O.sample([0.0, 5.0], 0.99, top_p=0.0)[0] == 1        # one at least
    assert O.sample([0.0, math.inf, -3.4e38], 0.99)[0] == 1


# ---------------------------------------------------------------------------
# refusals: addresses that nothing reads
# ---------------------------------------------------------------------------
OK, ARG, UNSUPPORTED, ALIAS = 0, 1, 2, 3
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    base._build_if_missing()
    import transformer_xl_relative_txl_gb300 as txl

    return txl.lib


def test_embed_forward_refusals(lib):
    f = lambda tok=A, tab=B, out=C, T=4, V=8, d=16, td=1, od=1: lib.txl_embed_forward(tok, tab, out, T, V, d, 1.0, td, od, None)  # noqa: E731
    assert f(T=0) == OK and f(T=0, tok=None) == OK
    assert f(T=-1) == ARG and f(V=0) == ARG and f(d=0) == ARG and f(td=2) == ARG and f(od=-1) == ARG
    assert f(tok=None) == ARG and f(tab=None) == ARG and f(out=None) == ARG
    assert f(tok=A + 2) == ARG and f(tab=B + 1) == ARG and f(out=C + 2, od=0) == ARG
    assert f(V=(1 << 24) + 1) == UNSUPPORTED and f(d=(1 << 20) + 1) == UNSUPPORTED and f(T=(1 << 30) + 1) == UNSUPPORTED
    assert f(out=B + 8 * 16 * 2 - 2) == ALIAS and f(out=A + 12) == ALIAS and f(tab=C + 4 * 16 * 2 - 2) == ALIAS


def test_embed_backward_refusals(lib):
    f = lambda tok=A, dout=B, dt=C, T=4, V=8, d=16, acc=0, ty=1: lib.txl_embed_backward(tok, dout, dt, T, V, d, 1.0, acc, ty, None)  # noqa: E731
    assert f(T=0, acc=1) == OK
    assert f(T=-1) == ARG and f(V=0) == ARG and f(d=-3) == ARG and f(ty=5) == ARG
    assert f(tok=None) == ARG and f(dout=None) == ARG and f(dt=None) == ARG and f(dt=None, T=0) == ARG
    assert f(tok=A + 1) == ARG and f(dout=B + 1) == ARG and f(dt=C + 2) == ARG
    assert f(V=(1 << 24) + 1) == UNSUPPORTED and f(d=(1 << 20) + 1) == UNSUPPORTED and f(T=(1 << 30) + 1) == UNSUPPORTED
    assert f(dt=B + 4 * 16 * 2 - 4) == ALIAS and f(dt=A) == ALIAS


def test_dense_w4_refusals(lib):
    f = lambda x=A, c=B, s=C, y=D, m=2, n=16, k=64, g=32, b=None, yt=1: lib.txl_dense_w4(x, c, s, y, m, n, k, g, b, 0, yt, None)  # noqa: E731
    assert f(m=0) == OK
    assert f(m=-1) == ARG and f(n=0) == ARG and f(k=0) == ARG and f(yt=3) == ARG
    assert f(g=16) == UNSUPPORTED and f(g=48, k=96) == UNSUPPORTED and f(g=64, k=96) == UNSUPPORTED
    assert f(g=0) == UNSUPPORTED and f(g=-32) == UNSUPPORTED and f(g=256, k=256) == UNSUPPORTED and f(n=12) == UNSUPPORTED
    assert f(m=(1 << 20) + 1) == UNSUPPORTED and f(n=(1 << 30) + 8) == UNSUPPORTED and f(k=(1 << 24) + 32) == UNSUPPORTED
    assert f(x=None) == ARG and f(c=None) == ARG and f(s=None) == ARG and f(y=None) == ARG
    assert f(x=A + 8) == ARG and f(c=B + 4) == ARG and f(s=C + 2) == ARG and f(y=D + 1) == ARG and f(b=E + 2) == ARG
    assert f(y=A) == ALIAS and f(y=B + 16 * 32 - 2) == ALIAS and f(y=C) == ALIAS and f(y=D, b=D + 60) == ALIAS


def test_sample_refusals(lib):
    def f(z=A, rs=100, n=2, V=100, u=B, t=None, k=None, p=None, mp=None, tok=C, pr=None, ty=1):
        return lib.txl_sample(z, rs, n, V, u, t, k, p, mp, tok, pr, ty, None)

    assert f(n=0) == OK
    assert f(n=-1) == ARG and f(V=0) == ARG and f(rs=99) == ARG and f(ty=2) == ARG
    assert f(V=(1 << 18) + 1, rs=1 << 19) == UNSUPPORTED and f(n=65536) == UNSUPPORTED and f(rs=(1 << 40) + 1) == UNSUPPORTED
    assert f(z=None) == ARG and f(u=None) == ARG and f(tok=None) == ARG
    assert f(z=A + 1) == ARG and f(u=B + 2) == ARG and f(t=D + 1) == ARG and f(pr=E + 3) == ARG and f(tok=C + 2) == ARG
    assert f(tok=A + 396) == ALIAS and f(tok=B + 4) == ALIAS and f(pr=C + 4) == ALIAS and f(pr=D, mp=D) == ALIAS
    assert f(pr=E, k=E + 4) == ALIAS and f(tok=A + 4 * 300, rs=600) == ALIAS


def test_binding_refuses_host_tensors(lib):
    import transformer_xl_relative_txl_gb300 as txl

    i, f, b = torch.zeros(2, dtype=torch.int32), torch.zeros(2), torch.zeros(2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        txl.txl_embed_forward(i, torch.zeros(4, 32), torch.zeros(2, 32))
    with pytest.raises(ValueError):
        txl.txl_embed_backward(i, b, torch.zeros(4, 32))
    with pytest.raises(ValueError):
        txl.txl_dense_w4(b, torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(1, 8, dtype=torch.bfloat16), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        txl.txl_sample(b, f, i)
    with pytest.raises(TypeError):
        txl.txl_sample(None, f, i)
    assert ctypes.sizeof(ctypes.c_longlong) == 8


# ---------------------------------------------------------------------------
# what the kernels' sources say
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["embed", "dense_w4", "sample"])
def test_nothing_is_touched_ahead_of_the_wait(name):
    """A kernel that starts while the one before it runs reads and writes no global memory, no other CTA's, and lets no
    kernel start, until it has waited; and it waits whatever its arguments."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_xl_relative_txl_gb300", "csrc", name + ".cu")
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    bodies = re.findall(r"__global__ void\s+__launch_bounds__.*?\{(.*?)\n\}\n", text, re.S)
    assert len(bodies) == {"embed": 2, "dense_w4": 1, "sample": 1}[name]
    for body in bodies:
        ahead, wait, _ = body.partition("grid_dep_wait();")
        assert wait
        assert not re.search(r"__ldg|load|copy16|fetch|atomic|\bred\b|prefetch|map_shared_rank|launch_dependents|return|p\.\w+\[|kPowers", ahead)


@pytest.mark.parametrize("name", ["embed", "dense_w4", "sample"])
def test_the_cap_on_shared_memory_is_no_call_s_own(name):
    """Two threads' calls of one kernel must not undo each other's cap: it is a constant of the kernel."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_xl_relative_txl_gb300", "csrc", name + ".cu")
    with open(path) as f:
        text = re.sub(r"\s+", " ", f.read())
    caps = re.findall(r"cudaFuncSetAttribute\(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (.*?)\);", text)
    assert caps == [{"embed": "sizeof(GradSmem) + kMaxLocal * sizeof(int)", "dense_w4": "S::smem(kMaxX)",
                     "sample": "sizeof(Shared) + max_cells<T>() * kCell * sizeof(T)"}[name]]
