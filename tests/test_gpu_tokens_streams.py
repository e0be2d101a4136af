"""The operators around the layers on streams of the caller's and beside each other: outputs that no earlier call can
have left, work that runs only behind what its own stream holds, calls in flight at the same time."""

import threading

import numpy as np
import pytest
import torch

from gpu_util import dev
from test_gpu_tokens import BF, F32, _ints, _product, _tensor, txl  # noqa: F401

pytestmark = pytest.mark.gpu


class Step:
    """Ids to rows, a product, the next ids, the gradient of the first, with inputs and outputs of its own."""

    def __init__(self, txl, seed, V=500, d=256, T=64):  # noqa: F811
        rng = np.random.default_rng(seed)
        self.txl, self.table = txl, _tensor(rng.standard_normal((V, d)), BF)
        _, self.codes, self.scales = _product(rng, T, d, V // 8 * 8, 64)
        self.tokens, self.u = _ints(rng.integers(-1, V, T)), _tensor(rng.random(T), F32)
        self.k, self.p = _ints(np.full(T, 20)), torch.full((T,), 0.9, device=dev())
        self.h, self.logits = torch.empty(T, d, device=dev(), dtype=BF), torch.empty(T, self.codes.shape[0], device=dev())
        self.out, self.grad = torch.empty(T, device=dev(), dtype=torch.int32), torch.empty(V, d, device=dev())
        self.outputs = (self.h, self.logits, self.out, self.grad)

    def calls(self, stream=None):
        """Each reads what the one before it wrote."""
        self.txl.txl_embed_forward(self.tokens, self.table, self.h, scale=0.5, stream=stream)
        self.txl.txl_dense_w4(self.h, self.codes, self.scales, self.logits, stream=stream)
        self.txl.txl_sample(self.logits, self.u, self.out, top_k=self.k, top_p=self.p, stream=stream)
        self.txl.txl_embed_backward(self.out, self.h, self.grad, scale=0.5, stream=stream)

    def spoil(self):
        """No output is left that a call would have to write."""
        for t in self.outputs:
            t.fill_(-7 if t.dtype == torch.int32 else float("nan"))

    def want(self):
        """The outputs, alone, on the default stream."""
        self.spoil()
        torch.cuda.synchronize()
        self.calls()
        torch.cuda.synchronize()
        assert not self.h.isnan().any() and not self.logits.isnan().any() and not self.grad.isnan().any() and (self.out >= 0).all()
        return [t.clone() for t in self.outputs]

    def differ(self, want):
        """How many outputs differ, on the device."""
        return sum((a != b).sum() for a, b in zip(self.outputs, want))


@pytest.mark.parametrize("how", ["stream", "handle", "current"])
def test_calls_run_on_the_given_stream(txl, how):  # noqa: F811
    """The ids come only behind a long wait on the side stream: a call that ran elsewhere would take what was there."""
    step = Step(txl, 20)
    wrong = _ints(np.full(64, 3))
    right = step.tokens.clone()
    want = step.want()
    side = torch.cuda.Stream()
    step.tokens.copy_(wrong)
    step.spoil()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # a fifth of a second or so
        step.tokens.copy_(right)
        if how == "current":
            step.calls()
    if how == "stream":
        step.calls(stream=side)
    elif how == "handle":
        step.calls(stream=side.cuda_stream)
    assert not side.query()  # the calls wait for nothing
    side.synchronize()
    assert int(step.differ(want)) == 0


def test_calls_on_two_streams_at_once(txl):  # noqa: F811
    """Two steps, each on a stream of its own, nothing between them; each round's outputs are looked at on its stream and
    spoilt before the next."""
    steps = [Step(txl, 21), Step(txl, 22)]
    wants = [s.want() for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.default_stream()]
    bad = []
    torch.cuda.synchronize()
    for _ in range(50):
        for step, want, stream in zip(steps, wants, streams):
            with torch.cuda.stream(stream):
                step.spoil()
                step.calls()
                bad.append(step.differ(want))
    torch.cuda.synchronize()
    assert [int(b) for b in bad] == [0] * len(bad)


def test_replays_of_a_graph_beside_calls(txl):  # noqa: F811
    """A captured step, replayed on one stream while its like runs call by call on another; every replay's outputs."""
    steps = [Step(txl, 23), Step(txl, 24)]
    wants = [s.want() for s in steps]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps[0].calls()
    bad = []
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(side):
            steps[0].spoil()
            graph.replay()
            bad.append(steps[0].differ(wants[0]))
        steps[1].spoil()
        steps[1].calls()
        bad.append(steps[1].differ(wants[1]))
    torch.cuda.synchronize()
    assert [int(b) for b in bad] == [0] * len(bad)


def test_every_call_of_many_threads(txl):  # noqa: F811
    """Calls of other sizes from several threads at once, each with outputs of its own that hold nothing before it: not
    one that returns without having written."""
    lib, ptr, rounds, slots = txl.lib, torch.Tensor.data_ptr, 12, 25
    rng = np.random.default_rng(25)
    jobs = []
    for V, k, n in ((64, 128, 64), (30000, 4096, 256), (2000, 512, 64), (20000, 2048, 128)):
        x, codes, scales = _product(rng, 4, k, n, 32)
        job = dict(V=V, k=k, n=n, x=x, codes=codes, scales=scales, z=_tensor(rng.standard_normal((2, V)), F32),
                   u=torch.full((2,), 0.5, device=dev()), tokens=_ints(rng.integers(0, V, 100)), dout=_tensor(rng.standard_normal((100, 16)), F32),
                   out=torch.empty(slots, 2, device=dev(), dtype=torch.int32), y=torch.empty(slots, 4, n, device=dev(), dtype=BF),
                   grad=torch.empty(slots, V, 16, device=dev()), stream=torch.cuda.Stream())
        alone = [torch.full_like(job[t][0], -7) for t in ("out", "y", "grad")]
        txl.txl_sample(job["z"], job["u"], alone[0])
        txl.txl_dense_w4(x, codes, scales, alone[1])
        txl.txl_embed_backward(job["tokens"], job["dout"], alone[2])
        jobs.append((job, alone))
    torch.cuda.synchronize()
    failed, differ, start = [], [], threading.Barrier(len(jobs))

    def run(job, alone):
        s = job["stream"].cuda_stream
        with torch.cuda.stream(job["stream"]):
            for _ in range(rounds):
                for t in ("out", "y", "grad"):
                    job[t].fill_(-7)
                start.wait()
                for i in range(slots):
                    failed.append(lib.txl_sample(ptr(job["z"]), job["V"], 2, job["V"], ptr(job["u"]), None, None, None, None, ptr(job["out"][i]), None, 0, s))
                    failed.append(lib.txl_dense_w4(ptr(job["x"]), ptr(job["codes"]), ptr(job["scales"]), ptr(job["y"][i]), 4, job["n"], job["k"], 32, None, 0, 1, s))
                    failed.append(lib.txl_embed_backward(ptr(job["tokens"]), ptr(job["dout"]), ptr(job["grad"][i]), 100, job["V"], 16, 1.0, 0, 0, s))
                differ.append(sum((job[t] != w).sum() for t, w in zip(("out", "y", "grad"), alone)))

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(failed) == 3 * slots * rounds * len(jobs) and not any(failed), (sum(f != 0 for f in failed), len(failed))
    assert [int(d) for d in differ] == [0] * rounds * len(jobs)
