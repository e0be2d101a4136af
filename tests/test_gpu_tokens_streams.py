"""The operators around the layers on streams of the caller's and beside each other: outputs that no earlier call can
have left, work that runs only behind what its own stream holds, calls in flight at the same time."""

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
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
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
