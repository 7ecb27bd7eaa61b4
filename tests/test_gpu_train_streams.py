"""The attention gradient on several streams and in graphs, in both its forms:
200 rows x 4 heads are one launch, 321 and 505 rows a launch of row values in the
workspace and the main one.  Every buffer exists, and is filled, before the side
streams start, and lives until they are done."""
import pytest
import torch

import audio_video_flow_gb300 as h3
from test_gpu_train_ops import attention_backward, attention_case, check_attention, ok

pytestmark = pytest.mark.gpu

SHAPES = [(321, 4), (505, 3), (200, 4)]


class Call:
    """One call's inputs, outputs and workspace."""

    def __init__(self, S, H, seed, ws=None):
        self.S, self.H = S, H
        self.load(attention_case(S, H, seed))
        self.grads = torch.full((S, H, 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.ws = ws
        if ws is None:
            self.ws = torch.full((h3.h3_attention_backward_workspace_bytes(S, H),), 255, dtype=torch.uint8, device="cuda")

    def load(self, case):
        if not hasattr(self, "qkv"):
            self.qkv = torch.empty(self.S, self.H, 3, 128, dtype=torch.bfloat16, device="cuda")
            self.rest = [torch.empty_like(t) for t in case[3:]]
        for i in range(3):
            self.qkv[:, :, i].copy_(case[i])
        for to, t in zip(self.rest, case[3:]):
            to.copy_(t)

    def run(self, stream=None):
        q, k, v = (self.qkv[:, :, i] for i in range(3))
        dq, dk, dv = (self.grads[:, :, i] for i in range(3))
        h3.h3_attention_backward(self.S, self.H, q, k, v, q.stride(0), q.stride(1), *self.rest, dq, dk, dv,
                                 dq.stride(0), dq.stride(1), self.ws, stream)


def reference(S, H, seed):
    case = attention_case(S, H, seed)
    _, buf = attention_backward(case)
    ok()
    return case, buf


def test_calls_on_several_streams_at_once():
    calls = [Call(S, H, S) for S, H in SHAPES]
    want = [reference(S, H, S)[1] for S, H in SHAPES]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c.run(s)
    ok()
    for c, w in zip(calls, want):
        assert torch.equal(c.grads, w)


def test_a_call_follows_what_its_stream_wrote():
    """Inputs copied, the gradient and a copy of its result queued on a side
    stream without a wait in between, over and over."""
    for S, H in SHAPES:
        sets = [reference(S, H, seed) for seed in (1, 2)]
        c = Call(S, H, 1)
        kept = [torch.empty_like(c.grads) for _ in range(10)]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for i, to in enumerate(kept):
                c.load(sets[i & 1][0])
                c.run()
                to.copy_(c.grads)
        ok()
        for i, to in enumerate(kept):
            assert torch.equal(to, sets[i & 1][1]), (S, i)


@pytest.mark.parametrize("S, H", SHAPES)
def test_captured_and_replayed(S, H):
    c = Call(S, H, 1)
    sets = [reference(S, H, seed) for seed in (2, 3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for case, want in sets:
        c.load(case)
        c.grads.fill_(7.0)
        graph.replay()
        graph.replay()
        ok()
        assert torch.equal(c.grads, want)
    check_attention(sets[1][0], [c.grads[:, :, i] for i in range(3)], "replayed")


def test_graphs_that_share_a_workspace_replayed_in_order():
    """Two graphs and calls outside them with one workspace, on one stream: the
    next call waits for the one before."""
    big = max(h3.h3_attention_backward_workspace_bytes(S, H) for S, H in SHAPES)
    ws = torch.empty(big, dtype=torch.uint8, device="cuda")
    calls = [Call(S, H, S, ws) for S, H in SHAPES]
    want = [reference(S, H, S)[1] for S, H in SHAPES]
    torch.cuda.synchronize()
    graphs = []
    for c in calls[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run()
            c.run()
    for _ in range(5):
        graphs[0].replay()
        calls[2].run()
        graphs[1].replay()
        calls[0].run()
    ok()
    for c, w in zip(calls, want):
        assert torch.equal(c.grads, w)
