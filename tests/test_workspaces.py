"""The binding's default workspaces: one per stream and per graph captured on it,
zero before the first kernel that uses it whatever the other streams are doing.
"""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
gpu = pytest.mark.gpu


def test_one_per_stream_and_capture(monkeypatch):
    from block_sparse_attention_fa_gb300 import fa
    monkeypatch.setattr(fa, "_default_ws", {})
    monkeypatch.setattr(fa, "_ws_slot", lambda idx: torch.zeros(256, dtype=torch.uint8))
    of = fa._workspace_of
    a, b = of(0, 111, 0), of(0, 222, 0)
    in_graph, in_next = of(0, 111, 7), of(0, 111, 8)
    assert of(0, 111, 7) is in_graph
    first_in_graph = of(0, 333, 9)                            # no eager call before
    assert len({id(x.tensor) for x in (a, b, in_graph, in_next, first_in_graph, of(0, 333, 0))}) == 6
    assert of(0, 111, 0) is a and of(0, 222, 0) is b
    # a stream's check covers its graphs
    assert a.graphs == [in_graph, in_next] and b.graphs == [] and of(0, 333, 0).graphs == [first_in_graph]


class Step:
    """A training step under a window with sinks."""

    def __init__(self, seed, T, window, sinks):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda h: torch.randn(1, h, T, 128, generator=gen, device="cuda").to(torch.bfloat16)   # noqa: E731
        self.q, self.k, self.v, self.g = rand(8), rand(2), rand(2), rand(8)
        self.T, self.mask = T, dict(window=window, sinks=sinks)

    def __call__(self, **kw):
        from block_sparse_attention_fa_gb300 import fa
        bm = fa.block_mask("sink_window", 1, 1, self.T, self.T, device="cuda", **self.mask, **kw)
        o, lse = fa.fwd(self.q, self.k, self.v, bm, **kw)
        return (o, lse, *fa.bwd(self.q, self.k, self.v, o, lse, self.g, bm, **kw))


@gpu
def test_graphs_at_once():
    from block_sparse_attention_fa_gb300 import fa
    steps = [Step(1, 3000, 300, 4), Step(2, 2500, 700, 130), Step(3, 1200, 10, 0)]
    want = [s() for s in steps]
    graphs, got = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(s())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    fa.default_workspace("cuda").check()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@gpu
def test_first_call_on_another_stream():
    """The current stream is busy: nothing that it still has to do belongs to the other stream's workspace."""
    s = Step(4, 2000, 200, 4)
    want = s()
    for _ in range(3):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        for _ in range(3):
            got = s(stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        again = s(stream=side)
        torch.cuda.synchronize()
        for x, y, z in zip(want, got, again):
            assert torch.equal(x, y) and torch.equal(x, z)


@gpu
def test_a_streams_check_covers_its_graphs():
    from block_sparse_attention_fa_gb300 import fa
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    table, q = i32([0, 1], [1, 9]).reshape(2, 2), torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    args = (q, kc, kc.clone(), table, i32(20, 20), i32(0, 1, 2))
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        fa.fwd_paged(*args, max_q_len=1)
    g.replay()
    torch.cuda.synchronize()
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda", side).check()
    assert e.value.status == fa.ERR_DEVICE_CHECK and "sequence 1" in str(e.value)
    fa.default_workspace("cuda", side).check()


FRESH = r"""
import torch
from tests.test_workspaces import Step
from block_sparse_attention_fa_gb300 import fa
s = Step(5, 1500, 100, 3)
junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
del junk
graphs, got = [], []
for _ in range(2):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got.append(s())
    graphs.append(g)
for g in reversed(graphs):
    g.replay()
torch.cuda.synchronize()
want = s()
fa.default_workspace("cuda").check()
for r in got:
    assert all(torch.equal(x, y) for x, y in zip(r, want))
print("same")
"""


@gpu
def test_first_call_in_a_capture():
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
