"""The workspace that a plan makes for itself, when graphs are captured before the
plan has run.  Results are compared bit for bit with those of another plan that
ran eagerly: a plan's results are deterministic."""

import pytest
import torch

import prefill_q8_mxfp4_amd as q
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt,act,widths", [("q8_0", "f32", (5, 16)), ("mxfp4", "bf16", (3, 300)),
                                            ("int8", "bf16", (20, 70))])
def test_graphs_captured_before_the_plan_has_run(fmt, act, widths):
    """An eager call between the captures and their replays, and replays in the
    other order than the captures: the counters are zero for each."""
    n, k = 512, 4096
    g = torch.Generator().manual_seed(3)
    if fmt == "int8":
        codes = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int64).to(torch.int8)
        w = q.pack_int8(codes.to(DEV), torch.rand(n, generator=g).to(DEV))
    else:
        w = torch.from_numpy(q.pack_logical(synth.gen_weights(fmt, n, k, seed=31))).to(DEV)
    dt = torch.float32 if act == "f32" else torch.bfloat16
    xs = [torch.randn(B, k, generator=g).to(dt).to(DEV) for B in widths]
    warm, cold = q.Plan(fmt, n, k, act=act), q.Plan(fmt, n, k, act=act)
    assert all(cold.workspace_bytes(B) > 0 for B in widths)
    q.init_device(torch.device(DEV))
    want = [warm.run(x, w, torch.empty(x.shape[0], n, device=DEV)) for x in xs]
    torch.cuda.synchronize()
    graphs, ys, captures = [], [], []
    for x in reversed(xs):                      # the wide one first: both take its workspace
        y, graph = torch.empty(x.shape[0], n, device=DEV), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cold.run(x, w, y)
            cold.run(x, w, y)
            captures.append(q._capture_id(torch.cuda.current_stream()))
        graphs.insert(0, graph)
        ys.insert(0, y)
    assert None not in captures and captures[0] != captures[1]
    assert q._capture_id(torch.cuda.current_stream()) is None
    for rep in range(3):
        for x, graph, y, ref in zip(xs, graphs, ys, want):
            eager = cold.run(x, w, torch.full_like(ref, float("nan")))
            torch.cuda.synchronize()
            assert torch.equal(eager, ref), (rep, x.shape[0])
            y.fill_(float("nan"))
            cold._ws_graph[1].fill_(255)        # no eager call's: each graph zeroes it for itself
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref), (rep, x.shape[0])
