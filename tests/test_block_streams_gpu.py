"""The norms and the gated feed-forward called at once on two streams, and
captured into two graphs with workspaces of the graphs' own."""
import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say
from test_gated_gpu import BF16, case as gated_case
from test_norm_gpu import F32, case as norm_case


def work(dev, seed):
    """A call of every entry point, and the tensors that it reads."""
    v = norm_case(dev, 1500, 1024, (F32, F32, BF16), gate=True, span=64, kind=1, seed=seed)
    g = gated_case(dev, 300, 512, 640, BF16, seed=seed, dh_sigma=1e-2)

    def run(stream=None):
        out, n, stats, kept = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=v["dn"].dtype, keep=True, stream=stream,
                                                   **v["how"])
        back = blr.blr_norm_backward(v["dn"], v["dout"], kept, v["f"], v["w"], stats, stream=stream, **v["how"])
        h, tape = blr.blr_gated_forward(g["x"], g["w_gate"], g["w_up"], keep=True, stream=stream)
        x = blr.blr_checkpoint_save(g["x"], stream=stream)
        more = blr.blr_gated_backward(x, g["dh"], g["w_gate"], g["w_up"], tape, stream=stream)
        again = blr.blr_gated_backward(g["x"], g["dh"], g["w_gate"], g["w_up"], stream=stream)
        return [out, n, stats, *kept, *back, h, *tape, *x, *more, *again]

    return run, [v["x"], v["f"], g["x"], g["dh"]]


@pytest.mark.gpu
def test_two_streams_at_once(dev):
    import torch
    runs = [work(dev, seed)[0] for seed in (1, 2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    say("two streams at once")
    for _ in range(3):
        got = [[], []]
        for _ in range(4):
            for i in (0, 1):
                got[i] = runs[i](streams[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(want[i], got[i]))


@pytest.mark.gpu
def test_two_graphs(dev):
    """Outputs and workspaces come from each graph's own memory; the graphs are
    replayed in turn and at once, with eager work between."""
    import torch
    both = [work(dev, seed) for seed in (3, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for run, _ in both:
            run()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [], []
    for run, _ in both:
        graphs.append(torch.cuda.CUDAGraph())
        say("capture")
        with torch.cuda.graph(graphs[-1]):
            held.append(run())
    streams = [torch.cuda.Stream() for _ in both]
    for i in range(4):
        for _, inputs in both:
            for t in inputs:
                t.copy_(torch.randn(t.shape, device=dev))
        want = [[t.clone() for t in run()] for run, _ in both]
        torch.cuda.synchronize()
        say(f"replay {i}")
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s if i & 1 else torch.cuda.current_stream()):
                graph.replay()
        torch.cuda.synchronize()
        for w, h in zip(want, held):
            assert all(torch.equal(a, b) for a, b in zip(w, h))
