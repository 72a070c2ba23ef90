"""Calls without a workspace of the caller's: each has scratch of its own, also in graphs that are replayed at once and after
larger calls."""
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import synth

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("M", [8, 64, 300])
def test_graphs_replayed_at_once_share_no_scratch(M):
    d, f = 1024, 2048
    Wp, gamma = bl.pack_weights(synth.weights(d, d, 0.02, seed=1).cuda())
    Wr, gammas = bl.pack_weights_rowwise(synth.weights(d, d, 0.02, seed=2).cuda())
    packs = [t for n, k, s in ((f, d, 3), (f, d, 4), (d, f, 5)) for t in bl.pack_weights(synth.weights(n, k, 0.02, seed=s).cuda())]

    def step(x):
        out = []
        for _ in range(4):
            out += [bl.forward(Wp, gamma, x), bl.forward_rowwise(Wr, gammas, x), bl.forward_ex(Wp, gamma, [d], x, rmsnorm=True),
                    bl.ffn(*packs, x, residual=x)]
        return out

    xs = [synth.activations(M, d, seed=s).cuda() for s in (6, 7)]
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    graphs = []
    for x in xs:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            out = step(x)
        graphs.append((g, s, out))
    big = synth.activations(2000, d, seed=8).cuda()
    bl.ffn(*packs, big)  # more scratch than any call before
    bl.forward(Wp, gamma, big)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, out in graphs:
            with torch.cuda.stream(s):
                for o in out:
                    o.zero_()
                g.replay()
        torch.cuda.synchronize()
        for (_, _, out), ref in zip(graphs, want):
            assert all(torch.equal(o, r) for o, r in zip(out, ref))
