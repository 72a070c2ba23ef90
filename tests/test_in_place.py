"""Outputs in the place of a call's input: h += layer(h) on one tensor, with another stream at work so that some blocks of a
kernel start late."""
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import synth

gpu = pytest.mark.gpu


def check(call, x, side, load):
    want = call(x, None)
    copies = [x.clone() for _ in range(50)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            load @ load
    for h in copies:
        call(h, h)
    torch.cuda.synchronize()
    assert all(torch.equal(h, want) for h in copies)


@gpu
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 40])
@pytest.mark.parametrize("K", [512, 2560, 4096])
def test_updates_in_place(M, K):
    side, load = torch.cuda.Stream(), torch.ones((4096, 4096), dtype=torch.bfloat16, device="cuda")
    x = synth.activations(M, K, seed=K, outliers=True).cuda()
    W = synth.weights(K, K, 0.02, seed=1).cuda()
    Wp, gamma = bl.pack_weights(W)
    Wr, gammas = bl.pack_weights_rowwise(W)
    check(lambda h, out: bl.forward(Wp, gamma, h, residual=h, out=out), x, side, load)
    check(lambda h, out: bl.forward_rowwise(Wr, gammas, h, residual=h, out=out), x, side, load)
    for norm in (False, True):
        check(lambda h, out: bl.forward_ex(Wp, gamma, [K], h, rmsnorm=norm, residual=h, out=out), x, side, load)
    f = 768
    up, down = [synth.weights(f, K, 0.02, seed=s).cuda() for s in (2, 3)], synth.weights(K, f, 0.02, seed=4).cuda()
    packs = [t for w in (*up, down) for t in bl.pack_weights(w)]
    check(lambda h, out: bl.ffn(*packs, h, residual=h, out=out), x, side, load)
