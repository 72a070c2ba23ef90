"""8-bit layers: weights and activations that are not finite, and the one-token kernel where a block takes many tiles."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import synth
from tests.gpu_util import np_

gpu = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 5, 200])
def test_weights_that_are_not_finite_reach_their_own_row_only(M, dtype):
    N, K = 70, 1040
    W = synth.weights(N, K, 0.02, seed=1).to(dtype).cuda()
    x = synth.activations(M, K, seed=2).cuda()
    clean_q, clean_step = bl.pack_weights_int8(W)
    clean = bl.forward_int8(clean_q, clean_step, x)
    bad = {0: (5, NAN), 13: (K - 1, INF), 40: (0, -INF), 69: (1023, NAN)}
    for n, (k, v) in bad.items():
        W[n, k] = v
    W[40, 7] = NAN  # beside an infinity
    Wq, step = bl.pack_weights_int8(W)
    rows = torch.zeros(N, dtype=torch.bool, device="cuda")
    rows[list(bad)] = True
    assert (Wq[rows] == 0).all() and torch.equal(Wq[~rows], clean_q[~rows]) and torch.equal(step[~rows], clean_step[~rows])
    assert torch.isnan(step[[0, 40, 69]]).all() and torch.isinf(step[13])
    y = bl.forward_int8(Wq, step, x)
    assert torch.isnan(y[:, rows]).all() and torch.equal(y[:, ~rows], clean[:, ~rows])
