"""8-bit layers: weights and activations that are not finite, and the one-token kernel where a block takes many tiles."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import synth
from tests.gpu_util import np_
from tests.test_int8 import ref_forward

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


@gpu
@pytest.mark.parametrize("N,K", [(28672, 2048), (20003, 1024), (9489, 512), (24000, 1000 // 16 * 16)])
def test_one_token_with_more_tiles_than_blocks(N, K):
    """Blocks of the one-token kernel that go round: weights loaded anew, sums in either half of the exchange."""
    Wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    step = torch.rand(N, device="cuda") + 0.5
    x = synth.activations(1, K, seed=N, outliers=True).cuda()
    res = torch.randn(1, N, device="cuda").to(torch.bfloat16)
    codes, s, _ = bl.quant_act(x)
    acc = codes.double() @ Wq.double().t()
    y = (acc.float() * step) * s.reciprocal()[:, None]
    for residual in (None, res):
        want = y if residual is None else residual.float() + y
        got, ga = bl.forward_int8(Wq, step, x, residual=residual, want_acc=True)
        assert torch.equal(ga.double(), acc) and torch.equal(got, want.to(torch.bfloat16))
        assert torch.equal(bl.forward_int8(Wq, step, x, residual=residual, out_dtype=torch.float32), want)
    acc, y = ref_forward(np_(Wq), np_(step), np_(x.float()), rmsnorm=True)
    got, ga = bl.forward_int8(Wq, step, x, rmsnorm=True, want_acc=True, out_dtype=torch.float32)
    assert np.array_equal(np_(ga), acc) and np.array_equal(np_(got), y)
    assert bl.get_device_error() == 0


@gpu
@pytest.mark.parametrize("rmsnorm", [False, True])
@pytest.mark.parametrize("N,K", [(300, 512), (300, 4000), (9000, 256)])
def test_a_row_does_not_depend_on_how_many_there_are(N, K, rmsnorm):
    """Zeros, huge and tiny values, infinities and NaN: one token alone, few and many give the same row, and the rows
    beside them are what they are without them."""
    Wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    step = torch.rand(N, device="cuda") + 0.5
    x = synth.activations(200, K, seed=3).cuda()
    plain = bl.forward_int8(Wq, step, x, rmsnorm=rmsnorm)
    special = [0.0, 1e-38, 3e38, INF, -INF, NAN]
    at = [0, 3, 17, 64, 128, 199]
    for m, v in zip(at, special):
        x[m, K // 2] = v
    x[0] = 0.0
    x[3] = 1e-38
    for M in (200, 100, 7):
        y = bl.forward_int8(Wq, step, x[:M].contiguous(), rmsnorm=rmsnorm)
        for m in range(M):
            if m in at:
                alone = bl.forward_int8(Wq, step, x[m:m + 1].contiguous(), rmsnorm=rmsnorm)
                assert torch.equal(y[m:m + 1].view(torch.int16), alone.view(torch.int16)), (M, m)
        rest = [m for m in range(M) if m not in at]
        assert torch.equal(y[rest], plain[rest])


@gpu
@pytest.mark.parametrize("M", [1, 2, 17, 100, 300])
@pytest.mark.parametrize("K", [512, 2560, 8192])
def test_update_in_place(M, K):
    """x, the residual and the output one tensor (h += layer(h)), and an output that overlaps part of x; with another stream
    at work, so that some blocks start late."""
    Wq = torch.randint(-127, 128, (K, K), dtype=torch.int8, device="cuda")
    step = torch.rand(K, device="cuda") * 1e-4
    x = synth.activations(M, K, seed=K, outliers=True).cuda()
    side, a = torch.cuda.Stream(), torch.ones((4096, 4096), dtype=torch.bfloat16, device="cuda")
    for norm in (False, True):
        want = bl.forward_int8(Wq, step, x, rmsnorm=norm, residual=x)
        copies = [x.clone() for _ in range(50)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                a @ a
        for h in copies:
            assert bl.forward_int8(Wq, step, h, rmsnorm=norm, residual=h, out=h) is h
        torch.cuda.synchronize()
        assert all(torch.equal(h, want) for h in copies)
    if M == 1:
        buf = torch.empty(2 * K, dtype=torch.bfloat16, device="cuda")
        buf[:K] = x[0]
        want = bl.forward_int8(Wq, step, x)
        assert torch.equal(bl.forward_int8(Wq, step, buf[:K].view(1, K), out=buf[K // 2:K // 2 + K].view(1, K)), want)
