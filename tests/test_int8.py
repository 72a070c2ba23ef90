"""8-bit linear layers: packed codes, accumulators and outputs bit for bit against the definition."""
import ctypes

import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
import oracle
from bitlinear_w1_a8_02_b200 import synth
from tests.gpu_util import bits, np_

gpu = pytest.mark.gpu
A = 0x10000
OK, NULL, SHAPE, ALIGN, DTYPE, WS, UNSUP = 0, 1, 2, 3, 4, 5, 6


def ref_pack(W):
    top = np.maximum(np.abs(W).max(1), np.float32(1e-30))
    step = (top / np.float32(127)).astype(np.float32)
    return np.clip(np.rint((W / step[:, None]).astype(np.float32)), -127, 127).astype(np.int8), step


def ref_forward(Wq, step, x, rmsnorm=False, residual=None):
    """x fp32 (bf16 values) -> (acc int64, y fp32), each step of the definition one fp32 operation."""
    if rmsnorm:
        mean = (x.astype(np.float64) ** 2).sum(1) / x.shape[1]
        r = (np.float32(1) / np.sqrt((mean.astype(np.float32) + np.float32(1e-5)).astype(np.float32))).astype(np.float32)
        x = (x * r[:, None]).astype(np.float32)
    s = (np.float32(127) / np.maximum(np.abs(x).max(1), np.float32(1e-5))).astype(np.float32)
    q = np.clip(np.rint((x * s[:, None]).astype(np.float32)), -128, 127)
    acc = (q.astype(np.float64) @ Wq.astype(np.float64).T).astype(np.int64)  # below 2^53: exact
    y = ((acc.astype(np.float32) * step[None]).astype(np.float32) * (np.float32(1) / s)[:, None]).astype(np.float32)
    if residual is not None:
        y = (residual + y).astype(np.float32)
    return acc, y


def test_refusals():
    L = bl.lib()
    P = ctypes.c_void_p
    pk = L.bitlinear_pack_weights_int8
    assert pk(P(A), 7, 8, 16, P(A), P(A), None) == DTYPE
    for n, k in ((0, 16), (8, 12), (8, 20), (8, 0), (1 << 25, 16), (8, 131088)):
        assert pk(P(A), 0, n, k, P(A), P(A), None) == SHAPE, (n, k)
    assert pk(None, 0, 8, 16, P(A), P(A), None) == NULL
    assert pk(P(A), 0, 8, 16, None, P(A), None) == NULL
    assert pk(P(A + 8), 0, 8, 16, P(A), P(A), None) == ALIGN
    assert pk(P(A), 0, 8, 16, P(A + 4), P(A), None) == ALIGN
    need = L.bitlinear_workspace_bytes(bl.BL_OP_FORWARD_INT8, 2, 8, 32)

    def fw(**kw):
        a = dict(Wq=A, ws_=A, N=8, K=32, x=A, M=2, rms=0, res=None, y=A, ydt=0, acc=None, ws=A, wsb=need)
        a.update(kw)
        return L.bitlinear_forward_int8(a["Wq"], a["ws_"], a["N"], a["K"], a["x"], a["M"], a["rms"], a["res"], a["y"], a["ydt"],
                                        a["acc"], a["ws"], a["wsb"], None)

    assert fw(M=0) == OK and fw(N=0) == OK
    for kw, want in ((dict(ydt=3), DTYPE), (dict(K=24), SHAPE), (dict(K=0), SHAPE), (dict(K=131088), SHAPE), (dict(M=-1), SHAPE),
                     (dict(M=65536), SHAPE), (dict(N=-1), SHAPE), (dict(rms=2), SHAPE), (dict(Wq=None), NULL), (dict(x=None), NULL),
                     (dict(y=None), NULL), (dict(ws_=None), NULL), (dict(Wq=A + 8), ALIGN), (dict(x=A + 2), ALIGN),
                     (dict(y=A + 2, ydt=1), ALIGN), (dict(y=A + 1), ALIGN), (dict(acc=A + 2), ALIGN), (dict(res=A + 1), ALIGN),
                     (dict(ws=None), NULL), (dict(ws=A + 16), ALIGN), (dict(wsb=need - 1), WS)):
        assert fw(**kw) == want, kw
    if not torch.cuda.is_available():
        assert fw() == UNSUP


def test_reference_by_hand():
    W = np.array([[127, -1, 0, 63.4], [0, 0, 0, 0]], np.float32) / 2
    q, s = ref_pack(W)
    assert q.tolist() == [[127, -1, 0, 63], [0, 0, 0, 0]] and s[0] == 0.5
    acc, y = ref_forward(q, s, np.array([[1.0, 2.0, 0.0, -127.0]], np.float32))
    assert acc.tolist() == [[127 - 2 - 63 * 127, 0]] and y[0, 0] == acc[0, 0] * 0.5


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (130, 2560), (33, 6912)])
def test_pack(N, K, dtype):
    W = synth.weights(N, K, 0.02, seed=N, dtype=dtype)
    W[0] = 0
    W[N // 2, K - 1] = 3.0
    Wq, step = bl.pack_weights_int8(W.cuda())
    rq, rs = ref_pack(np_(W.float()))
    assert np.array_equal(np_(Wq), rq) and np.array_equal(np_(step), rs)


SHAPES = [(1, 16), (17, 48), (257, 80), (640, 2560), (2560, 2560), (1000, 6912), (19001, 256), (31, 28672), (5000, 4000)]


@gpu
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 64, 128, 129, 300])
@pytest.mark.parametrize("N,K", SHAPES)
def test_forward(M, N, K):
    W = synth.weights(N, K, 0.02, seed=3)
    Wq, step = bl.pack_weights_int8(W.cuda())
    rq, rs = ref_pack(np_(W.float()))
    x = synth.activations(M, K, seed=M, outliers=True)
    res = synth.activations(M, N, seed=5, outliers=False)
    acc, y = ref_forward(rq, rs, np_(x.float()))
    got, ga = bl.forward_int8(Wq, step, x.cuda(), want_acc=True)
    assert np.array_equal(np_(ga), acc)
    assert np.array_equal(bits(got), oracle.f32_to_bf16(y))
    got = bl.forward_int8(Wq, step, x.cuda(), out_dtype=torch.float32)
    assert np.array_equal(np_(got), y)
    acc, y = ref_forward(rq, rs, np_(x.float()), rmsnorm=True, residual=np_(res.float()))
    got, ga = bl.forward_int8(Wq, step, x.cuda(), rmsnorm=True, residual=res.cuda(), want_acc=True)
    assert np.array_equal(np_(ga), acc) and np.array_equal(bits(got), oracle.f32_to_bf16(y))
    assert bl.get_device_error() == 0


@gpu
@pytest.mark.parametrize("N", [40001, 40004, 40008])
@pytest.mark.parametrize("M", [1, 2, 16, 40, 64, 65, 100, 128, 150])
def test_many_rows(M, N):
    """More tiles of weights than the device holds at once; rows of every alignment, each kind of output."""
    K = 208
    Wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    step = torch.rand(N, device="cuda")
    x = synth.activations(M, K, seed=M, outliers=True).cuda()
    res = torch.randn(M, N, device="cuda").to(torch.bfloat16)
    codes, s, _ = bl.quant_act(x)
    acc = codes.double() @ Wq.double().t()
    y = (acc.float() * step) * s.reciprocal()[:, None]
    for residual in (None, res):
        want = y if residual is None else residual.float() + y
        got, ga = bl.forward_int8(Wq, step, x, residual=residual, want_acc=True)
        assert torch.equal(ga.double(), acc) and torch.equal(got, want.to(torch.bfloat16))
        assert torch.equal(bl.forward_int8(Wq, step, x, residual=residual), want.to(torch.bfloat16))
        assert torch.equal(bl.forward_int8(Wq, step, x, residual=residual, out_dtype=torch.float32), want)
    assert bl.get_device_error() == 0


@gpu
@pytest.mark.parametrize("M", [1, 2])
@pytest.mark.parametrize("K", [4080, 4096, 4112, 32752, 32768, 40928, 40944, 131072])
def test_lengths_around_the_kernel_choice(M, K):
    Wq = torch.randint(-127, 128, (35, K), dtype=torch.int8, device="cuda")
    x = synth.activations(M, K, seed=1).cuda()
    _, acc = bl.forward_int8(Wq, torch.ones(35, device="cuda"), x, want_acc=True)
    codes, _, _ = bl.quant_act(x)
    assert torch.equal(acc.double(), codes.double() @ Wq.double().t())


@gpu
@pytest.mark.parametrize("M", [3, 200])
def test_extreme_codes(M):
    """Every code at its largest magnitude over the longest K of the checks: accumulators near 2^31."""
    K, N = 131072, 40
    Wq = torch.full((N, K), -127, dtype=torch.int8, device="cuda")
    Wq[1::2] = 127
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    y, acc = bl.forward_int8(Wq, torch.ones(N, device="cuda"), x, want_acc=True)
    want = torch.where(torch.arange(N, device="cuda") % 2 == 1, 127 * 127 * K, -127 * 127 * K).to(torch.int32)
    assert torch.equal(acc, want.expand(M, N))
    assert torch.equal(y, (want.float() * (1.0 / 127.0)).to(torch.bfloat16).expand(M, N))


@gpu
@pytest.mark.parametrize("M", [5, 70])
def test_slices_streams_and_graph(M):
    """Weights, steps and outputs that start inside larger tensors; another stream; a replayed graph."""
    K, N = 512, 328
    W = synth.weights(N + 3, K, 0.02, seed=1).cuda()
    Wq, step = bl.pack_weights_int8(W)
    x = synth.activations(M, K, seed=2).cuda()
    whole = bl.forward_int8(Wq, step, x)
    buf = torch.empty(M * N + 1, dtype=torch.bfloat16, device="cuda")
    out = buf[1:].view(M, N)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bl.forward_int8(Wq[3:], step[3:], x, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, whole[:, 3:])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = bl.forward_int8(Wq, step, x)
    x.copy_(synth.activations(M, K, seed=8).cuda())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, bl.forward_int8(Wq, step, x)) and not torch.equal(y, whole)
    with pytest.raises(ValueError):
        bl.forward_int8(Wq, step[:5], x)
    with pytest.raises(ValueError):
        bl.forward_int8(Wq, step, x, out=out)
    with pytest.raises(ValueError):
        bl.forward_int8(Wq, step, x, out_dtype=torch.float16)
    assert bl.forward_int8(Wq, step, x[:0]).shape == (0, N + 3)
