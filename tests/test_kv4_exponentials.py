"""The exponentials of the kernel for many rows, a quarter of them a cubic, in the bound of its results; and its results beside
those of the decode kernel on the same cache."""
import os
import re

import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import build
from tests import kv4_reference as ref
from tests.gpu_util import np_
from tests.test_kv4 import Batch

gpu = pytest.mark.gpu
CUBIC = 7.5e-5  # largest relative error of the cubic, above the 2^-22 of the instruction


def test_the_cubic():
    """The coefficients in the source, evaluated in 64 bits over the range that is left after the exponent is taken off."""
    with open(os.path.join(build.CSRC, "kv4_tile.cu")) as f:
        body = re.search(r"float2 exp2_poly\(.*?\n}\n", f.read(), re.S).group(0)
    c = [float(x) for x in re.findall(r"make_float2\((0\.\d+)f, \1f\)", body)]
    assert len(c) == 4
    f = np.linspace(-0.5, 0.5, 100001)
    err = np.abs((((c[0] * f + c[1]) * f + c[2]) * f + c[3]) / 2.0 ** f - 1)
    assert 7e-5 < err.max() < CUBIC


def attention(q, k, v, ks, first, scale, exp_error):
    """kv4_reference.attention with the exponentials' relative error in numerator and denominator: twice it, of the weighted
    mean of |v|."""
    out, bound = ref.attention(q, k, v, ks, first, scale)
    for i in range(q.shape[0]):
        m = min(len(k), first + i + 1)
        if m > 0:
            z = scale * (q[i] @ k[:m].T)
            w = np.exp(z - z.max(-1, keepdims=True))
            bound[i] += 2 * exp_error * (w / w.sum(-1, keepdims=True)) @ np.abs(v[:m])
    return out, bound


def filled(lens, D, H, Hk, P, seed, spread):
    b = Batch(lens, D, H, Hk, P, seed=seed)
    n = sum(kv for _, kv in lens)
    b.fill((b.rng.standard_normal((n, Hk, D)) * spread).astype(np.float32), b.rng.standard_normal((n, Hk, D)).astype(np.float32) + 1)
    return b, torch.from_numpy(b.rng.standard_normal((b.M, H, D))).to(torch.bfloat16).cuda()


@gpu
@pytest.mark.parametrize("spread", [0.05, 1.0, 4.0])  # weights alike, ordinary, and a few that outweigh the others
@pytest.mark.parametrize("lens,D,H,Hk", [([(70, 70)], 128, 8, 2), ([(33, 500), (1, 2000)], 64, 8, 2), ([(257, 300), (5, 129)], 128, 5, 5)])
def test_many_rows_within_the_bound(lens, D, H, Hk, spread):
    b, q = filled(lens, D, H, Hk, 64, 1, spread)
    out, g = np_(bl.kv4_attention(q, *b.args(), b.max_q).double()), H // Hk
    for s, (k, ks, v) in enumerate(b.stored()):
        rows = slice(b.starts[s], b.starts[s + 1])
        for h in range(Hk):
            heads = slice(h * g, (h + 1) * g)
            want, bound = attention(np_(q.double())[rows, heads], k[:, h], v[:, h], ks[:, h], lens[s][1] - lens[s][0], D ** -0.5, CUBIC)
            assert (np.abs(out[rows, heads] - want) <= bound).all(), (s, h)


@gpu
@pytest.mark.parametrize("D,H,Hk,n", [(128, 8, 2, 90), (64, 20, 5, 300)])
def test_a_prompt_and_its_tokens_one_by_one_agree(D, H, Hk, n):
    """Every token of a prompt in one call, and each as a sequence of one token that ends there, on the same pages: each within
    its kernel's bound of the same values, so within both of each other."""
    b, q = filled([(n, n)], D, H, Hk, 16, 2, 1.0)
    prompt = np_(bl.kv4_attention(q, *b.args(), n).double())
    ones = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    single = np_(bl.kv4_attention(q, b.cache, b.d_table.expand(n, -1), ones[1:].contiguous(), ones, 1).double())
    (k, ks, v), = b.stored()
    g, qd = H // Hk, np_(q.double())
    for h in range(Hk):
        heads = slice(h * g, (h + 1) * g)
        args = qd[:, heads], k[:, h], v[:, h], ks[:, h], 0, D ** -0.5
        both = attention(*args, CUBIC)[1] + ref.attention(*args)[1]
        assert (np.abs(prompt[:, heads] - single[:, heads]) <= both).all(), h
