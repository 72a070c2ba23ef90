"""Scores of any size: rows whose softmax has to come out of scores far from zero, and scores beyond fp32's range."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from tests import kv4_reference as ref
from tests.gpu_util import np_
from tests.test_kv4 import Batch
from tests.test_kv4_scale import filled

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("new", [1, 4, 30])
def test_scores_above_fp32_make_their_rows_nan(new):
    """Finite queries and keys whose product passes fp32: NaN where the key is seen, and nowhere else."""
    b = filled(8, 2, new, 1.0, seed=3)
    k = b.rng.standard_normal((340 + 2 * new, 2, 128)).astype(np.float32)
    huge = 300 + new - (new + 1) // 2  # one of the first sequence's own tokens, in head 0
    k[huge, 0] = 2.0 ** 100
    b.fill(k, b.rng.standard_normal(k.shape).astype(np.float32))
    q = torch.from_numpy(np.abs(b.rng.standard_normal((b.M, 8, 128))) + 1).to(torch.bfloat16).cuda()
    plain = bl.kv4_attention(q, *b.args(), new)
    assert not torch.isnan(plain).any()  # 2^107: one key outweighs the others, and that is all
    q[:new] *= 2.0 ** 60
    out = np_(bl.kv4_attention(q, *b.args(), new, scale=1.0).float())
    want = np.zeros(out.shape, bool)
    want[huge - 300:new, :4] = True
    assert np.array_equal(np.isnan(out), want)


@gpu
@pytest.mark.parametrize("new", [1, 4, 30])
@pytest.mark.parametrize("exponent", [10, 20, 24, 28, 31, 33, 40, 70, 100])
def test_scores_of_any_size_have_a_softmax(exponent, new):
    """Keys so large that the best one outweighs all others: each row is that key's value. Rows whose two best keys lie closer
    than fp32 sums tell apart are left out (the error as in kv4_reference.attention). The others, at most 2570 of them, weigh
    e^-40 each at the most. The best one's weight p is whatever lies near the row's reference, not 1: it enters the product
    rounded to bf16 (2^-8) and the denominator as it is, and the result is rounded to bf16 (2^-8); fp32's own roundings, a
    few 2^-23, are in the 1%."""
    b = Batch([(new, 2500 + new), (new, 70 + new)], 128, 8, 2, 64, seed=exponent)
    n = 2570 + 2 * new
    b.fill((b.rng.standard_normal((n, 2, 128)) * 2.0 ** exponent).astype(np.float32), b.rng.standard_normal((n, 2, 128)).astype(np.float32))
    q = torch.from_numpy(b.rng.standard_normal((b.M, 8, 128))).to(torch.bfloat16).cuda()
    out = np_(bl.kv4_attention(q, *b.args(), new).double())
    qd, checked = np_(q.double()), 0
    for s, (k, ks, v) in enumerate(b.stored()):
        first = b.lens[s][1] - new
        for i in range(new):
            for h in range(8):
                m, x, kv = first + i + 1, qd[s * new + i, h], h // 4
                z = 128 ** -0.5 * (k[:m, kv] @ x)
                err = 128 ** -0.5 * 65 * 2.0 ** -23 * 23 * (ks[:m, kv].astype(np.float64) @ np.abs(x).reshape(4, 32).sum(1)).max()
                best = np.argsort(z)[-2:]
                if z[best[1]] - z[best[0]] > 40 + 2 * err:
                    have, want = out[s * new + i, h], v[best[1], kv]
                    assert (np.abs(have - want) <= 1.01 * 2.0 ** -7 * np.abs(want) + m * np.exp(-40) * np.abs(v[:m, kv]).max()).all(), (s, i, h)
                    checked += 1
    assert checked > 8 * new


@gpu
@pytest.mark.parametrize("new", [1, 4, 30])
@pytest.mark.parametrize("exponent", [24, 31, 40, 90, 118])
def test_keys_far_below_the_others_weigh_nothing(exponent, new):
    """The first keys' scores are -2^exponent and less, the others' are ordinary."""
    low, n = 700, 1300 + new
    b = Batch([(new, n)], 128, 8, 2, 64, seed=exponent + new)
    k = b.rng.standard_normal((n, 2, 128)).astype(np.float32)
    k[:low] = -(2.0 ** exponent)
    b.fill(k, b.rng.standard_normal((n, 2, 128)).astype(np.float32))
    q = torch.from_numpy(np.abs(b.rng.standard_normal((b.M, 8, 128))) + 0.5).to(torch.bfloat16).cuda()
    out = np_(bl.kv4_attention(q, *b.args(), new).double())
    (k, ks, v), = b.stored()
    for h in range(2):
        want, bound = ref.attention(np_(q.double())[:, 4 * h:4 * h + 4], k[low:, h], v[low:, h], ks[low:, h], n - new - low, 128 ** -0.5)
        assert (np.abs(out[:, 4 * h:4 * h + 4] - want) <= bound).all()
