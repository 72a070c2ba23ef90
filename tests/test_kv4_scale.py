"""The attention's scale over the range that it takes."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from tests.test_kv4 import OK, SHAPE, UNSUP, Batch, _call

gpu = pytest.mark.gpu


def test_scales_outside_the_range_are_refused():
    inside = OK if torch.cuda.is_available() else UNSUP
    for scale in (2.0 ** -100, 2.0 ** 100):
        if not torch.cuda.is_available():  # with a device the addresses would have to be real
            assert _call("attention", scale=scale) == inside
    for scale in (2.0 ** 100 * 1.001, 2.0 ** -100 * 0.999, 2.36e38, 3e38, 1e-45, 0.0):
        assert _call("attention", scale=scale) == SHAPE


def filled(heads, Hk, new, kmag, seed):
    b = Batch([(new, 300 + new), (new, 40 + new)], 128, heads, Hk, 64, seed=seed)
    n = 340 + 2 * new
    b.fill((b.rng.standard_normal((n, Hk, 128)) * kmag).astype(np.float32), b.rng.standard_normal((n, Hk, 128)).astype(np.float32))
    return b


@gpu
@pytest.mark.parametrize("new", [1, 4, 30])  # heads of a group x new tokens: 4 and 16 rows, and more than the decode kernel takes
@pytest.mark.parametrize("scale,qmag,kmag", [(2.0 ** 100, 2.0 ** -101, 0.2), (2.0 ** 94, 2.0 ** -95, 0.2), (2.0 ** 96, 0.5, 2.0 ** -97),
                                             (64.0, 2.0 ** 90, 2.0 ** -97), (2.0 ** 50, 2.0 ** 46, 2.0 ** -97),
                                             (2.0 ** -100, 2.0 ** 97, 1.0), (2.0 ** -100, 2.0 ** -20, 2.0 ** 116)])
def test_scales_near_the_ends(scale, qmag, kmag, new):
    """Scores of ordinary size from scales, queries and keys that are not."""
    b = filled(8, 2, new, kmag, seed=new)
    q = torch.from_numpy(b.rng.standard_normal((b.M, 8, 128)) * qmag).to(torch.bfloat16).cuda()
    assert float(q.abs().max()) * max(1.0, scale) < 2.0 ** 100
    out = bl.kv4_attention(q, *b.args(), new, scale=scale)
    assert bl.get_device_error() == 0 and not torch.isnan(out).any()
    b.check(q, out, scale=scale)
