"""The attention side at the far ends of its sizes: hundreds of appended rows, up to the most sequences a batch may have."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from tests import kv4_reference as ref
from tests import test_kv4 as small
from tests.gpu_util import np_
from tests.test_kv4 import Batch, table

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,D,H,Hk,P", [
    ([(381, 381)], 128, 20, 5, 64),                      # with the two padding rows one below and one at the change of kernels
    ([(382, 500)], 128, 20, 5, 64),
    ([(383, 383)], 64, 15, 5, 32),                       # keys' and queries' octets in one warp
    ([(200, 300), (0, 9), (1, 77), (190, 190)], 64, 3, 1, 16),   # one step of a warp holds a whole token
    ([(300, 700), (99, 99), (1, 1)], 128, 64, 8, 256),   # eight warps a token
    ([(257, 300), (150, 400)], 128, 128, 16, 128),       # and more than eight
    ([(400, 401)], 64, 8, 8, 64),
])
def test_append_of_many_rows(lens, D, H, Hk, P, interleaved):
    small.test_append_bits(lens, D, H, Hk, P, interleaved)


def lengths(S, seed, most, every):
    """S short sequences, some idle or without new tokens; every `every`-th brings up to `most` new tokens."""
    rng = np.random.default_rng(seed)
    out = []
    for s in range(S):
        n = int(rng.integers(1, most + 1)) if s % every == 0 else int(rng.choice([0, 1, 1, 1]))
        kv = int(rng.integers(0, 40))
        out.append((n, 0 if s % 11 == 5 else max(kv, n) if s % every == 0 else kv))
    return out


@gpu
@pytest.mark.parametrize("most,every", [(2, 3), (4, 5), (40, 37)])  # 4 and 16 rows of a head, and more than the decode kernel takes
@pytest.mark.parametrize("S", [161, 400, 1025, 1100, 4096])
def test_many_sequences(S, most, every):
    """Append, read-back and attention of batches with more sequences than the kernels look at in one go."""
    lens = lengths(S, S + most, most, every)
    b = Batch(lens, 64, 8, 2, 16, seed=S)
    n = sum(kv for _, kv in lens)
    b.fill(b.rng.standard_normal((n, 2, 64)).astype(np.float32), b.rng.standard_normal((n, 2, 64)).astype(np.float32))
    q, k, v = b.qkv()
    cs = table(b.max_kv, 64)
    out = torch.zeros((b.M, 8, 64), dtype=torch.bfloat16, device="cuda")
    rot = bl.kv4_append(q, k, v, cs, *b.args(), out=out)
    seq = np.repeat(np.arange(S), np.diff(b.starts))
    pos = b.d_len.cpu().numpy()[seq] - b.starts[seq + 1] + np.arange(b.M)
    live = pos >= 0
    row = np_(cs)[np.maximum(pos, 0)][:, None]
    assert np.array_equal(np_(rot.float())[live], ref.bf16_round(ref.rotate(np_(q.float()), row))[live])
    assert (np_(rot.float())[~live] == 0).all()
    kc, ks, vc, vs = ref.entry(ref.rotate(np_(k.float()), row), np_(v.float()))
    rk, rv = bl.kv4_read(*b.args(), b.M)
    assert np.array_equal(np_(rk.double())[live], ref.values(ref.pack(kc), ks)[live])
    assert np.array_equal(np_(rv.double())[live], ref.values(ref.pack(vc), vs)[live])
    o = bl.kv4_attention(rot, *b.args(), b.max_q)
    assert bl.get_device_error() == 0
    b.check(rot, o)
