"""Batches that the attention side has to refuse or to count rightly: starts out of order, many sequences."""
import random

import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from tests.gpu_util import np_
from tests.test_kv4 import Batch

gpu = pytest.mark.gpu
BAD = 10
INT_MAX = 2 ** 31 - 1


# --------------------------------------------------------------------------- units of work, restated (CPU)
#
# The kernel for many rows lays the units of all sequences in one line and counts them in 32 bits: per key/value head and
# tile of 256 rows, four units and one per block of 128 keys. The host refuses a call unless
# (M Hq / 256 + S Hkv) (W P / 128 + 8) < 2^31, which is a bound if all sequences together have at most M rows.

def host_accepts(M, Hq, Hkv, S, room):
    return (M * Hq // 256 + S * Hkv) * (room // 128 + 8) <= INT_MAX


def sequence_units(start, end, length, M, max_q, group, hkv, room):
    """Units of one sequence by the checks on it alone; 0 where it is refused."""
    n = end - start
    if n <= 0 or start < 0 or end > M or n > max_q or length < 0 or length > room:
        return 0
    total = 0
    for t in range(-(-n * group // 256)):
        last = min(n - 1, ((t + 1) * 256 - 1) // group)
        total += 4 + max(1, -(-(length - n + last + 1) // 128))
    return total * hkv


def batch_units(q_start, kv_len, M, max_q, group, hkv, room, in_order=True):
    """All units, and none where q_start decreases (`in_order`)."""
    if in_order and any(a > b for a, b in zip(q_start, q_start[1:])):
        return 0
    one = {}
    return sum(one.setdefault(k, sequence_units(*k, M, max_q, group, hkv, room)) for k in zip(q_start, q_start[1:], kv_len))


def test_units_of_a_batch_in_order_fit_32_bits():
    rng = random.Random(0)
    for _ in range(400):
        hkv, group = rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 4, 8, 100])
        S, M, room = rng.randint(1, 60), rng.randint(1, 400), 128 * rng.randint(1, 4000)
        if not host_accepts(M, hkv * group, hkv, S, room):
            continue
        cuts = sorted(rng.choices(range(M + 1), k=S + 1))
        lens = [rng.choice([room, rng.randint(0, room)]) for _ in range(S)]
        units = batch_units(cuts, lens, M, M, group, hkv, room)
        assert units <= (M * hkv * group // 256 + S * hkv) * (room // 128 + 8) <= INT_MAX


# 0, M, 0, M, ...: every second sequence has all rows. The host's bound holds, the sum passes 2^31.
WRAP = dict(S=4096, M=4096, heads=64, hkv=8, room=1 << 18)


def test_units_of_a_decreasing_batch_would_wrap():
    w = WRAP
    assert host_accepts(w["M"], w["heads"], w["hkv"], w["S"], w["room"])
    starts, lens = [0, w["M"]] * (w["S"] // 2) + [0], [w["room"]] * w["S"]
    args = (starts, lens, w["M"], w["M"], w["heads"] // w["hkv"], w["hkv"], w["room"])
    assert batch_units(*args, in_order=False) > INT_MAX
    assert batch_units(*args) == 0


# --------------------------------------------------------------------------- GPU

@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_decreasing_starts_are_reported(rows):
    """Starts that go back, inside a group of 32 sequences and from one group to the next; nothing outside the rows is
    written, and the batch in order works afterwards."""
    S = 70
    b = Batch([(rows, rows + 5)] * S, 64, 4, 2, 16, seed=1)
    n = S * (rows + 5)
    b.fill(b.rng.standard_normal((n, 2, 64)).astype(np.float32), b.rng.standard_normal((n, 2, 64)).astype(np.float32))
    q = torch.from_numpy(b.rng.standard_normal((b.M, 4, 64))).to(torch.bfloat16).cuda()
    good = bl.kv4_attention(q, *b.args(), rows)
    assert bl.get_device_error() == 0
    for at in (1, 2, 31, 32, 33, 64, S - 1):
        starts = b.d_start.clone()
        starts[at] = int(b.starts[at + 1]) + rows  # sequence `at` now starts behind its end
        wide = torch.full((b.M + 2, 4, 64), -7.0, dtype=torch.bfloat16, device="cuda")
        bl.kv4_attention(q, b.cache, b.d_table, b.d_len, starts, 3 * rows, out=wide[1:-1])
        assert bl.get_device_error() == BAD, at
        assert (np_(wide[0].float()) == -7.0).all() and (np_(wide[-1].float()) == -7.0).all()
    assert torch.equal(bl.kv4_attention(q, *b.args(), rows), good) and bl.get_device_error() == 0


@gpu
def test_starts_whose_units_would_wrap():
    """The batch of test_units_of_a_decreasing_batch_would_wrap: reported, and the next call is right."""
    w, D, P = WRAP, 64, 256
    cache = bl.kv4_cache(1, w["hkv"], P, D, "cuda")
    table = torch.zeros((1, w["room"] // P), dtype=torch.int32, device="cuda").expand(w["S"], -1)
    lens = torch.full((w["S"],), w["room"], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, w["M"]] * (w["S"] // 2) + [0], dtype=torch.int32, device="cuda")
    q = torch.ones((w["M"], w["heads"], D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, -7.0)
    bl.kv4_attention(q, cache, table, lens, starts, w["M"], out=out)
    assert bl.get_device_error() == BAD and (out == -7.0).all()
    starts[1:] = w["M"]
    lens[:] = w["M"]
    bl.kv4_attention(q, cache, table, lens, starts, w["M"], out=out)
    assert bl.get_device_error() == 0 and (out == 0.0).all()  # the cache holds zeros
