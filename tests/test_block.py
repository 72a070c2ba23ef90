"""A decoder block on the library's calls, and the vocabulary head behind it: every stage against its own
reference on the bits that it was given, the block against the stages, prompts against single tokens."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
import oracle
from bitlinear_w1_a8_02_b200 import synth
from tests import kv4_reference as ref
from tests.gpu_util import bits, np_
from tests.test_int8 import ref_forward, ref_pack
from tests.test_kv4 import Batch, table

gpu = pytest.mark.gpu
D, HEADS, KV_HEADS, DIM, F, VOCAB = 64, 8, 2, 512, 768, 1003
ROWS = [HEADS * D, KV_HEADS * D, KV_HEADS * D]


def weights():
    shapes = [(ROWS[0], DIM), (ROWS[1], DIM), (ROWS[2], DIM), (DIM, HEADS * D), (F, DIM), (F, DIM), (DIM, F)]
    return [synth.weights(n, k, 0.02, seed=i) for i, (n, k) in enumerate(shapes)]


def stacked(W):
    parts = [oracle.pack_weights(bits(w)) for w in W]
    return np.concatenate([p[0] for p in parts]), [p[1] for p in parts]


@gpu
@pytest.mark.parametrize("lens", [[(1, 1), (1, 70), (1, 33)], [(37, 37), (1, 20), (2, 90)]])
def test_stages_and_block(lens):
    W = weights()
    block = bl.Block.pack(*[w.cuda() for w in W])
    b = Batch(lens, D, HEADS, KV_HEADS, 16, seed=1)
    n = sum(kv for _, kv in lens)
    b.fill(b.rng.standard_normal((n, KV_HEADS, D)).astype(np.float32), b.rng.standard_normal((n, KV_HEADS, D)).astype(np.float32))
    h = synth.activations(b.M, DIM, seed=3)
    cs = table(b.max_kv, D)
    before = [t.clone() for t in (b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps)]

    # Q/K/V of the normed input
    Wp, g = stacked(W[:3])
    qkv = bl.forward_ex(block.Wqkv, block.gqkv, ROWS, h.cuda(), rmsnorm=True)
    assert np.array_equal(bits(qkv), oracle.forward_ex(Wp, g, ROWS, bits(h), rmsnorm=True)["y"])
    # rotation and cache
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split(ROWS, 1))
    rot = bl.kv4_append(q, k, v, cs, *b.args())
    pos = np.concatenate([np.arange(kv - m, kv) for m, kv in lens])
    row = np_(cs)[pos][:, None]
    assert np.array_equal(np_(rot.float()), ref.bf16_round(ref.rotate(np_(q.float()), row)))
    kc, ks, vc, vs = ref.entry(ref.rotate(np_(k.float()), row), np_(v.float()))
    rk, rv = bl.kv4_read(*b.args(), b.M)
    assert np.array_equal(np_(rk.double()), ref.values(ref.pack(kc), ks)) and np.array_equal(np_(rv.double()), ref.values(ref.pack(vc), vs))
    # attention
    o = bl.kv4_attention(rot, *b.args(), b.max_q)
    b.check(rot, o)
    # output projection, FFN
    Wp, g = stacked(W[3:4])
    h1 = bl.forward_ex(block.Wo, block.go, [DIM], o.flatten(1), rmsnorm=True, residual=h.cuda())
    assert np.array_equal(bits(h1), oracle.forward_ex(Wp, g, [DIM], bits(o.flatten(1)), rmsnorm=True, residual=bits(h))["y"])
    h2 = bl.ffn(block.Wg, block.gg, block.Wu, block.gu, block.Wd, block.gd, h1, residual=h1)
    p = [oracle.pack_weights(bits(w)) for w in W[4:]]
    assert np.array_equal(bits(h2), oracle.ffn_layer(p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], bits(h1), residual=bits(h1))["y"])
    # the vocabulary head
    head = synth.weights(VOCAB, DIM, 0.02, seed=9)
    Wq, step = bl.pack_weights_int8(head.cuda())
    logits = bl.forward_int8(Wq, step, h2, rmsnorm=True, out_dtype=torch.float32)
    assert np.array_equal(np_(logits), ref_forward(*ref_pack(np_(head.float())), np_(h2.float()), rmsnorm=True)[1])

    # the block is those calls; the cache starts over
    for t, old in zip((b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps), before):
        t.copy_(old)
    got = bl.decoder_block(block, h.cuda(), HEADS, b.cache, cs, b.d_table, b.d_len, b.d_start, b.max_q)
    assert bl.get_device_error() == 0 and torch.equal(got, h2)


@gpu
def test_prompt_and_single_tokens_fill_the_same_cache():
    """A prompt in one call, and the same tokens one by one: a token's Q/K/V do not depend on the others in one block,
    so its cache entries are the same bits, and the attention outputs agree within both paths' bounds."""
    W = weights()
    block = bl.Block.pack(*[w.cuda() for w in W])
    n = 40
    cs = table(n, D)
    h = synth.activations(n, DIM, seed=5).cuda()
    one = Batch([(n, n)], D, HEADS, KV_HEADS, 16, seed=2)
    bl.decoder_block(block, h, HEADS, one.cache, cs, one.d_table, one.d_len, one.d_start, n)
    many = bl.Kv4Cache(*[torch.zeros_like(t) for t in (one.cache.k_codes, one.cache.k_steps, one.cache.v_codes, one.cache.v_steps)])
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(n):
        length = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        bl.decoder_block(block, h[i:i + 1], HEADS, many, cs, one.d_table, length, start, 1)
    a = bl.kv4_read(one.cache, one.d_table, one.d_len, one.d_start, n)
    b = bl.kv4_read(many, one.d_table, one.d_len, one.d_start, n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_block_in_a_graph_decodes_step_by_step():
    """One captured step, replayed with growing lengths and new inputs, against the same calls made directly."""
    W = weights()
    block = bl.Block.pack(*[w.cuda() for w in W])
    lens = [(1, 20), (1, 3)]
    b = Batch(lens, D, HEADS, KV_HEADS, 16, seed=4, spare_pages=6)
    n = 23
    b.fill(b.rng.standard_normal((n, KV_HEADS, D)).astype(np.float32), b.rng.standard_normal((n, KV_HEADS, D)).astype(np.float32))
    free = [p for p in range(b.pages) if p not in b.table[0, :2] and p not in b.table[1, :1]]
    tab = torch.tensor([[*b.table[0, :2], free[0]], [b.table[1, 0], free[1], free[2]]], dtype=torch.int32, device="cuda")
    cs = table(48, D)
    copies = [bl.Kv4Cache(*[t.clone() for t in (b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps)]) for _ in range(2)]
    h = synth.activations(2, DIM, seed=1).cuda()
    length = b.d_len.clone()
    warm = bl.Kv4Cache(*[t.clone() for t in (b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps)])
    bl.decoder_block(block, h, HEADS, warm, cs, tab, length, b.d_start, 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bl.decoder_block(block, h, HEADS, copies[0], cs, tab, length, b.d_start, 1)
    for step in range(12):
        h.copy_(synth.activations(2, DIM, seed=100 + step).cuda())
        g.replay()
        want = bl.decoder_block(block, h, HEADS, copies[1], cs, tab, length, b.d_start, 1)
        assert torch.equal(out, want), step
        length += 1
    assert bl.get_device_error() == 0
