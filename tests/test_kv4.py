"""The 4-bit paged cache and the attention over it: codes, steps and rotated queries bit for bit
against the definition, attention against 64 bits, refusals on the host."""
import struct

import numpy as np
import pytest
import torch

import bitlinear_w1_a8_02_b200 as bl
from bitlinear_w1_a8_02_b200 import binding
from tests import kv4_reference as ref
from tests.gpu_util import np_

gpu = pytest.mark.gpu
THETA = 500000.0


# --------------------------------------------------------------------------- the reference itself (CPU)

def test_reference_steps_and_codes():
    # absmax 7 * 1.03125: the step between 1 and 1.0625 rounds to the even 1; 7.5 and more never appears
    x = np.zeros((1, 32), np.float32)
    x[0, :3] = [7.0, -3.5, 0.4]
    c, s = ref.quantise(x)
    assert s[0, 0] == 1.0 and c[0, :4].tolist() == [7, -4, 0, 0]
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((4000, 64)) * 10.0 ** rng.uniform(-20, 20, (4000, 1))).astype(np.float32)
    c, s = ref.quantise(x)
    assert np.abs(c).max() == 7
    err = np.abs(c * np.repeat(s, 32, -1).astype(np.float64) - x)
    assert (err <= 0.5 * np.repeat(s, 32, -1) * (1 + 2.0 ** -23)).all()  # no value is clipped
    v = c * np.repeat(s, 32, -1).astype(np.float64)
    assert np.array_equal(ref.bf16_round(v.astype(np.float32)), v)  # bf16 numbers exactly
    for k in (16.0, 24.0):
        assert np.array_equal(ref.bf16_round((k * s).astype(np.float32)), (k * s).astype(np.float32))
    assert np.array_equal(ref.unpack(ref.pack(c)), c)


def test_reference_attention_is_a_plain_mean_for_equal_scores():
    v = np.arange(8.0).reshape(4, 2).repeat(16, 1)
    out, bound = ref.attention(np.zeros((2, 1, 32)), np.ones((4, 32)), v, np.ones((4, 1)), 2, 1.0)
    assert np.allclose(out[0, 0], v[:3].mean(0)) and np.allclose(out[1, 0], v.mean(0)) and (bound > 0).all()


# --------------------------------------------------------------------------- refusals on the host (CPU)

A = 0x10000
OK, NULL, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 5, 6


def _call(fn, **kw):
    c = dict(kc=A, ks=A, vc=A, vs=A, num_pages=10, page_size=64, kv_heads=2, head_dim=128)
    b = dict(q_start=A, kv_len=A, page_table=A, table_stride=4, S=3, W=4)
    a = dict(q=A, q_stride=1024, k=A, k_stride=256, v=A, v_stride=256, M=3, Hq=8, cs=A, max_pos=100, il=0, out=A,
             o_stride=1024, max_q=1, scale=0.1, ws=A, wsb=binding.workspace_bytes(bl.BL_OP_KV4_ATTENTION, 1, 4, 128),
             cache=True, batch=True)
    for k, v in kw.items():
        next(d for d in (c, b, a) if k in d)[k] = v
    C = struct.pack("=QQQQqiiii", *[x or 0 for x in c.values()], 0) if a["cache"] else None  # bl_kv4_cache
    B = struct.pack("=QQQqii", *[x or 0 for x in b.values()]) if a["batch"] else None        # bl_kv4_batch
    L = bl.lib()
    if fn == "append":
        return L.bitlinear_kv4_append(a["q"], a["q_stride"], a["k"], a["k_stride"], a["v"], a["v_stride"], a["M"], a["Hq"],
                                      a["cs"], a["max_pos"], a["il"], C, B, a["out"], a["o_stride"], None)
    if fn == "read":
        return L.bitlinear_kv4_read(C, B, a["M"], a["k"], a["v"], None)
    return L.bitlinear_kv4_attention(a["q"], a["q_stride"], a["M"], a["Hq"], a["max_q"], a["scale"], C, B, a["out"],
                                     a["o_stride"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", ["append", "read", "attention"])
def test_refusals_cache_and_batch(fn):
    assert _call(fn, M=0) == OK
    for kw, want in ((dict(cache=False), NULL), (dict(batch=False), NULL), (dict(kc=None), NULL), (dict(vs=None), NULL),
                     (dict(q_start=None), NULL), (dict(page_table=None), NULL), (dict(kc=A + 8), ALIGN),
                     (dict(ks=A + 2), ALIGN), (dict(kv_len=A + 2), ALIGN), (dict(head_dim=96), SHAPE),
                     (dict(head_dim=0), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=8), SHAPE),
                     (dict(page_size=512), SHAPE), (dict(page_size=0), SHAPE), (dict(num_pages=0), SHAPE),
                     (dict(num_pages=1 << 31), SHAPE), (dict(kv_heads=0), SHAPE), (dict(S=0), SHAPE), (dict(S=4097), SHAPE),
                     (dict(W=0), SHAPE), (dict(W=1 << 24), SHAPE), (dict(table_stride=-1), SHAPE), (dict(M=-1), SHAPE),
                     (dict(M=65536), SHAPE), (dict(S=4096, W=1 << 18), SHAPE)):
        assert _call(fn, **kw) == want, kw


def test_refusals_rows():
    for fn in ("append", "attention"):
        for kw, want in ((dict(q=None), NULL), (dict(out=None), NULL), (dict(q=A + 8), ALIGN), (dict(q_stride=1028), ALIGN),
                         (dict(q_stride=1016), SHAPE), (dict(o_stride=512), SHAPE), (dict(Hq=7), SHAPE), (dict(Hq=0), SHAPE),
                         (dict(Hq=2048), SHAPE)):
            assert _call(fn, **kw) == want, (fn, kw)
    for kw, want in ((dict(k=None), NULL), (dict(v=A + 2), ALIGN), (dict(k_stride=128), SHAPE), (dict(cs=None), NULL),
                     (dict(cs=A + 4), ALIGN), (dict(max_pos=0), SHAPE), (dict(il=2), SHAPE), (dict(o_stride=2048), SHAPE)):
        assert _call("append", **kw) == want, kw
    for kw, want in ((dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE),
                     (dict(scale=float("inf")), SHAPE), (dict(max_q=-1), SHAPE), (dict(M=65535, Hq=1024, q_stride=131072, o_stride=131072, W=1 << 18), SHAPE), (dict(ws=None), NULL), (dict(ws=A + 16), ALIGN),
                     (dict(wsb=1000), WS), (dict(max_q=3, Hq=16, q_stride=2048, o_stride=2048, wsb=binding.workspace_bytes(bl.BL_OP_KV4_ATTENTION, 1, 4, 128)), WS)):
        assert _call("attention", **kw) == want, kw


def test_valid_calls_without_a_device_are_unsupported():
    if torch.cuda.is_available():
        pytest.skip("a device is here: the addresses are not real")
    for fn in ("append", "read", "attention"):
        assert _call(fn) == UNSUP


def test_binding_refuses_cpu_tensors():
    codes, steps = torch.zeros((2, 1, 16, 32), dtype=torch.uint8), torch.zeros((2, 1, 16, 2), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bl.Kv4Cache(codes, steps, codes, steps)


# --------------------------------------------------------------------------- GPU

class Batch:
    """A batch with its cache on the GPU: ragged lengths, shuffled pages, unused memory full of NaN steps."""

    def __init__(self, lens, D, heads, kv_heads, page, seed=0, spare_rows=0, spare_pages=3, fused=True):
        self.lens, self.D, self.H, self.Hk, self.P = lens, D, heads, kv_heads, page
        rng = self.rng = np.random.default_rng(seed)
        self.starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.M = int(self.starts[-1]) + spare_rows
        used = [-(-kv // page) for _, kv in lens]
        width = max(max(used), 1)
        self.pages = sum(used) + spare_pages
        order = rng.permutation(self.pages)
        # entries past a sequence's last page are out of range: they must not be read
        self.table = np.full((len(lens), width + 1), 1 << 30, np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = order[at:at + n]
            at += n
        dev = "cuda"
        self.d_table = torch.from_numpy(self.table).to(dev)[:, :width]
        self.d_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev)
        self.d_start = torch.from_numpy(self.starts).to(dev)
        codes = lambda: torch.from_numpy(rng.integers(0, 256, (self.pages, kv_heads, page, D // 2), dtype=np.uint8)).to(dev)  # noqa: E731
        steps = lambda: torch.full((self.pages, kv_heads, page, D // 32), float("nan"), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.cache = bl.Kv4Cache(codes(), steps(), codes(), steps())
        self.max_q = max(q for q, _ in lens)
        self.max_kv = max(max(kv for _, kv in lens), 1)

    def args(self):
        return self.cache, self.d_table, self.d_len, self.d_start

    def qkv(self, scale=1.0):
        """Rows of a stacked projection with a few loud channels, and its three column blocks."""
        width = (self.H + 2 * self.Hk) * self.D
        x = self.rng.standard_normal((self.M, width)).astype(np.float32) * scale
        x[:, self.rng.integers(0, width, width // 100 + 1)] *= 20
        t = torch.from_numpy(x).to(torch.bfloat16).cuda()
        return [b.unflatten(1, (-1, self.D)) for b in t.split([self.H * self.D, self.Hk * self.D, self.Hk * self.D], 1)]

    def fill(self, k, v):
        """Store fp32 keys and values [sum kv, Hk, D] of all tokens in the cache, through the reference."""
        kc, ks, vc, vs = ref.entry(k, v)
        at = 0
        new = (ref.pack(kc), ks.view(np.uint32) >> 16, ref.pack(vc), vs.view(np.uint32) >> 16)
        host = [np_(t.view(torch.int16) if t.dtype == torch.bfloat16 else t) for t in (self.cache.k_codes, self.cache.k_steps, self.cache.v_codes, self.cache.v_steps)]
        for s, (_, kv) in enumerate(self.lens):
            for p in range(kv):
                page, off = self.table[s, p // self.P], p % self.P
                for arr, val in zip(host, new):
                    arr[page, :, off] = val[at].astype(np.uint16).view(np.int16) if arr.dtype == np.int16 else val[at]
                at += 1
        for t, h in zip((self.cache.k_codes, self.cache.k_steps, self.cache.v_codes, self.cache.v_steps), host):
            t.copy_(torch.from_numpy(h).view(t.dtype).cuda())

    def stored(self):
        """Per sequence: (key values, key steps, value values) fp64 [kv, Hk, ...] as the cache holds them."""
        a = [np_(t) if t.dtype == torch.uint8 else np_(t.float()) for t in (self.cache.k_codes, self.cache.k_steps, self.cache.v_codes, self.cache.v_steps)]
        for s, (_, kv) in enumerate(self.lens):
            page = self.table[s, np.arange(kv) // self.P]
            off = np.arange(kv) % self.P
            kc, ks, vc, vs = (x[page, :, off] for x in a)
            yield ref.values(kc, ks), ks, ref.values(vc, vs)

    def check(self, q, out, scale=None):
        q, got = np_(q.float()).astype(np.float64), np_(out.float()).astype(np.float64)
        g = self.H // self.Hk
        scale = self.D ** -0.5 if scale is None else scale
        for s, (k, ks, v) in enumerate(self.stored()):
            n, kv = self.lens[s]
            a, b = self.starts[s], self.starts[s + 1]
            for h in range(self.Hk):
                want, bound = ref.attention(q[a:b, h * g:(h + 1) * g], k[:, h], v[:, h], ks[:, h], kv - n, scale)
                have = got[a:b, h * g:(h + 1) * g]
                assert np.array_equal(np.isnan(want), np.isnan(have)), (s, h)
                bad = np.argwhere(~(np.abs(have - want) <= bound) & ~np.isnan(want))
                assert bad.size == 0, (s, h, bad[:3].tolist(), have[tuple(bad[0])], want[tuple(bad[0])], bound[tuple(bad[0])])


def table(max_pos, D):
    a = np.arange(max_pos)[:, None] * THETA ** (-np.arange(0, D, 2) / D)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


APPEND = [
    # lens (new, cached), D, heads, kv heads, page
    ([(1, 1)], 128, 20, 5, 64),
    ([(1, 17), (1, 1), (1, 64), (1, 65)], 128, 8, 8, 16),
    ([(5, 5), (0, 9), (3, 40), (1, 300)], 64, 15, 5, 32),
    ([(130, 130), (7, 1000), (33, 64)], 128, 20, 5, 128),
    ([(2, 2), (9, 260)], 64, 16, 1, 256),
    ([(1, 5)] * 70, 64, 4, 4, 16),
]


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,D,H,Hk,P", APPEND)
def test_append_bits(lens, D, H, Hk, P, interleaved):
    b = Batch(lens, D, H, Hk, P, spare_rows=2)
    q, k, v = b.qkv()
    k[0, 0, :32] = 0.0            # a group of zeros
    v[0, Hk - 1, 32:64] = 1e-38   # and one below the smallest step
    cs = table(b.max_kv, D)
    before = [t.clone() for t in (b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps)]
    out = torch.full((b.M, H, D), -7.0, dtype=torch.bfloat16, device="cuda")
    got = bl.kv4_append(q, k, v, cs, *b.args(), interleaved=interleaved, out=out)
    assert got is out and bl.get_device_error() == 0
    qn, kn, vn, csn = np_(q.float()), np_(k.float()), np_(v.float()), np_(cs)
    written = np.zeros((b.pages, P), bool)
    arrays = (b.cache.k_codes, b.cache.k_steps, b.cache.v_codes, b.cache.v_steps)
    host = [np_(t) if t.dtype == torch.uint8 else np_(t.view(torch.int16)) for t in arrays]
    for s, (n, kv) in enumerate(lens):
        for i in range(n):
            m, p = b.starts[s] + i, kv - n + i
            row = csn[p][None]
            want_q = ref.bf16_round(ref.rotate(qn[m], row, interleaved))
            assert np.array_equal(np_(out[m].float()), want_q), (s, i)
            kc, ks, vc, vs = ref.entry(ref.rotate(kn[m], row, interleaved), vn[m])
            page, off = b.table[s, p // P], p % P
            written[page, off] = True
            for have, want in zip(host, (ref.pack(kc), ks, ref.pack(vc), vs)):
                if want.dtype != np.uint8:
                    want = (want.view(np.uint32) >> 16).astype(np.uint16).view(np.int16)
                assert np.array_equal(have[page, :, off], want), (s, i)
    assert (np_(out[int(b.starts[-1]):].float()) == -7.0).all()  # padding rows
    for t, old in zip(host, before):
        old = np_(old) if old.dtype == torch.uint8 else np_(old.view(torch.int16))
        assert np.array_equal(t.transpose(0, 2, 1, 3)[~written], old.transpose(0, 2, 1, 3)[~written])
    # read back
    rk, rv = bl.kv4_read(*b.args(), b.M)
    for s, (kk, _, vv) in enumerate(b.stored()):
        n, kv = lens[s]
        a, e = b.starts[s], b.starts[s + 1]
        assert np.array_equal(np_(rk[a:e].double()), kk[kv - n:]) and np.array_equal(np_(rv[a:e].double()), vv[kv - n:])


@gpu
def test_append_ties_and_neighbours():
    """Values on, just above and just below every half code, for every significand of the step, at several exponents."""
    D, Hk, n = 128, 16, 64
    b = Batch([(n, n)], D, Hk, Hk, 64)
    k = np.zeros((n, Hk, D), np.float32)
    for t in range(n):
        for h in range(Hk):
            step = np.float32((16 + h) * 2.0 ** (t % 32 - 20))
            k[t, h, 0::32] = 7 * step  # the largest of each group: the step comes out as `step`
            half = (np.arange(-6.5, 7.0, 1.0) * step).astype(np.float32)
            for g, x in enumerate((half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf)), half)):
                k[t, h, 32 * g + 1:32 * g + 15] = x
    q, _, _ = b.qkv()
    # bf16 inputs: half codes fit; their fp32 neighbours come from a rotation by an angle whose cosine is 1 +- 2^-23
    cs = torch.zeros((n, D), device="cuda")
    cs[:, :D // 2] = 1.0
    for c in (1.0, float(np.nextafter(np.float32(1), np.float32(2))), float(np.nextafter(np.float32(1), np.float32(0)))):
        cs[:, 1:15] = c
        cs[:, 33:47] = c
        kk = torch.from_numpy(k).to(torch.bfloat16).cuda()
        bl.kv4_append(q, kk, kk, cs, *b.args())
        kc, ks, vc, vs = ref.entry(ref.rotate(np_(kk.float()), np_(cs)[:, None]), np_(kk.float()))
        page = b.table[0, np.arange(n) // 64]
        for have, want in ((b.cache.k_codes, ref.pack(kc)), (b.cache.v_codes, ref.pack(vc))):
            assert np.array_equal(np_(have)[page, :, np.arange(n) % 64], want)
        for have, want in ((b.cache.k_steps, ks), (b.cache.v_steps, vs)):
            assert np.array_equal(np_(have.float())[page, :, np.arange(n) % 64], want)


@gpu
def test_append_in_place_and_idle_sequences():
    lens = [(1, 4), (1, 0), (3, 2)]  # an idle sequence; one whose first token has no position
    b = Batch(lens, 128, 8, 2, 16)
    q, k, v = b.qkv()
    before = np_(q.float())
    bl.kv4_append(q, k, v, table(8, 128), *b.args(), out=q)
    assert bl.get_device_error() == 0
    got = np_(q.float())
    cs = np_(table(8, 128))
    for m, p in ((0, 3), (1, None), (2, None), (3, 0), (4, 1)):
        want = before[m] if p is None else ref.bf16_round(ref.rotate(before[m], cs[p][None]))
        assert np.array_equal(got[m], want), m
    o = bl.kv4_attention(q, *b.args(), 3)
    assert (np_(o[1].float()) == 0).all() and (np_(o[2].float()) == 0).all()
    b.check(q, o)


ATTEND = [
    ([(1, 1)], 128, 20, 5, 64),
    ([(1, 16), (1, 15), (1, 17), (1, 64), (1, 63), (1, 65), (1, 129)], 128, 4, 1, 16),
    ([(1, 777), (1, 3), (1, 4096)], 128, 20, 5, 32),
    ([(1, 700), (1, 9)], 128, 8, 8, 64),      # a head of its own each
    ([(1, 500), (1, 1), (0, 77), (1, 0)], 128, 12, 1, 128),  # 12 heads share one; no new token; idle
    ([(1, 333), (1, 90)], 128, 48, 3, 256),   # 16 heads share one
    ([(1, 200)], 128, 40, 2, 64),             # 20
    ([(2, 90), (3, 3), (1, 257), (4, 512)], 128, 8, 2, 64),
    ([(1, 65), (1, 640), (1, 31)], 64, 16, 4, 16),
    ([(3, 100), (2, 2), (5, 1030)], 64, 15, 5, 128),
    ([(1, 300)], 64, 24, 2, 32),
    ([(40, 40), (17, 130), (1, 513)], 128, 20, 5, 32),
    ([(129, 300), (64, 64)], 64, 6, 6, 64),
    ([(257, 700), (5, 5), (1, 900)], 128, 8, 2, 16),
    ([(1, 1 + 37 * i % 300) for i in range(150)], 64, 4, 2, 16),
]


@gpu
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(case):
    lens, D, H, Hk, P = ATTEND[case]
    b = Batch(lens, D, H, Hk, P, seed=case, spare_rows=2)
    n = sum(kv for _, kv in lens)
    loud = 1 + 9 * (b.rng.random(D) < 0.05)
    b.fill((b.rng.standard_normal((n, Hk, D)) * loud).astype(np.float32), b.rng.standard_normal((n, Hk, D)).astype(np.float32))
    q = torch.from_numpy(b.rng.standard_normal((b.M, H, D)) * 2).to(torch.bfloat16).cuda()
    out = torch.full((b.M, H, D), -7.0, dtype=torch.bfloat16, device="cuda")
    bl.kv4_attention(q, *b.args(), b.max_q, out=out)
    assert bl.get_device_error() == 0
    b.check(q, out)
    assert (np_(out[int(b.starts[-1]):].float()) == -7.0).all()
    again = bl.kv4_attention(q, *b.args(), b.max_q)
    real = slice(0, int(b.starts[-1]))
    assert torch.equal(out[real].view(torch.int16), again[real].view(torch.int16))


@gpu
@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_attention_scale_and_strides(scale):
    """A sharp and a flat softmax; q and out as column blocks of wider rows."""
    b = Batch([(1, 900), (2, 70), (40, 200)], 128, 8, 2, 64, seed=5)
    n = 1170
    b.fill(b.rng.standard_normal((n, 2, 128)).astype(np.float32), b.rng.standard_normal((n, 2, 128)).astype(np.float32) + 1)
    wide = torch.from_numpy(b.rng.standard_normal((b.M, 12 * 128)) * 3).to(torch.bfloat16).cuda()
    q = wide[:, 256:256 + 1024].unflatten(1, (8, 128))
    o = torch.full((b.M, 10 * 128), -7.0, dtype=torch.bfloat16, device="cuda")
    bl.kv4_attention(q, *b.args(), 40, scale=scale, out=o[:, 128:128 + 1024].unflatten(1, (8, 128)))
    b.check(q, o[:, 128:128 + 1024].unflatten(1, (8, 128)), scale=scale)
    assert (np_(o[:, :128].float()) == -7.0).all() and (np_(o[:, 1152:].float()) == -7.0).all()


@gpu
@pytest.mark.parametrize("new", [4, 90])
def test_marked_tokens_reach_only_rows_that_see_them(new):
    """A NaN key, an infinite value and a huge value: rows that see the token are NaN in its head, others are not."""
    lens = [(new, 100 + new), (new, 60 + new)]
    b = Batch(lens, 128, 8, 2, 32, seed=3)
    n = sum(kv for _, kv in lens)
    k, v = (b.rng.standard_normal((n, 2, 128)).astype(np.float32) for _ in range(2))
    k[100 + new - 3, 0, 5] = np.nan             # sequence 0, third token from the end, head 0
    v[100 + new - 2, 1, 127] = np.inf           # sequence 0, second from the end, head 1
    v[100 + new + 60 + new - 1, 0, 64] = 2e36   # sequence 1, its last token, head 0
    b.fill(k, v)
    q = torch.from_numpy(b.rng.standard_normal((b.M, 8, 128))).to(torch.bfloat16).cuda()
    out = np_(bl.kv4_attention(q, *b.args(), new).float())
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[new - 3:new, :4] = True
    want[new - 2:new, 4:] = True
    want[2 * new - 1, :4] = True
    assert np.array_equal(nan, want)
    b.check(q, torch.from_numpy(out))
    # and the append marks them the same way
    c = Batch([(1, 1)], 128, 8, 2, 32)
    qq, kk, vv = c.qkv()
    kk[0, 1, 64] = float("nan")
    vv[0, 0, 9] = -float("inf")
    bl.kv4_append(qq, kk, vv, table(1, 128), *c.args())
    rk, rv = bl.kv4_read(*c.args(), 1)
    assert torch.isnan(rk).all() and (rv == 0).all()


@gpu
@pytest.mark.parametrize("new", [1, 90])
def test_queries_without_a_softmax(new):
    """A NaN or infinite query makes its row NaN in its head, also where every score is -inf; others are as before."""
    lens = [(new, 900 + new), (new, 40 + new)]
    b = Batch(lens, 128, 8, 2, 32, seed=6)
    n = sum(kv for _, kv in lens)
    k = b.rng.standard_normal((n, 2, 128)).astype(np.float32)
    k[:, :, 7] = 1.0 + np.abs(k[:, :, 7])  # one sign: an infinite query there has scores of one sign
    b.fill(k, b.rng.standard_normal((n, 2, 128)).astype(np.float32))
    q = torch.from_numpy(b.rng.standard_normal((b.M, 8, 128))).to(torch.bfloat16).cuda()
    want = np_(bl.kv4_attention(q, *b.args(), new).float())
    q[0, 1, 7] = -float("inf")
    q[new - 1, 5, 7] = float("inf")
    q[2 * new - 1, 2, 100] = float("nan")
    got = np_(bl.kv4_attention(q, *b.args(), new).float())
    bad = np.zeros(got.shape[:2], bool)
    bad[0, 1] = bad[new - 1, 5] = bad[2 * new - 1, 2] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], want[~bad])


@gpu
@pytest.mark.parametrize("heads", [4, 60])
def test_a_later_key_may_outweigh_all_before_it_by_any_factor(heads):
    """One key, at each column of a block in turn, whose weight is 2^gap times that of everything before it."""
    D, Hk, n = 64, heads // 20 or 1, 512
    b = Batch([(1, n)] * 128, D, heads, Hk, 64, seed=11)
    k = np.zeros((128, n, Hk, D), np.float32)
    v = np.full((128, n, Hk, D), 7.0, np.float32)
    k[np.arange(128), 256 + np.arange(128)] = 7.0
    v[np.arange(128), 256 + np.arange(128)] = -3.5
    b.fill(k.reshape(-1, Hk, D), v.reshape(-1, Hk, D))
    for gap in (1, 9, 12, 100, 126, 127.4, 128, 150, 260, 390, 500, 1100):
        q = torch.full((128, heads, D), gap * np.log(2) / (7 * D * D ** -0.5), dtype=torch.bfloat16, device="cuda")
        out = bl.kv4_attention(q, *b.args(), 1)
        if gap < 30:
            b.check(q, out)
        else:  # the rest weighs less than 512 * 2^-30
            assert (np_(out.float()) == -3.5).all(), gap


@gpu
@pytest.mark.parametrize("heads", [4, 20])
def test_scores_that_overflow_downwards_leave_the_rest(heads):
    """Keys whose score is -inf in fp32 weigh nothing; those behind them do, however low their scores."""
    D, n = 64, 700
    b = Batch([(1, n)] * 3, D, heads, 1, 64, seed=12)
    k = np.full((3, n, 1, D), -3.75e-4, np.float32)
    v = np.full((3, n, 1, D), 7.0, np.float32)
    k[:, :300] = -1e35
    v[:, :300] = -7.0
    b.fill(k.reshape(-1, 1, D), v.reshape(-1, 1, D))
    q = torch.full((3, heads, D), 1e5, dtype=torch.bfloat16, device="cuda")
    assert (np_(bl.kv4_attention(q, *b.args(), 1).float()) == 7.0).all()


@gpu
def test_attention_reads_far_pages_and_shared_ones():
    """Pages whose byte offsets pass 2^31 (and 2^32 in the codes of both arrays), a prefix two sequences share."""
    D, Hk, P = 128, 8, 256
    pages = 34000  # 34000 * 8 * 256 * 64 bytes = 4.46 GB of codes each
    small = Batch([(1, 600), (1, 700), (40, 520)], D, 16, Hk, P, seed=9)
    n = 1820
    small.fill(small.rng.standard_normal((n, Hk, D)).astype(np.float32), small.rng.standard_normal((n, Hk, D)).astype(np.float32))
    small.table[1, 0] = small.table[0, 0]  # shared prefix page
    dev = "cuda"
    big = [torch.empty((pages, *t.shape[1:]), dtype=t.dtype, device=dev) for t in (small.cache.k_codes, small.cache.k_steps, small.cache.v_codes, small.cache.v_steps)]
    used = [p for s, (_, kv) in enumerate(small.lens) for p in small.table[s, : -(-kv // P)].tolist()]
    far = {p: pages - 1 - i for i, p in enumerate(dict.fromkeys(used))}
    for p, f in far.items():
        for t, o in zip(big, (small.cache.k_codes, small.cache.k_steps, small.cache.v_codes, small.cache.v_steps)):
            t[f] = o[p]
    tab = torch.tensor([[far.get(int(p), 0) for p in row[:3]] for row in small.table], dtype=torch.int32, device=dev)
    q = torch.from_numpy(small.rng.standard_normal((small.M, 16, D))).to(torch.bfloat16).cuda()
    cache = bl.Kv4Cache(*big)
    out = bl.kv4_attention(q, cache, tab, small.d_len, small.d_start, 40)
    assert bl.get_device_error() == 0
    small.check(q, out)
    # appended and read back there too
    qq, k, v = small.qkv()
    bl.kv4_append(qq, k, v, table(700, D), cache, tab, small.d_len, small.d_start)
    bl.kv4_append(qq, k, v, table(700, D), small.cache, torch.from_numpy(small.table[:, :3].copy()).cuda(), small.d_len, small.d_start)
    a, b = bl.kv4_read(cache, tab, small.d_len, small.d_start, small.M), bl.kv4_read(small.cache, torch.from_numpy(small.table[:, :3].copy()).cuda(), small.d_len, small.d_start, small.M)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_attention_long_sequence(new):
    b = Batch([(new, 70001), (new, 200)], 64, 4, 1, 256, seed=2)
    n = 70201
    rng = b.rng
    b.cache.k_codes.copy_(torch.from_numpy(rng.integers(0x11, 0x100, b.cache.k_codes.shape, dtype=np.uint8)).cuda())
    for t in (b.cache.k_steps, b.cache.v_steps):
        t.copy_(torch.from_numpy(ref.five_bits(rng.uniform(0.1, 0.5, t.shape).astype(np.float32))).cuda())
    q = torch.from_numpy(rng.standard_normal((b.M, 4, 64))).to(torch.bfloat16).cuda()
    out = bl.kv4_attention(q, *b.args(), new)
    assert bl.get_device_error() == 0 and n
    b.check(q, out)


@gpu
@pytest.mark.parametrize("new,heads,D", [(1, 1, 64), (1, 3, 128), (2, 4, 64), (5, 3, 128), (7, 3, 64), (5, 4, 128), (30, 4, 128), (43, 3, 64)])
def test_few_rows_in_many_pieces(new, heads, D):
    """One long sequence whose keys all blocks share, beside one that a single block holds."""
    b = Batch([(new, 9001), (new, new + 3)], D, heads, 1, 64, seed=new)
    n = 9001 + new + 3
    k = b.rng.standard_normal((n, 1, D)).astype(np.float32)
    k[:3000] *= 3  # maxima that differ from piece to piece
    b.fill(k, b.rng.standard_normal((n, 1, D)).astype(np.float32))
    q = torch.from_numpy(b.rng.standard_normal((b.M, heads, D))).to(torch.bfloat16).cuda()
    out = bl.kv4_attention(q, *b.args(), new)
    assert bl.get_device_error() == 0
    b.check(q, out)


@gpu
def test_bad_batches_are_reported_and_stay_inside():
    """Every case is one that the kernels' own bounds checks catch."""
    BAD = 10

    def fresh():
        b = Batch([(1, 100), (2, 50)], 128, 8, 2, 16, seed=1)
        b.fill(np.ones((150, 2, 128), np.float32), np.ones((150, 2, 128), np.float32))
        q, k, v = b.qkv()
        return b, q, k, v

    def both(b, q, k, v, max_q=2, max_pos=200):
        bl.kv4_append(q, k, v, table(max_pos, 128), *b.args())
        one = bl.get_device_error()
        bl.kv4_attention(q, *b.args(), max_q)
        return one, bl.get_device_error()

    assert both(*fresh()) == (0, 0)
    b, q, k, v = fresh()
    b.d_table[0, 6] = b.pages  # the page of the new token
    assert both(b, q, k, v) == (BAD, BAD)
    b, q, k, v = fresh()
    b.d_table[1, 0] = -1       # a page that only attention reads
    assert both(b, q, k, v) == (0, BAD)
    b, q, k, v = fresh()
    b.d_len[1] = 10000         # longer than the table's row
    assert both(b, q, k, v) == (BAD, BAD)
    b, q, k, v = fresh()
    b.d_len[1] = -5
    assert both(b, q, k, v) == (BAD, BAD)
    b, q, k, v = fresh()
    assert both(b, q, k, v, max_q=1) == (0, BAD)
    assert both(b, q, k, v, max_pos=99) == (BAD, 0)
    b, q, k, v = fresh()
    b.d_start[2] = 1000        # past the rows of q
    assert both(b, q, k, v, max_q=1 << 20) == (BAD, BAD)
    assert bl.get_device_error() == 0
    # the sequences that are in order keep their results
    b, q, k, v = fresh()
    good = bl.kv4_attention(q, *b.args(), 2)
    b.d_len[1] = 10000
    part = bl.kv4_attention(q, *b.args(), 2)
    assert torch.equal(good[:1], part[:1]) and bl.get_device_error() == BAD


@gpu
def test_streams_graphs_and_two_calls_at_once():
    b = Batch([(1, 3000), (1, 40), (1, 900)], 128, 20, 5, 64, seed=4)
    n = 3940
    b.fill(b.rng.standard_normal((n, 5, 128)).astype(np.float32), b.rng.standard_normal((n, 5, 128)).astype(np.float32))
    q, k, v = b.qkv()
    cs = table(3000, 128)
    rot = bl.kv4_append(q, k, v, cs, *b.args())
    want = bl.kv4_attention(rot, *b.args(), 1)
    b.check(rot, want)
    torch.cuda.synchronize()
    # two streams at once: scratch is each call's own
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(bl.kv4_attention(rot, *b.args(), 1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[0] + outs[1])
    # two captured graphs, replayed at once
    graphs, res = [], []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = bl.kv4_append(q, k, v, cs, *b.args())
            res.append(bl.kv4_attention(r, *b.args(), 1))
        graphs.append(g)
    for r in res:
        r.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in res)
    # the lengths are read by the replay, not by the capture
    b.lens = [(1, 2500), (1, 40), (1, 900)]
    b.d_len[0] = 2500
    graphs[0].replay()
    torch.cuda.synchronize()
    b.check(bl.kv4_append(q, k, v, cs, *b.args()), res[0])


@gpu
def test_binding_refusals():
    b = Batch([(1, 5)], 64, 4, 2, 16)
    q, k, v = b.qkv()
    cs = table(5, 64)
    for f in (lambda: bl.kv4_attention(q.float(), *b.args(), 1), lambda: bl.kv4_attention(q[:, :, :32], *b.args(), 1),
              lambda: bl.kv4_attention(q.transpose(1, 2).contiguous().transpose(1, 2), *b.args(), 1),
              lambda: bl.kv4_attention(q, b.cache, b.d_table.long(), b.d_len, b.d_start, 1),
              lambda: bl.kv4_attention(q, b.cache, b.d_table, b.d_len, b.d_start[:1], 1),
              lambda: bl.kv4_append(q, k[:, :1], v, cs, *b.args()), lambda: bl.kv4_append(q, k, v, cs[:, :32].contiguous(), *b.args()),
              lambda: bl.kv4_append(q, k, v, cs.cpu(), *b.args()),
              lambda: bl.Kv4Cache(b.cache.k_codes, b.cache.k_steps[:1], b.cache.v_codes, b.cache.v_steps)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(bl.BitLinearError):
        bl.kv4_attention(q, *b.args(), 1, scale=-1.0)
    assert bl.kv4_attention(q[:0], b.cache, b.d_table, b.d_len, torch.zeros(2, dtype=torch.int32, device="cuda"), 1).shape == (0, 4, 64)
