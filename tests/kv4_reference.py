"""The 4-bit paged cache and the attention over it, written plainly in numpy: the
quantisation and rotation as the definition's fp32 steps (so codes and steps are
compared bit for bit), the attention in 64 bits with the error that the kernel's
roundings allow."""
import numpy as np

GROUP = 32


def bf16_round(x):
    """fp32 -> the nearest bf16 (ties to even), as fp32; NaN stays NaN."""
    x = np.asarray(x, np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def rotate(x, cos_sin, interleaved=False):
    """x [..., D] fp32 (bf16 values), cos_sin [..., D] fp32."""
    D = x.shape[-1]
    c, s = cos_sin[..., :D // 2], cos_sin[..., D // 2:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :D // 2], x[..., D // 2:])
    with np.errstate(all="ignore"):
        ra = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        rb = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    if interleaved:
        return np.stack([ra, rb], -1).reshape(x.shape)
    return np.concatenate([ra, rb], -1)


def five_bits(t):
    """Positive fp32 -> the nearest value of five significant bits, ties to even."""
    m, e = np.frexp(t.astype(np.float64))
    return np.ldexp(np.rint(m * 32.0), e - 5).astype(np.float32)


def quantise(x):
    """x [..., D] fp32 -> (codes int [-7, 7] [..., D], steps fp32 [..., D / 32])."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)
        step = np.where(top < 2.0 ** -100, 0, five_bits((top / np.float32(7)).astype(np.float32))).astype(np.float32)
        c = np.where(step[..., None] > 0, np.rint((g / step[..., None]).astype(np.float32)), 0)
    return np.where(np.isfinite(c), c, 0).astype(np.int64).reshape(x.shape), step


def entry(k, v):
    """What one call stores for keys and values [..., D] fp32: (kc, ks, vc, vs), marked tokens included."""
    with np.errstate(all="ignore"):
        bad = ~((np.abs(k) < 2.0 ** 120).all(-1) & (np.abs(v) < 2.0 ** 120).all(-1))[..., None]
        kc, ks = quantise(k)
        vc, vs = quantise(v)
    return (np.where(bad, 0, kc), np.where(bad, np.float32(np.nan), ks), np.where(bad, 0, vc), np.where(bad, np.float32(0), vs))


def pack(c):
    """Codes [..., D] -> bytes [..., D / 2], dim by dim as the format says."""
    D = c.shape[-1]
    G = D // GROUP
    out = np.zeros((*c.shape[:-1], D // 2), np.uint8)
    for d in range(D):
        word = (d % GROUP // 8) * G + d // GROUP
        bit = 4 * (d % 8)
        out[..., 4 * word + bit // 8] |= ((c[..., d] + 8) << (bit % 8)).astype(np.uint8)
    return out


def unpack(b):
    """Bytes [..., D / 2] -> codes [..., D]."""
    D = 2 * b.shape[-1]
    G = D // GROUP
    out = np.zeros((*b.shape[:-1], D), np.int64)
    for d in range(D):
        word = (d % GROUP // 8) * G + d // GROUP
        bit = 4 * (d % 8)
        out[..., d] = (b[..., 4 * word + bit // 8].astype(np.int64) >> (bit % 8) & 15) - 8
    return out


def values(codes, steps):
    """fp64 values of packed codes [..., D / 2] and steps [..., D / 32]."""
    with np.errstate(all="ignore"):
        return unpack(codes) * np.repeat(steps.astype(np.float64), GROUP, -1)


def attention(q, k, v, ksteps, first, scale):
    """Causal attention in 64 bits: q [n, heads, D], k and v [len, D] of the one head they share, token i sees keys
    0 .. first + i. Returns (out, bound): how far a result with bf16 weights, fp32 sums and a bf16 output may be off.

    The bound, by term:
      * the weights p_j are rounded to bf16, half a step each (2^-8): 2^-8 sum p |v| / sum p;
      * a score is off by e_j: sums of n q over 32 dims plus -8 sum q, up to 65 terms, each partial sum at most 15 + 8
        times sum |q|, each sum off by at most 2^-23 of it (accumulators may truncate), times the step, over all groups
        (sums of c step q over 128 dims, partial sums at most 7 step sum |q|, are off by less); that moves p_j by a
        factor exp(scale e), in numerator and denominator;
      * fp32 sums over the keys: len terms, 2^-23 each, in numerator and denominator; exp2 and the scalings: 2^-20;
      * the result is rounded to bf16: 2^-8 of it."""
    n, heads, D = q.shape
    length = k.shape[0]
    out = np.zeros((n, heads, D))
    bound = np.zeros((n, heads, D))
    for i in range(n):
        m = min(length, first + i + 1)
        if m <= 0:
            continue
        with np.errstate(all="ignore"):
            z = scale * (q[i] @ k[:m].T)
            p = np.exp(z - z.max(-1, keepdims=True))
            w = p / p.sum(-1, keepdims=True)
            out[i] = w @ v[:m]
            spread = w @ np.abs(v[:m])
            per_group = np.abs(q[i]).reshape(heads, -1, GROUP).sum(-1)  # [heads, G]
            e = scale * 65 * 2.0 ** -23 * 23 * (per_group @ ksteps[:m].astype(np.float64).T).max(-1, keepdims=True)
            bound[i] = spread * (2.0 ** -8 + 2 * np.expm1(e) + 2 * m * 2.0 ** -23 + 2.0 ** -20) + np.abs(out[i]) * 2.0 ** -8
    return out, bound * 1.01 + 1e-30
