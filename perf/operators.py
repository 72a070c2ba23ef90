"""What is measured of the attention side of a decoder block and of the 8-bit product.

Three operators, each in its plain form (elementary torch operations) and, with
``own``, through the library's calls:

  append   rotate q and k of a batch's new tokens, quantise k and v to 4 bits,
           write them to their pages, and read the stored values back
  attend   attention of the batch's tokens over the 4-bit paged cache
  product  8-bit integer product with a scale for each token and channel

A batch is ``seqs`` sequences with ``q_min``..``q_max`` new tokens each and
``kv_min``..``kv_max`` tokens in the cache, the new ones among them; the lengths
follow from the case alone (``ragged`` seeds them), the values from the seed.
"""
import random

import torch

own = False

GROUP = 32        # dims that share one quantisation step
THETA = 500000.0  # base of the rotation's wavelengths


# --------------------------------------------------------------------------- cases

def _batch(op, name, seqs, q, kv, heads, kv_heads, dim, page, ragged):
    return {"name": name, "op": op, "seqs": seqs, "q_min": q[0], "q_max": q[1], "kv_min": kv[0], "kv_max": kv[1],
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged}


def _product(name, M, N, K, out, rmsnorm):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "out": out, "rmsnorm": rmsnorm}


def listed():
    return [
        # one chat answering: the new token of one sequence (heads of a 2560-wide block: 2560 / 640 rows)
        _batch("append", "append_one", 1, (1, 1), (4001, 4001), 20, 5, 128, 64, 1),
        # a serving step: one token of each running sequence, small pages (heads of an 8192-wide block)
        _batch("append", "append_step", 64, (1, 1), (1, 8192), 64, 8, 128, 16, 2),
        # prompts of a few users admitted together
        _batch("append", "append_prompts", 6, (100, 4096), (100, 4096), 20, 5, 128, 64, 3),
        # one chat answering
        _batch("attend", "decode_one", 1, (1, 1), (4001, 4001), 20, 5, 128, 64, 4),
        # a serving step of many sequences of very different lengths
        _batch("attend", "decode_step", 64, (1, 1), (1, 8192), 20, 5, 128, 32, 5),
        # few long documents, one token each
        _batch("attend", "decode_long", 2, (1, 1), (100001, 131072), 64, 8, 128, 128, 6),
        # a few tokens a sequence at once (speculation), narrow heads
        _batch("attend", "verify", 16, (2, 4), (33, 4096), 16, 4, 64, 16, 7),
        # prompts of a few users admitted together
        _batch("attend", "prompts", 6, (100, 4096), (100, 4096), 20, 5, 128, 64, 8),
        # the next chunk of a long prompt
        _batch("attend", "chunk", 1, (2047, 2047), (30001, 30001), 20, 5, 128, 256, 9),
        # the vocabulary head of one token: final norm, fp32 logits, an odd vocabulary
        _product("head_one", 1, 100003, 2560, "fp32", True),
        # an 8-bit layer in a serving step
        _product("layer_step", 16, 6912, 2560, "bf16", False),
        # an 8-bit layer over prompts
        _product("layer_prompts", 2048, 28672, 8192, "bf16", False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["append", "step", "prompts", "chunk", "few_rows", "many_rows"])
    heads, kv_heads, dim = rng.choice([(20, 5, 128), (16, 4, 64), (64, 8, 128), (8, 8, 128), (15, 5, 64), (12, 1, 128)])
    page = rng.choice([16, 32, 64, 128, 256])
    ragged = rng.randrange(1 << 20)
    if kind == "append":
        q = _log(rng, 1, 4096)
        seqs = _log(rng, 1, max(1, min(128, 16384 // q)))
        case = _batch("append", "", seqs, (max(1, q // 3), q), (q, q + _log(rng, 1, 4096)), heads, kv_heads, dim, page, ragged)
    elif kind == "step":
        kv = _log(rng, 17, 65536)
        seqs = _log(rng, 1, max(1, min(128, 500000 // (kv * kv_heads))))
        q = rng.choice([1, 1, 1, 2, 3, 5])
        case = _batch("attend", "", seqs, (1, q), (max(q, kv // 8), kv), heads, kv_heads, dim, page, ragged)
    elif kind == "prompts":
        q = _log(rng, 17, 3000)
        seqs = _log(rng, 1, max(1, min(16, 10000 // q)))
        case = _batch("attend", "", seqs, (max(1, q // 4), q), (q, q), 20, 5, dim, page, ragged)
    elif kind == "chunk":
        q = _log(rng, 17, 1500)
        case = _batch("attend", "", 1, (q, q), (q + 1, q + _log(rng, 100, 20000)), 20, 5, dim, page, ragged)
    else:
        N, K = rng.choice([(2560, 2560), (6912, 2560), (2560, 6912), (8192, 8192), (28672, 8192)])
        N += rng.choice([0, 0, 1, 7, 333])
        M = _log(rng, 1, 16) if kind == "few_rows" else _log(rng, 17, 2000)
        case = _product("", M, N, K, rng.choice(["bf16", "fp32"]), rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence."""
    r = random.Random(case["ragged"])
    got = []
    for _ in range(case["seqs"]):
        q = r.randint(case["q_min"], case["q_max"])
        whole = case["kv_max"] == case["q_max"]  # prompts: nothing was in the cache before
        got.append((q, q if whole else r.randint(max(q, case["kv_min"]), case["kv_max"])))
    return got


def work(case):
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": N * K + 4 * N + 2 * M * K + out * M * N, "flops": 2.0 * M * N * K}
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    rows = sum(q for q, _ in lens)
    token = 2 * Hk * (D // 2 + 2 * (D // GROUP))  # one token's codes and steps
    if case["op"] == "append":
        # q, k, v and the table's rows in; q, the cache's entries and the values read back out
        return {"bytes": rows * (2 * (H + 2 * Hk) * D + 4 * D + 2 * H * D + token + token + 4 * Hk * D), "flops": 6.0 * rows * (H + Hk) * D}
    pairs = sum(q * (kv - q) + q * (q + 1) // 2 for q, kv in lens)
    return {"bytes": sum(kv for _, kv in lens) * token + 4 * rows * H * D, "flops": 4.0 * pairs * H * D}


# --------------------------------------------------------------------------- inputs

def _full(x, like):
    return torch.full((), x, dtype=like.dtype, device=like.device)  # a divisor on the device: a true division


def _quantise(x):
    """x [..., D] fp32 -> (codes uint8 0..15 [..., D], steps fp32 [..., D / 32])."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    top = g.abs().amax(-1)
    bits = (top / _full(7.0, top)).view(torch.int32)
    bits = (bits + 0x3FFFF + ((bits >> 19) & 1)) & ~0x7FFFF  # five significant bits, ties to even
    step = torch.where(top < 2.0 ** -100, torch.zeros_like(top), bits.view(torch.float32))
    code = torch.round(g / torch.where(step > 0, step, torch.ones_like(step)).unsqueeze(-1))
    code = torch.where((step > 0).unsqueeze(-1), code, torch.zeros_like(code))
    return (code + 8).to(torch.uint8).reshape(x.shape), step


def _pack(code):
    """Codes [..., D] -> bytes [..., D / 2]: octet t (8 dims) of group g is word t * (D / 32) + g, dim j of it in bits 4j.."""
    D = code.shape[-1]
    c = code.reshape(*code.shape[:-1], D // GROUP, 4, 8).transpose(-3, -2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(*code.shape[:-1], D // 2)


def _unpack(byte, step):
    """The fp32 values [..., D] of packed bytes [..., D / 2] and steps [..., D / 32]."""
    D = 2 * byte.shape[-1]
    c = torch.stack([byte & 15, byte >> 4], -1).reshape(*byte.shape[:-1], 4, D // GROUP, 8).transpose(-3, -2)
    return ((c.to(torch.float32) - 8.0).reshape(*byte.shape[:-1], D // GROUP, GROUP) * step.to(torch.float32).unsqueeze(-1)).reshape(*byte.shape[:-1], D)


def _normal(g, shape, spread=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * spread


def _activations(g, rows, width):
    """Normal values with a few loud channels, as layers of a model see them."""
    x = _normal(g, (rows, width))
    x[:, torch.randperm(width, generator=g, device="cuda")[: width // 100]] *= 20.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(g, M, K).to(torch.bfloat16)
        W = _normal(g, (N, K), 0.02)
        top = W.abs().amax(1)
        wstep = top / _full(127.0, top)
        Wq = torch.round(W / wstep.unsqueeze(1)).clamp_(-127, 127).to(torch.int8)
        return {"op": "product", "x": x, "Wq": Wq, "wstep": wstep, "rmsnorm": case["rmsnorm"],
                "out": torch.float32 if case["out"] == "fp32" else torch.bfloat16}
    H, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case)
    rows = sum(q for q, _ in lens)
    starts, at = [0], 0
    for q, _ in lens:
        at += q
        starts.append(at)
    width = max(-(-kv // P) for _, kv in lens)
    used = [-(-kv // P) for _, kv in lens]
    pages = sum(used) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table, at = torch.zeros((len(lens), width), dtype=torch.int32), 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    s = {"op": case["op"], "H": H, "Hk": Hk, "D": D, "P": P, "rows": rows, "max_q": max(q for q, _ in lens), "max_kv": max(kv for _, kv in lens),
         "table": table.cuda(), "kv_len": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
         "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda")}
    shape = (pages, Hk, P)
    if case["op"] == "append":
        # what the stacked projection of a block gives: q, k and v side by side in one row
        qkv = _activations(g, rows, (H + 2 * Hk) * D).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, Hk * D, Hk * D], 1))
        far = torch.arange(s["max_kv"], device="cuda", dtype=torch.float64).unsqueeze(1)
        angle = far * THETA ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros((*shape, D // 2), dtype=torch.uint8, device="cuda")
            s[name + "_steps"] = torch.zeros((*shape, D // GROUP), dtype=torch.bfloat16, device="cuda")
        return s
    s["q"] = _normal(g, (rows, H, D), 2.0).to(torch.bfloat16)
    for name in ("k", "v"):
        code, step = _quantise(_normal(g, (*shape, D)))
        s[name + "_codes"], s[name + "_steps"] = _pack(code), step.to(torch.bfloat16)
    return s


# --------------------------------------------------------------------------- plain forms

def _where(s):
    """Sequence and position of each row, and its place in the cache (page, offset)."""
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = s["kv_len"][seq].long() - s["q_start"][seq + 1].long() + row
    return seq, pos, s["table"][seq, pos // s["P"]].long(), pos % s["P"]


def _append(s):
    D = s["D"]
    _, pos, page, at = _where(s)
    cos, sin = s["cos_sin"][pos].unsqueeze(1).split(D // 2, 2)

    def rotate(x):
        a, b = x.to(torch.float32).split(D // 2, 2)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], 2)

    values = []
    for name, x in (("k", rotate(s["k"])), ("v", s["v"].to(torch.float32))):
        code, step = _quantise(x)
        s[name + "_codes"][page, :, at] = _pack(code)
        s[name + "_steps"][page, :, at] = step.to(torch.bfloat16)
        values.append(_unpack(s[name + "_codes"][page, :, at], s[name + "_steps"][page, :, at]).to(torch.bfloat16))
    return {"q": rotate(s["q"]).to(torch.bfloat16), "k": values[0], "v": values[1]}


def _attend(s):
    H, Hk, D, P, n = s["H"], s["Hk"], s["D"], s["P"], s["max_q"]
    S, W = s["table"].shape
    page = s["table"].long()
    k, v = (_unpack(s[x + "_codes"][page], s[x + "_steps"][page]).transpose(1, 2).reshape(S, Hk, W * P, D) for x in ("k", "v"))
    seq, pos, _, _ = _where(s)
    at = torch.arange(s["rows"], device="cuda") - s["q_start"][seq]
    q = torch.zeros((S, n, H, D), dtype=torch.float32, device="cuda")
    q[seq, at] = s["q"].to(torch.float32)
    q = q.reshape(S, n, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, (H // Hk) * n, D)
    last = torch.zeros((S, n), dtype=torch.int64, device="cuda")
    last[seq, at] = pos
    score = (q @ k.transpose(2, 3)) * (D ** -0.5)
    hidden = torch.arange(W * P, device="cuda") > last.unsqueeze(2)
    score.view(S, Hk, H // Hk, n, W * P).masked_fill_(hidden[:, None, None], float("-inf"))
    score -= score.amax(3, keepdim=True)
    score.exp_()
    out = (score @ torch.where((torch.arange(W * P, device="cuda") < s["kv_len"].unsqueeze(1))[:, None, :, None], v, torch.zeros_like(v))) / score.sum(3, keepdim=True)
    out = out.reshape(S, Hk, H // Hk, n, D).permute(0, 3, 1, 2, 4).reshape(S, n, H, D)
    return out[seq, at].to(torch.bfloat16)


def _codes(x, rmsnorm):
    """Codes of each token's activations as fp32 whole numbers, and their scales."""
    x = x.to(torch.float32)
    if rmsnorm:
        mean = x.double().square().sum(1) / x.shape[1]
        x = x * torch.sqrt(mean.to(torch.float32) + 1e-5).reciprocal().unsqueeze(1)
    top = x.abs().amax(1).clamp_min(1e-5)
    scale = _full(127.0, top) / top
    return torch.round(x * scale.unsqueeze(1)).clamp_(-128, 127), scale


def _product_plain(s):
    code, scale = _codes(s["x"], s["rmsnorm"])
    acc = code @ s["Wq"].to(torch.float32).t()
    return (acc * s["wstep"] * scale.reciprocal().unsqueeze(1)).to(s["out"])


# --------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        import bitlinear_w1_a8_02_b200 as bl

        if s["op"] == "product":
            return bl.forward_int8(s["Wq"], s["wstep"], s["x"], rmsnorm=s["rmsnorm"], out_dtype=s["out"])
        cache = bl.Kv4Cache(s["k_codes"], s["k_steps"], s["v_codes"], s["v_steps"])
        if s["op"] == "append":
            q = bl.kv4_append(s["q"], s["k"], s["v"], s["cos_sin"], cache, s["table"], s["kv_len"], s["q_start"])
            k, v = bl.kv4_read(cache, s["table"], s["kv_len"], s["q_start"], s["rows"])
            return {"q": q, "k": k, "v": v}
        return bl.kv4_attention(s["q"], cache, s["table"], s["kv_len"], s["q_start"], s["max_q"])
    return {"product": _product_plain, "append": _append, "attend": _attend}[s["op"]](s)


# --------------------------------------------------------------------------- the definition in 64 bits

def _exact_group(x):
    """Values that a group-quantised fp64 x stands for."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top = g.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / 7.0)
    step = torch.ldexp(torch.round(m * 32.0), e - 5)
    return (torch.round(g / torch.where(step > 0, step, torch.ones_like(step))) * step).reshape(x.shape)


def _exact_values(s, name, page):
    """fp64 values [tokens, D] of one head's pages: (codes [pages, P, D / 2], steps) -> by the layout's definition."""
    byte, step = s[name + "_codes"][page], s[name + "_steps"][page].double()
    D, G = s["D"], s["D"] // GROUP
    out = torch.empty((*byte.shape[:-1], D), dtype=torch.float64, device=byte.device)
    for d in range(D):
        group, octet, j = d // GROUP, d % GROUP // 8, d % 8
        b = byte[..., 4 * (octet * G + group) + j // 2]
        out[..., d] = ((b >> (4 * (j % 2)) & 15).double() - 8) * step[..., group]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        x = s["x"].float()
        if s["rmsnorm"]:  # the normed activations and the scale are fp32 by definition
            x = x * (1.0 / torch.sqrt((s["x"].double().pow(2).mean(1)).float() + 1e-5))[:, None]
        scale = torch.div(torch.full_like(x[:, 0], 127.0), x.abs().max(1).values.clamp(min=1e-5))
        code = torch.round(x * scale[:, None]).double()
        y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
        for n in range(0, case["N"], 8192):
            y[:, n:n + 8192] = (code @ s["Wq"][n:n + 8192].double().t()) * s["wstep"][n:n + 8192].double() / scale.double()[:, None]
        return y
    D, P, Hk = s["D"], s["P"], s["Hk"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    if case["op"] == "append":
        pos = torch.cat([torch.arange(kv - (b - a), kv, device="cuda") for a, b, kv in zip(starts, starts[1:], lens)])
        cs = s["cos_sin"].double()[pos][:, None]
        c, z = cs[..., : D // 2], cs[..., D // 2:]

        def turn(x):
            a, b = x.double()[..., : D // 2], x.double()[..., D // 2:]
            return torch.cat((a * c - b * z, a * z + b * c), -1)

        return {"q": turn(s["q"]), "k": _exact_group(turn(s["k"])), "v": _exact_group(s["v"].double())}
    out = torch.zeros((s["rows"], s["H"], D), dtype=torch.float64, device="cuda")
    group = s["H"] // Hk
    for i, (a, b, kv) in enumerate(zip(starts, starts[1:], lens)):
        page = s["table"][i, : -(-kv // P)].long()
        for h in range(Hk):
            one = {"D": D, **{x: s[x][:, h] for x in ("k_codes", "k_steps", "v_codes", "v_steps")}}
            k, v = (_exact_values(one, x, page).reshape(-1, D)[:kv] for x in ("k", "v"))
            for j in range(a, b, 512):  # rows at a time
                rows = torch.arange(j, min(b, j + 512), device="cuda")
                q = s["q"][rows, h * group:(h + 1) * group].double()
                z = torch.einsum("rgd,kd->rgk", q, k) * D ** -0.5
                seen = torch.arange(kv, device="cuda") <= (kv - b + rows)[:, None]
                p = torch.softmax(z.masked_fill(~seen[:, None], float("-inf")), -1)
                out[rows, h * group:(h + 1) * group] = torch.einsum("rgk,kd->rgd", p, v)
    return out
