"""Cases that measure the low-bit serving operators: MXFP4 weights (E2M1 values with a power-of-two scale for every 32
along a row) and a paged cache of 8-bit keys and values with a power-of-two scale for every page and head.

``run`` computes an operator in its plain form, or, where ``own`` is true, through the library's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 32  # values that share an MXFP4 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ROPE_BASE = 10000.0
EXP_MIN, EXP_MAX = -100, 120  # the exponents a cache scale takes
WORKSPACE = 64 << 20
#: query heads and key/value heads
HEADS = ((32, 32), (64, 8), (40, 8), (28, 4), (8, 1))


def listed():
    return [
        # export of the 8192 x 28672 layer after tuning: weights with their learned offsets and clip factors in, fake-quantised
        # weights, codes and scales out
        {"name": "quantise 8192x28672", "op": "quantise", "rows": 8192, "cols": 28672},
        # one tuning step's way back through the quantiser, 4096 x 4096 layer
        {"name": "quantise gradient 4096x4096", "op": "quantise_grad", "rows": 4096, "cols": 4096},
        # one token through a 4096-wide projection: launch latency counts
        {"name": "product 1 token 4096x4096", "op": "product", "tokens": 1, "rows": 4096, "cols": 4096},
        # a small decode batch through the largest layer: bound by the weights' bytes
        {"name": "product 5 tokens 8192x28672", "op": "product", "tokens": 5, "rows": 8192, "cols": 28672},
        # a large decode batch or a short prompt through the same layer
        {"name": "product 256 tokens 8192x28672", "op": "product", "tokens": 256, "rows": 8192, "cols": 28672},
        # a prompt of one calibration sample's length through a gate projection
        {"name": "product 2048 tokens 11008x4096", "op": "product", "tokens": 2048, "rows": 11008, "cols": 4096},
        # a decode batch adds one token to each of its sequences
        {"name": "append 64x1", "op": "append", "seqs": 64, "new": 1, "len": 8191, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": 1},
        # eight prompts fill their pages
        {"name": "append 8x2048", "op": "append", "seqs": 8, "new": 2048, "len": 2048, "q_heads": 32, "kv_heads": 32, "dim": 128,
         "page": 128, "ragged": 0},
        # one user, a short answer so far: the smallest call
        {"name": "attend 1x129", "op": "attend", "seqs": 1, "new": 1, "len": 129, "q_heads": 32, "kv_heads": 32, "dim": 128,
         "page": 16, "ragged": 0},
        # a decode batch with sequences of every length
        {"name": "attend 64 up to 8191", "op": "attend", "seqs": 64, "new": 1, "len": 8191, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": 2},
        # two long documents, one token each: few rows over a long axis
        {"name": "attend 2x131000", "op": "attend", "seqs": 2, "new": 1, "len": 131000, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 128, "ragged": 0},
        # the last pieces of two prompts that were cut into pieces
        {"name": "attend 2x512 of 4000", "op": "attend", "seqs": 2, "new": 512, "len": 4000, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "ragged": 3},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quantise", "quantise_grad", "product", "product", "append", "attend", "attend"))
    if op in ("quantise", "quantise_grad"):
        rows, cols = _log(rng, 1, 8192), BLOCK * _log(rng, 1, 896)
        return {"op": op, "rows": rows if op == "quantise" else min(rows, 4096 * 4096 // cols), "cols": cols}
    if op == "product":
        rows, cols = _log(rng, 8, 11008), BLOCK * _log(rng, 2, 896)
        rows = min(rows, 8192 * 28672 // cols)
        tokens = min(_log(rng, 1, 2048), 2048 * 11008 * 4096 // (rows * cols))
        return {"op": op, "tokens": tokens, "rows": rows, "cols": cols}
    q_heads, kv_heads = rng.choice(HEADS)
    c = {"op": op, "q_heads": q_heads, "kv_heads": kv_heads, "dim": rng.choice((64, 128, 128)), "page": rng.choice((16, 32, 64, 128)),
         "ragged": rng.randrange(1, 1 << 20)}
    seqs = _log(rng, 1, 64)
    if op == "append":
        new = rng.choice((1, 1, _log(rng, 2, 2048)))
        new = max(1, min(new, 8 * 2048 * 96 // (seqs * (q_heads + 2 * kv_heads))))
        most = 64 * 8191 * 8 // (seqs * kv_heads)  # the listed batch's cache
        return {**c, "seqs": seqs, "new": min(new, most), "len": min(new + _log(rng, 1, 8192), most)}
    new = rng.choice((1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 512)))
    most = 64 * 4096 * 8 // (seqs * kv_heads)  # the bytes of the listed batch
    most = min(most, 2 * 512 * 64 * 4000 // (seqs * new * q_heads), 131000)  # the scores of the listed prompt pieces
    new = min(new, max(1, most))
    return {**c, "seqs": seqs, "new": new, "len": max(new, _log(rng, 1, max(2, most)))}


def _lengths(case):
    """New tokens and lengths (these included) of each sequence, by the case alone. Ragged: one sequence has the full length, the others any."""
    s, new, most = case["seqs"], case["new"], case["len"]
    if not case["ragged"]:
        return [new] * s, [most] * s
    r = random.Random(case["ragged"] * 7919 + s)
    news = [new] + [r.randint(max(1, new // 2), new) for _ in range(s - 1)]
    return news, [most] + [r.randint(min(n, most), most) for n in news[1:]]


# ---- plain forms: MXFP4 -------------------------------------------------------


def _pow2(e):
    """2^e in 32 bits for whole e, exactly."""
    return torch.ldexp(torch.ones((), device=e.device, dtype=torch.float64), e.double()).float()


def _mx_scale(w, alpha):
    """The exponent of each block's scale: that of the largest magnitude times alpha, less 2 (4 = 2^2 is the largest power of two of E2M1)."""
    top = w.abs().amax(2).double() * alpha.double()  # the product of 8 and 24 bits is whole here
    return (torch.frexp(top)[1] - 3).clamp(-127, 127).where(top > 0, -127)


def _mx_round(w, v, alpha):
    """Per value: its E2M1 index, sign and place among the borders' inside; per block: the scale and its exponent."""
    w = w.float().view(w.shape[0], -1, BLOCK)
    e = _mx_scale(w, alpha)
    x = _pow2(e).unsqueeze(2)
    t = w.double() / x.double() + v.view_as(w).double()  # next to a border 32 bits would round the wrong way
    t = torch.where(w.abs().amax(2, keepdim=True) > 0, t, 0.0)  # a block of zeros stays one
    m = t.abs()
    # ties go to the value whose mantissa is even: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    i = (m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    return w, e, x, t, i


def _quantise(w, v, alpha):
    n, k = w.shape
    w, e, x, t, i = _mx_round(w, v, alpha)
    grid = torch.tensor(E2M1, device=w.device)
    q = torch.where(t < 0, -grid[i.long()], grid[i.long()])
    return (q * x).bfloat16().view(n, k), (e + 127).byte(), torch.where(t.signbit(), i + 8, i).byte().view(n, k)


def _quantise_grad(g, w, v, alpha):
    n, k = w.shape
    w, e, x, t, i = _mx_round(w, v, alpha)
    grid = torch.tensor(E2M1, device=w.device)
    q = torch.where(t < 0, -grid[i.long()], grid[i.long()])
    live = (w.abs().amax(2) * alpha > 0).unsqueeze(2)
    g = torch.where(live, g.view_as(w), 0.0)
    inside = (t.abs() <= 6.0).float()
    slope = (g * (q - inside * (w / x))).sum(2)
    slope = torch.where(e > -127, slope * (x.squeeze(2) / alpha), 0.0)
    return (g * x * inside).view(n, k), slope


def _mx_values(codes, scales):
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1, BLOCK)
    return (grid[pair.int()] * _pow2(scales.int() - 127).unsqueeze(2)).view(codes.shape[0], -1)


# ---- plain forms: the cache ---------------------------------------------------


def _exponent(top):
    """The smallest e with top <= 448 * 2^e (448 = 1.75 * 2^8 is the largest E4M3 value), within EXP_MIN .. EXP_MAX."""
    f, e = torch.frexp(top)  # top = f * 2^e with f in [0.5, 1)
    e = torch.where(f <= 0.875, e - 9, e - 8)
    return torch.where(top > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)


def _append(s):
    qkv, cu, lens, table, page = s["qkv"], s["cu"].long(), s["lens"].long(), s["table"].long(), s["page"]
    hq, hkv, d = s["hq"], s["hkv"], s["dim"]
    t = torch.arange(s["tokens"], device=qkv.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = lens[seq] - cu[seq + 1] + t
    # the angles of far positions need 64 bits
    turn = at.double().unsqueeze(1) * torch.pow(ROPE_BASE, -torch.arange(0, d, 2, device=t.device, dtype=torch.float64) / d)
    c, n = turn.cos().float().unsqueeze(1), turn.sin().float().unsqueeze(1)
    x = qkv.float().view(s["tokens"], hq + 2 * hkv, d)
    a, b = x[:, : hq + hkv, : d // 2], x[:, : hq + hkv, d // 2 :]
    turned = torch.cat((a * c - b * n, b * c + a * n), 2)
    q_out = turned[:, :hq].bfloat16().reshape(s["tokens"], hq * d)
    where, slot = table[seq, at // page], at % page
    start = lens - (cu[1:] - cu[:-1])  # tokens that were there before
    old_page = table.gather(1, (start // page).clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1).clamp(min=0)
    kept = (start % page > 0) & (cu[1:] > cu[:-1])  # sequences whose first new token shares its page with older ones
    for_old = old_page[kept]
    for part, codes, scales in ((turned[:, hq:], s["k"], s["ks"]), (x[:, hq + hkv :], s["v"], s["vs"])):
        top = torch.zeros(scales.shape, device=t.device)
        top.index_reduce_(0, where, part.abs().amax(2), "amax")
        before = scales.int() - 127
        e = _exponent(top)
        e[for_old] = torch.maximum(e[for_old], before[for_old])
        # older tokens of a page whose scale grew
        was = codes[for_old]
        now = (was.view(torch.float8_e4m3fn).float() * _pow2(before[for_old] - e[for_old])[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        older = torch.arange(page, device=t.device) < (start % page)[kept].unsqueeze(1)
        codes[for_old] = torch.where(older[:, None, :, None], now, was)
        heads = torch.arange(hkv, device=t.device)
        codes[where[:, None], heads, slot[:, None]] = (part * _pow2(-e[where]).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[where] = (e[where] + 127).byte()
    s["q_out"].copy_(q_out)


def _attend(s):
    cu, lens, table, page = s["cu"].long(), s["lens"].long(), s["table"].long(), s["page"]
    hq, hkv, d, most = s["hq"], s["hkv"], s["dim"], s["max_new"]
    n, g = lens.shape[0], hq // hkv
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=lens.device)
    row = (cu[:-1, None] + i).clamp(max=s["tokens"] - 1)
    q = s["q"].float().view(-1, hkv, g, d)[row].permute(0, 2, 3, 1, 4).reshape(n, hkv, g * most, d)

    def pages(codes, scales):
        at = table.clamp(min=0)
        x = codes[at].view(torch.float8_e4m3fn).float() * _pow2(scales.int() - 127)[at][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)

    z = torch.matmul(q, pages(s["k"], s["ks"]).transpose(2, 3)) / math.sqrt(d)
    key = torch.arange(z.shape[3], device=z.device)
    seen = key <= (lens - new)[:, None, None] + i[:, None]  # [sequence, new token, key]
    z = torch.where(seen[:, None, None], z.view(n, hkv, g, most, -1), -torch.inf)
    top = z.amax(4, keepdim=True)
    p = torch.exp(z - torch.where(top > -torch.inf, top, 0.0))
    live = seen.any(1)[:, None, :, None]  # pages past a sequence's end hold anything
    o = torch.matmul(p.view(n, hkv, g * most, -1), torch.where(live, pages(s["v"], s["vs"]), 0.0)).view(n, hkv, g, most, d)
    o = o / p.sum(4, keepdim=True).clamp(min=1e-30)
    seq = torch.searchsorted(cu, torch.arange(s["tokens"], device=cu.device), right=True) - 1
    o = o.permute(0, 3, 1, 2, 4)[seq, torch.arange(s["tokens"], device=cu.device) - cu[seq]]
    s["out"].copy_(o.reshape(s["tokens"], hq * d))


# ---- states -------------------------------------------------------------------


def _weights(n, k, g):
    """Weights of a trained layer's look: small and normal, one in a thousand twenty times as large."""
    w = torch.empty(n, k, device="cuda").normal_(0.0, 0.02, generator=g)
    w[torch.empty(n, k, device="cuda").uniform_(generator=g) < 0.001] *= 20.0
    return w.bfloat16()


def _quantised(n, k, g):
    flat = torch.ones(n, k // BLOCK, device="cuda")
    _, scales, codes = _quantise(_weights(n, k, g), torch.zeros(n, k, device="cuda"), flat)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), scales


def _cache(pages, heads, page, dim, g):
    """Codes and scales of pages that a cache holds: normal values, channels of different size."""
    x = torch.empty(pages, heads, page, dim, device="cuda").normal_(generator=g)
    x *= torch.exp(torch.empty(heads, 1, dim, device="cuda").normal_(generator=g))
    e = _exponent(x.abs().amax((2, 3)))
    x *= _pow2(-e)[..., None, None]
    return x.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).byte()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]
    if op in ("quantise", "quantise_grad"):
        n, k = case["rows"], case["cols"]
        s = {"op": op, "w": _weights(n, k, g), "v": torch.empty(n, k, device="cuda").uniform_(-0.5, 0.5, generator=g),
             "alpha": torch.empty(n, k // BLOCK, device="cuda").uniform_(0.5, 1.0, generator=g)}
        if op == "quantise":
            s["w_hat"] = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
            s["codes"] = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(n, k // BLOCK, dtype=torch.uint8, device="cuda")
            s["scale_values"] = s["scales"].view(torch.float8_e8m0fnu)
        else:
            s["g"] = torch.empty(n, k, device="cuda").normal_(0.0, 1e-6, generator=g)
            s["dv"], s["dalpha"] = torch.empty(n, k, device="cuda"), torch.empty(n, k // BLOCK, device="cuda")
        return s
    if op == "product":
        codes, scales = _quantised(case["rows"], case["cols"], g)
        a = torch.empty(case["tokens"], case["cols"], device="cuda").normal_(generator=g)
        a[:, :: max(1, case["cols"] // 8)] *= 50.0  # a few channels are large
        # the workspace holds the weights in bf16 where the call wants that
        return {"op": op, "a": a.bfloat16(), "codes": codes, "scales": scales,
                "out": torch.empty(case["tokens"], case["rows"], dtype=torch.bfloat16, device="cuda"),
                "workspace": torch.empty(2 * case["rows"] * case["cols"] + 1024, dtype=torch.uint8, device="cuda")}
    news, lens = _lengths(case)
    hq, hkv, d, page, n = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
    per = -(-case["len"] // page)
    k, ks = _cache(n * per, hkv, page, d, g)
    v, vs = _cache(n * per, hkv, page, d, g)
    table = torch.randperm(n * per, device="cuda", generator=g).int().view(n, per)
    used = torch.tensor([-(-x // page) for x in lens], device="cuda")
    table[torch.arange(per, device="cuda") >= used.unsqueeze(1)] = -1
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    s = {"op": op, "k": k, "ks": ks, "v": v, "vs": vs, "table": table, "page": page, "hq": hq, "hkv": hkv, "dim": d, "tokens": cu[-1],
         "max_new": max(news), "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if op == "append":
        s["qkv"] = torch.empty(cu[-1], (hq + 2 * hkv) * d, device="cuda").normal_(0.0, 2.0, generator=g).bfloat16()
        s["q_out"] = torch.empty(cu[-1], hq * d, dtype=torch.bfloat16, device="cuda")
        s["values"] = [x.view(torch.float8_e4m3fn) for x in (k, v)] + [x.view(torch.float8_e8m0fnu) for x in (ks, vs)]
    else:
        s["q"] = torch.empty(cu[-1], hq * d, device="cuda").normal_(generator=g).bfloat16()
        s["out"] = torch.empty(cu[-1], hq * d, dtype=torch.bfloat16, device="cuda")
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    op = s["op"]
    if own:
        import post_weight_quantization_autoround_b200 as ar

        if op == "quantise":
            ar.ar_qdq_mxfp4(s["w"], s["v"], s["alpha"], W_hat=s["w_hat"], codes=s["codes"], scales=s["scales"])
        elif op == "quantise_grad":
            ar.ar_qdq_mxfp4_backward(s["g"], s["w"], s["v"], s["alpha"], s["dv"], s["dalpha"])
        elif op == "product":
            ar.ar_mxfp4_gemm(s["a"], s["codes"], s["scales"], s["out"], s["workspace"])
        elif op == "append":
            ar.ar_kv8_append(s["qkv"], s["cu"], s["lens"], s["table"], s["k"], s["v"], s["ks"], s["vs"], s["q_out"], s["max_new"],
                             rope_base=ROPE_BASE)
        else:
            ar.ar_attention_kv8(s["q"], s["cu"], s["lens"], s["table"], s["k"], s["v"], s["ks"], s["vs"], s["out"], s["max_new"],
                                s["workspace"])
    elif op == "quantise":
        w_hat, scales, codes = _quantise(s["w"], s["v"], s["alpha"])
        s["w_hat"].copy_(w_hat)
        s["scales"].copy_(scales)
        torch.bitwise_or(codes[:, 0::2], codes[:, 1::2] << 4, out=s["codes"])
    elif op == "quantise_grad":
        dv, dalpha = _quantise_grad(s["g"], s["w"], s["v"], s["alpha"])
        s["dv"].copy_(dv)
        s["dalpha"].copy_(dalpha)
    elif op == "product":
        s["out"].copy_(torch.matmul(s["a"].float(), _mx_values(s["codes"], s["scales"]).t()))
    elif op == "append":
        _append(s)
    else:
        _attend(s)
    if op == "quantise":
        return s["w_hat"], s["scale_values"]  # the fake-quantised weights are the values that the codes stand for
    if op == "quantise_grad":
        return s["dv"], s["dalpha"]
    if op == "append":
        return [s["q_out"]] + s["values"]
    return s["out"]


def work(case):
    op = case["op"]
    if op in ("quantise", "quantise_grad"):
        n = case["rows"] * case["cols"]
        if op == "quantise":  # weight, offset, clip factor in; fake-quantised weight, code, scale out
            return {"bytes": n * (2 + 4 + 2 + 0.5) + n / BLOCK * 5, "flops": 8 * n}
        return {"bytes": n * (4 + 2 + 4 + 4) + n / BLOCK * 8, "flops": 10 * n}
    if op == "product":
        t, n, k = case["tokens"], case["rows"], case["cols"]
        return {"bytes": n * k * (0.5 + 1 / BLOCK) + 2 * t * k + 2 * t * n, "flops": 2 * t * n * k}
    news, lens = _lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if op == "append":
        return {"bytes": sum(news) * d * (2 * (hq + 2 * hkv) + 2 * hq + 2 * hkv), "flops": sum(news) * d * (3 * (hq + hkv) + 4 * hkv)}
    pairs = sum(n * x - n * (n - 1) // 2 for n, x in zip(news, lens))
    return {"bytes": 2 * sum(lens) * hkv * d + 4 * sum(news) * hq * d, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """From the definitions, in 64 bits."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float8_e4m3fn

    def p2(e):
        return ((e.long() + 1023) << 52).view(torch.float64)  # a power function is off by a last bit, which ties would feel

    def floor_log2(x):
        """The largest whole f with 2^f <= x, whatever the logarithm's last bit."""
        f = torch.floor(torch.log2(x))
        f = f + (p2(f + 1) <= x)
        return f - (p2(f) > x).double()

    def e2m1(t):
        """Nearest of the E2M1 values: a multiple of 0.5 below 2, of 1 below 4, of 2 below 6, ties to the even multiple."""
        m = t.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        return torch.sign(t) * torch.clamp(torch.round(m / step) * step, max=6.0)

    def e4m3(x):
        step = p2(floor_log2(x.abs().clamp(min=2.0**-60)).clamp(min=-6) - 3)
        return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)

    if op in ("quantise", "quantise_grad"):
        n, k = s["w"].shape
        w, v, alpha = s["w"].double().view(n, -1, BLOCK), s["v"].double().view(n, -1, BLOCK), s["alpha"].double()
        x = p2(floor_log2((w.abs().amax(2) * alpha).clamp(min=2.0**-125)) - 2).unsqueeze(2)
        t = torch.where(w.abs().amax(2, keepdim=True) > 0, w / x + v, 0.0)
        if op == "quantise":
            return (e2m1(t) * x).view(n, k), x.squeeze(2)
        inside = t.abs() <= 6
        g = s["g"].double().view_as(w)
        return (g * x * inside).view(n, k), (g * (e2m1(t) - torch.where(inside, w / x, 0.0))).sum(2) * x.squeeze(2) / alpha
    if op == "product":
        n, k = case["rows"], case["cols"]
        code = torch.empty(n, k, dtype=torch.uint8, device="cuda")
        code[:, 0::2], code[:, 1::2] = s["codes"] % 16, s["codes"] // 16
        e, m = (code // 2 % 4).double(), (code % 2).double()
        w = torch.where(e > 0, (1 + m / 2) * p2(e - 1), m / 2) * torch.where(code > 7, -1.0, 1.0).double()
        w = w.view(n, -1, BLOCK) * p2(s["scales"].double() - 127).unsqueeze(2)
        return s["a"].double() @ w.view(n, k).t()

    news, lens = _lengths(case)
    hq, hkv, d, page = s["hq"], s["hkv"], s["dim"], s["page"]
    cu, table = s["cu"].tolist(), s["table"].long()
    if op == "append":
        values = [x.view(f8).double() for x in (s["k"], s["v"])]
        scales = [p2(x.double() - 127) for x in (s["ks"], s["vs"])]
        q_out = []
        for j, (new, total) in enumerate(zip(news, lens)):
            x = s["qkv"][cu[j] : cu[j + 1]].double().view(new, -1, d)
            at = torch.arange(total - new, total, device="cuda")
            z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                            at.double()[:, None] * ROPE_BASE ** (-2.0 * torch.arange(d // 2, device="cuda").double() / d))
            z = torch.complex(x[:, : hq + hkv, : d // 2], x[:, : hq + hkv, d // 2 :]) * z[:, None]
            turned = torch.cat((z.real, z.imag), 2)
            q_out.append(turned[:, :hq].reshape(new, hq * d))
            first = (total - new) // page
            span = (total - 1) // page + 1 - first
            for part, value, scale in ((turned[:, hq:], values[0], scales[0]), (x[:, hq + hkv :], values[1], scales[1])):
                there = table[j, first : first + span]
                old = (total - new) % page
                rows = torch.zeros(span * page, hkv, d, dtype=torch.float64, device="cuda")
                rows[old : old + new] = part
                rows = rows.view(span, page, hkv, d).transpose(1, 2)
                top = (rows.abs().amax((2, 3)) / 448).clamp(min=2.0**EXP_MIN)
                need = p2((floor_log2(top) + (p2(floor_log2(top)) < top)).clamp(max=EXP_MAX))
                if old:
                    need[0] = torch.maximum(need[0], scale[there[0]])
                    rows[0, :, :old] = value[there[0], :, :old] * scale[there[0]][:, None, None]
                got = value[there].clone()
                fill = torch.zeros(span * page, dtype=torch.bool, device="cuda")
                fill[: old + new] = True
                value[there] = torch.where(fill.view(span, 1, page, 1), e4m3(rows / need[..., None, None]), got)
                scale[there] = need
        return [torch.cat(q_out)] + values + scales
    out = []
    for j, (new, total) in enumerate(zip(news, lens)):
        there = table[j, : -(-total // page)]
        key, value = ((c[there].view(f8).double() * p2(e[there].double() - 127)[..., None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, :total]
                      for c, e in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        q = s["q"][cu[j] : cu[j + 1]].double().view(new, hkv, -1, d).permute(1, 2, 0, 3)
        z = q @ key.transpose(1, 2).unsqueeze(1) * d**-0.5
        late = torch.ones(new, total, dtype=torch.bool, device="cuda").triu(total - new + 1)
        o = torch.softmax(z.masked_fill(late, -torch.inf), 3) @ value.unsqueeze(1)
        out.append(o.permute(2, 0, 1, 3).reshape(new, hq * d))
    return torch.cat(out)
