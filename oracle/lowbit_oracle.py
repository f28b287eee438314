"""Plain numpy oracle of the MXFP4 format and of the paged 8-bit cache, in 64 bits, from the definitions in
include/autoround.h.  Test infrastructure: the product path never imports it.

Rounding goes by brute force over the code values (distance, then the even code), not by bit tricks.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
#: the 127 finite non-negative E4M3 values, by code
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])
BLOCK = 32
EXP_MIN, EXP_MAX = -100, 120


def nearest_code(x, grid):
    """Code of the grid value nearest to |x| (ties to the even code, saturating) and the sign bit."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return code, np.signbit(x)


def floor_log2(x: float) -> int:
    return math.frexp(x)[1] - 1


# ---- MXFP4 --------------------------------------------------------------------

def exact_side(a, b):
    """a + b in 64 bits; where that sum is itself rounded (an offset far below the value), the neighbour on the exact
    sum's side, so that comparisons with borders come out as for the exact sum."""
    s = a + b
    bb = s - a
    err = (a - (s - bb)) + (b - bb)  # what the rounding lost, exactly
    return np.where(err > 0, np.nextafter(s, np.inf), np.where(err < 0, np.nextafter(s, -np.inf), s))


def mxfp4_qdq(W, V=None, alpha=None):
    """W [N][K] (values of bf16), V [N][K], alpha [N][K/32]: codes [N][K] (sign << 3 | index), scale codes, W_hat,
    and the pieces the gradient needs."""
    W = np.asarray(W, np.float64)
    N, K = W.shape
    nb = K // BLOCK
    w = W.reshape(N, nb, BLOCK)
    v = np.zeros_like(w) if V is None else np.asarray(V, np.float64).reshape(w.shape)
    a = np.ones((N, nb)) if alpha is None else np.asarray(alpha, np.float64)
    amax = np.abs(w).max(2)
    top = amax * a
    e = np.array([max(floor_log2(t) - 2, -127) if t > 0 else -127 for t in top.ravel()]).reshape(N, nb)
    X = np.ldexp(1.0, e)[..., None]
    t = exact_side(w / X, v)
    t = np.where((amax > 0)[..., None], t, 0.0)
    code, neg = nearest_code(t, E2M1)
    q = np.where(neg, -E2M1[code], E2M1[code])
    return {"codes": (code | (neg << 3)).reshape(N, K).astype(np.uint8), "scales": (e + 127).astype(np.uint8),
            "W_hat": (q * X).reshape(N, K), "q": q, "t": t, "X": X[..., 0], "w": w, "a": a, "live": (amax > 0) & (a > 0)}


def mxfp4_backward(dW, W, V=None, alpha=None):
    """dV [N][K], dalpha [N][K/32] and, per block, the sum of the magnitudes that dalpha adds (for tolerances)."""
    r = mxfp4_qdq(W, V, alpha)
    g = np.where(r["live"][..., None], np.asarray(dW, np.float64).reshape(r["w"].shape), 0.0)
    m = np.abs(r["t"]) <= 6.0
    terms = g * (r["q"] - np.where(m, r["w"] / r["X"][..., None], 0.0))
    slope = np.where((r["scales"] > 0) & r["live"], r["X"] / np.where(r["a"] > 0, r["a"], 1.0), 0.0)
    N = r["w"].shape[0]
    return (g * r["X"][..., None] * m).reshape(N, -1), terms.sum(2) * slope, np.abs(terms).sum(2) * slope


def pack_fp4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def mxfp4_values(packed, scales):
    codes = np.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return (v.reshape(packed.shape[0], -1, BLOCK) * np.ldexp(1.0, scales.astype(int) - 127)[..., None]).reshape(v.shape)


# ---- the paged cache ----------------------------------------------------------

def exponent_for(top: float) -> int:
    """The smallest e with top <= 448 * 2^e, within the scale's range."""
    if top <= 0:
        return EXP_MIN
    e = floor_log2(top / 448.0)
    if top > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e, EXP_MIN), EXP_MAX)


def e4m3_codes(x):
    code, neg = nearest_code(x, E4M3)
    return (code | (neg << 7)).astype(np.uint8)


def e4m3_values(codes):
    """NaN codes come out as NaN."""
    v = np.append(E4M3, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def rotate(x, pos, base):
    """x [..., d] at position pos."""
    d = x.shape[-1]
    ang = pos * base ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def kv8_append(qkv, cu, lens, table, k, v, ks, vs, n_heads, base=10000.0):
    """Changes k, v, ks, vs in place as the library does; returns the rotated queries and, for every new key, its exact
    value with its page, head and place (the codes of values whose rotation rounds near a border may differ)."""
    _, n_kv, page, d = k.shape
    x = np.asarray(qkv, np.float64).reshape(qkv.shape[0], n_heads + 2 * n_kv, d)
    q_out = np.zeros((qkv.shape[0], n_heads, d))
    keys = []
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        start = lens[s] - n
        rows = x[cu[s]:cu[s + 1]].copy()
        for i in range(n):
            rows[i, :n_heads + n_kv] = rotate(rows[i, :n_heads + n_kv], start + i, base)
        q_out[cu[s]:cu[s + 1]] = rows[:, :n_heads]
        for pi in range(start // page, -(-lens[s] // page) if n else start // page):
            ph = table[s][pi]
            lo, hi = max(start, pi * page), min(lens[s], (pi + 1) * page)
            for h in range(n_kv):
                for part, pages, scales in ((0, k, ks), (1, v, vs)):
                    new = rows[lo - start:hi - start, n_heads + part * n_kv + h]
                    e = exponent_for(np.abs(new).max())
                    old = lo - pi * page
                    if old:
                        before = min(max(int(scales[ph, h]) - 127, EXP_MIN), EXP_MAX)
                        e = max(e, before)
                        if e > before:
                            pages[ph, h, :old] = e4m3_codes(e4m3_values(pages[ph, h, :old]) * 2.0 ** (before - e))
                    pages[ph, h, old:old + hi - lo] = e4m3_codes(new * 2.0 ** -e)
                    scales[ph, h] = e + 127
                    if part == 0:
                        keys.append((ph, h, old, new))
    return q_out, keys


def kv8_attention(q, cu, lens, table, k, v, ks, vs, n_heads, scale=None):
    """out [T][n_heads][d], lse [T][n_heads] and two magnitudes for tolerances: sum_j p_j |v_j|, and the sum over keys of
    the value codes' magnitudes in units of the largest term 2^(z log2 e + e_v), over the row sum."""
    _, n_kv, page, d = k.shape
    scale = d ** -0.5 if scale is None else scale
    T, group = q.shape[0], n_heads // n_kv
    q = np.asarray(q, np.float64).reshape(T, n_heads, d)
    out, lse = np.zeros((T, n_heads, d)), np.full((T, n_heads), -np.inf)
    mag, units = np.zeros((T, n_heads, d)), np.zeros((T, n_heads, d))
    zmag = np.zeros((T, n_heads))
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        L = lens[s]
        if n == 0 or L <= 0:
            continue
        pg = np.array([table[s][j // page] for j in range(L)])
        at = np.arange(L) % page
        for h in range(n_kv):
            kk = e4m3_values(k[pg, h, at]) * np.ldexp(1.0, ks[pg, h].astype(int) - 127)[:, None]
            vc = e4m3_values(v[pg, h, at])
            ev = vs[pg, h].astype(int) - 127
            for i in range(n):
                seen = L - n + i + 1
                if seen <= 0:
                    continue
                row = q[cu[s] + i, h * group:(h + 1) * group]
                z = row @ kk[:seen].T * scale
                top = z.max(1, keepdims=True)
                p = np.exp(z - top)
                tot = p.sum(1, keepdims=True)
                vv = vc[:seen] * np.ldexp(1.0, ev[:seen])[:, None]
                sl = (cu[s] + i, slice(h * group, (h + 1) * group))
                out[sl] = p @ vv / tot
                lse[sl] = (top + np.log(tot))[:, 0]
                mag[sl] = p @ np.abs(vv) / tot
                zmag[sl] = (np.abs(row) @ np.abs(kk[:seen]).T).max(1) * scale
                largest = (z / math.log(2) + ev[:seen]).max(1, keepdims=True)
                units[sl] = np.abs(vc[:seen]).sum(0)[None] * 2.0 ** (largest - top / math.log(2)) / tot
    return out, lse, mag, units, zmag
