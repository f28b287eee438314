"""Pins of the low-bit oracle (CPU): code values against torch's casts, hand-placed cases, finite differences."""
import numpy as np
import pytest
import torch

from oracle import lowbit_oracle as L


def test_code_values_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    got = L.e4m3_values(codes.numpy())
    assert np.array_equal(np.nan_to_num(ref, nan=9e9), np.nan_to_num(got, nan=9e9))


def test_e4m3_rounding_matches_torch_cast():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 8, 4000), L.E4M3, (L.E4M3[1:] + L.E4M3[:-1]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(L.e4m3_codes(x), ref)


@pytest.mark.parametrize("x,want", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0),
                                    (5.01, 6.0), (100.0, 6.0), (-0.75, -1.0), (0.2500001, 0.5)])
def test_e2m1_ties_go_to_even(x, want):
    code, neg = L.nearest_code(np.array([x]), L.E2M1)
    assert (-1.0 if neg[0] else 1.0) * L.E2M1[code[0]] == want


def test_mxfp4_by_hand():
    W = np.zeros((1, 64))
    W[0, 0], W[0, 1], W[0, 2] = 7.0, -3.4, 0.3  # largest 7: X = 2^(2-2) = 1; 7 saturates at 6
    r = L.mxfp4_qdq(W)
    assert list(r["scales"][0]) == [127, 0]
    assert list(r["W_hat"][0, :3]) == [6.0, -3.0, 0.5]
    assert not r["W_hat"][0, 32:].any() and not r["codes"][0, 32:].any()
    r = L.mxfp4_qdq(W, alpha=np.array([[0.5, 1.0]]))  # 3.5: X = 2^-1
    assert r["scales"][0, 0] == 126 and r["W_hat"][0, 1] == -3.0 and r["W_hat"][0, 2] == 0.25
    packed = L.pack_fp4(r["codes"])
    assert np.array_equal(L.mxfp4_values(packed, r["scales"]), r["W_hat"])


def test_mxfp4_values_on_the_grid_come_back():
    rng = np.random.default_rng(1)
    e = rng.integers(-20, 20, (5, 3))
    W = (rng.choice(np.concatenate([L.E2M1, -L.E2M1]), (5, 3, 32)))
    W[..., 0] = 6.0
    W = (W * np.ldexp(1.0, e)[..., None]).reshape(5, 96)
    assert np.array_equal(L.mxfp4_qdq(W)["W_hat"], W)


def test_mxfp4_gradient_is_that_of_the_surrogate():
    """With both roundings as the identity W_hat = X clamp(W / X + V, -6, 6) + (q - t) X held in the codes; by the rule
    dW_hat/dalpha = (q - m W/X) X / alpha.  Differences of s(alpha) (q_fixed + m (W/s - W/X)) about alpha check it, with
    s(alpha) = X alpha / alpha_0 the scale whose exponent is not rounded."""
    rng = np.random.default_rng(2)
    W, V = rng.normal(size=(3, 64)), rng.uniform(-0.5, 0.5, (3, 64))
    a = rng.uniform(0.5, 1.0, (3, 2))
    g = rng.normal(size=(3, 64))
    dV, da, _ = L.mxfp4_backward(g, W, V, a)
    r = L.mxfp4_qdq(W, V, a)
    m = np.abs(r["t"]) <= 6

    def loss(alpha, vv):
        s = (r["X"] * alpha / a)[..., None]
        return (g.reshape(r["w"].shape) * s * (r["q"] + m * (r["w"] / s - r["w"] / r["X"][..., None]) + m * (vv - r["v0"]))).sum()

    r["v0"] = V.reshape(r["w"].shape)
    h = 1e-6
    for i, j in [(0, 0), (1, 1), (2, 0)]:
        d = np.zeros_like(a)
        d[i, j] = h
        assert (loss(a + d, r["v0"]) - loss(a - d, r["v0"])) / (2 * h) == pytest.approx(da[i, j], rel=1e-6, abs=1e-9)
    for i, j in [(0, 5), (1, 40), (2, 63)]:
        d = np.zeros_like(V)
        d[i, j] = h
        vv = d.reshape(r["w"].shape)
        assert (loss(a, r["v0"] + vv) - loss(a, r["v0"] - vv)) / (2 * h) == pytest.approx(dV[i, j], rel=1e-6, abs=1e-9)
    assert not m.all() and m.any()


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.1, 1), (224.0, -1), (7.0, -6), (7.01, -5), (0.0, -100), (3e38, 120)])
def test_cache_exponent(top, e):
    assert L.exponent_for(top) == e


def test_append_then_read_returns_the_rotated_keys():
    """Two appends to one sequence: what the cache holds is the rotated input within E4M3's half step, also for tokens
    whose page's scale grew afterwards."""
    rng = np.random.default_rng(3)
    d, page, n_kv, n_heads = 64, 16, 2, 4
    k, v = (np.zeros((3, n_kv, page, d), np.uint8) for _ in range(2))
    ks, vs = (np.zeros((3, n_kv), np.uint8) for _ in range(2))
    table = [[2, 0]]
    a, b = rng.normal(size=(5, (n_heads + 2 * n_kv) * d)), 100 * rng.normal(size=(13, (n_heads + 2 * n_kv) * d))
    L.kv8_append(a, [0, 5], [5], table, k, v, ks, vs, n_heads)
    first = ks[2].copy()
    q, _ = L.kv8_append(b, [0, 13], [18], table, k, v, ks, vs, n_heads)
    assert (ks[2] > first).all()
    x = np.concatenate([a, b]).reshape(18, -1, d)
    for t in range(18):
        want = L.rotate(x[t, n_heads:n_heads + n_kv], t, 10000.0)
        got = L.e4m3_values(k[table[0][t // page], :, t % page]) * np.ldexp(1.0, ks[table[0][t // page]].astype(int) - 127)[:, None]
        step = np.ldexp(1.0, ks[table[0][t // page]].astype(int) - 127)[:, None] * 2.0 ** -10
        # one rounding (2^-4) and, for re-coded tokens, one more that only subnormal codes feel
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * 1.07 + 2 * step).all()
    assert np.allclose(q[12], L.rotate(x[17, :n_heads], 17, 10000.0))


def test_attention_against_a_direct_sum():
    rng = np.random.default_rng(4)
    d, page, n_kv, n_heads, Ln = 64, 16, 1, 2, 21
    k, v = (L.e4m3_codes(rng.normal(size=(2, n_kv, page, d))) for _ in range(2))
    ks, vs = (rng.integers(125, 130, (2, n_kv)).astype(np.uint8) for _ in range(2))
    q = rng.normal(size=(2, n_heads * d))
    out, lse, *_ = L.kv8_attention(q, [0, 2], [Ln], [[1, 0]], k, v, ks, vs, n_heads)
    kk = np.concatenate([L.e4m3_values(k[p, 0]) * 2.0 ** (int(ks[p, 0]) - 127) for p in (1, 0)])
    vv = np.concatenate([L.e4m3_values(v[p, 0]) * 2.0 ** (int(vs[p, 0]) - 127) for p in (1, 0)])
    for i in range(2):
        for h in range(n_heads):
            e = np.exp([q[i].reshape(n_heads, d)[h] @ kk[j] / 8 for j in range(Ln - 1 + i)])
            assert np.allclose(out[i, h], (e[:, None] * vv[:Ln - 1 + i]).sum(0) / e.sum())
            assert lse[i, h] == pytest.approx(np.log(e.sum()))
