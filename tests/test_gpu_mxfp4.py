"""MXFP4 on the GPU against the 64-bit oracle.

Codes, scales, W_hat and dV are exact on both sides (W / X and dW X are exact in fp32, the rounding decisions are
taken on exact sums), so they are compared bit for bit.  dalpha is a sum of 32 fp32 terms: each takes one rounding
of q - W/X and one of the fused multiply-add, a lane adds 8 in a row, two more additions join the lanes, the slope
takes one division and one product, so at most 14 roundings of 2^-24 apply to the sum of the terms' magnitudes.
The product: the weights are exact, the sums run in fp32 over K / 16 tensor-core steps (an accumulation error of at
most 2^-22 of the magnitudes' sum a step covers truncating adders, 32 more the joins), the output rounds to bf16
(half a step, 2^-8 relative)."""
import numpy as np
import pytest
import torch

import synth
from oracle import lowbit_oracle as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_autoround_b200 as m
    return m


def _inputs(N, K, seed, spread=0):
    """bf16 weights (as float32 values) with outliers, offsets, clip factors; spread: block scales over 2^+-spread."""
    rng = np.random.default_rng(seed)
    W = rng.normal(0, 0.02, (N, K)).astype(np.float32)
    W[rng.random((N, K)) < 0.01] *= 20
    if spread:
        W *= np.repeat(2.0 ** rng.integers(-spread, spread + 1, (N, K // 32)), 32, 1).astype(np.float32)
    W = torch.from_numpy(W).bfloat16()
    return W, rng.uniform(-0.5, 0.5, (N, K)).astype(np.float32), rng.uniform(0.5, 1.0, (N, K // 32)).astype(np.float32)


def _qdq(ar, W, V, a):
    N, K = W.shape
    Wd = W.cuda()
    Vd, ad = (None if x is None else torch.from_numpy(x).cuda() for x in (V, a))
    W_hat = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device="cuda")
    ar.ar_qdq_mxfp4(Wd, Vd, ad, W_hat, codes, scales)
    return W_hat, codes, scales


@pytest.mark.parametrize("N,K,with_v,with_a,spread", [(1, 32, True, True, 0), (37, 64, True, True, 3), (1000, 288, True, False, 30),
                                                      (64, 4096, False, False, 0), (3, 32, False, True, 0), (129, 1056, True, True, 100)])
def test_qdq_bit_exact(ar, N, K, with_v, with_a, spread):
    W, V, a = _inputs(N, K, N + K, spread)
    V, a = V if with_v else None, a if with_a else None
    W_hat, codes, scales = _qdq(ar, W, V, a)
    ref = L.mxfp4_qdq(W.double().numpy(), V, a)
    assert np.array_equal(scales.cpu().numpy(), ref["scales"])
    assert np.array_equal(codes.cpu().numpy(), L.pack_fp4(ref["codes"]))
    assert np.array_equal(W_hat.double().cpu().numpy(), ref["W_hat"])
    assert ar.ar_get_device_status() == ar.AR_OK and "qdq_mxfp4_kernel" in ar.ar_last_kernels()


def test_qdq_borders_and_zero_blocks(ar):
    """Sums that lie on or a last bit beside a border, where a rounded sum decides wrongly; blocks of zeros (also negative
    ones) with offsets; blocks whose scale is held at 2^-127."""
    rng = np.random.default_rng(5)
    W = np.zeros((8, 64), np.float32)
    W[:4, 0] = 4.0  # X = 1
    W[:4, 32] = 4.0
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    w = torch.from_numpy(rng.choice(np.array([0.5, 1.0, 1.5, 2.0, 3.0, 3.5, -2.0], np.float32), (4, 31)))
    W[:4, 1:32] = w
    W[4, :] = 0.0
    W[5, :] = -0.0
    W[6, :] = 2.0 ** -126 * rng.integers(-3, 4, 64)
    W[7, :32] = 3e38
    V = rng.uniform(-0.5, 0.5, (8, 64)).astype(np.float32)
    near = np.abs(borders[:, None, None] - W[None, :4, 1:32]).argmin(0)
    V[:4, 1:32] = borders[near] - W[:4, 1:32]
    V[0, 1:32] = np.nextafter(V[0, 1:32], np.float32(9))
    V[1, 1:32] = np.nextafter(V[1, 1:32], np.float32(-9))
    Wb = torch.from_numpy(W).bfloat16()
    W_hat, codes, scales = _qdq(ar, Wb, V, None)
    ref = L.mxfp4_qdq(Wb.double().numpy(), V, None)
    assert np.array_equal(scales.cpu().numpy(), ref["scales"])
    assert np.array_equal(codes.cpu().numpy(), L.pack_fp4(ref["codes"]))
    assert np.array_equal(W_hat.double().cpu().numpy(), ref["W_hat"])
    assert not codes[4:6].any() and not scales[4:6].any()


def test_qdq_scale_of_a_product_just_below_a_power_of_two(ar):
    """alpha * max rounds up to 4 in fp32; the exact product is below, so the exponent is one less."""
    W = np.zeros((1, 32), np.float32)
    W[0, 0] = 4.0625
    a = np.array([[np.nextafter(np.float32(4.0 / 4.0625), np.float32(0))]], np.float32)
    while np.float64(a[0, 0]) * 4.0625 >= 4.0:
        a = np.nextafter(a, np.float32(0))
    _, _, scales = _qdq(ar, torch.from_numpy(W).bfloat16(), None, a)
    assert scales.item() == L.mxfp4_qdq(W.astype(np.float64), None, a)["scales"][0, 0] == 127 + 1 - 2


def test_qdq_non_finite(ar):
    W, V, a = _inputs(4, 96, 3)
    W[0, 5], W[1, 40] = float("nan"), float("inf")
    W_hat, codes, scales = _qdq(ar, W, V, a)
    assert ar.ar_get_device_status() == ar.AR_ERR_NONFINITE
    assert scales[0, 0] == 255 and scales[1, 1] == 255 and (scales == 255).sum() == 2
    assert W_hat[0, :32].isnan().all() and W_hat[1, 32:64].isnan().all() and W_hat.isnan().sum() == 64
    assert not codes[0, :16].any()
    V[3, 3] = np.nan
    _qdq(ar, W[2:], V[2:], a[2:])
    assert ar.ar_get_device_status() == ar.AR_ERR_NONFINITE


@pytest.mark.parametrize("N,K,with_v,with_a", [(1, 32, True, True), (37, 96, True, True), (300, 1056, False, True), (64, 256, True, False)])
def test_backward(ar, N, K, with_v, with_a):
    W, V, a = _inputs(N, K, 7 * N + K)
    W[0, :32] = 0  # a block without a gradient
    V, a = V if with_v else None, a if with_a else None
    g = np.random.default_rng(K).normal(0, 1e-3, (N, K)).astype(np.float32)
    dV = torch.empty(N, K, device="cuda")
    da = torch.empty(N, K // 32, device="cuda")
    Vd, ad = (None if x is None else torch.from_numpy(x).cuda() for x in (V, a))
    ar.ar_qdq_mxfp4_backward(torch.from_numpy(g).cuda(), W.cuda(), Vd, ad, dV, da)
    rv, ra, mag = L.mxfp4_backward(g, W.double().numpy(), V, a)
    assert np.array_equal(dV.double().cpu().numpy(), rv)
    assert (np.abs(da.double().cpu().numpy() - ra) <= 14 * 2.0 ** -24 * mag).all()
    assert not da[0, 0] and not dV[0, :32].any()
    again = torch.empty_like(da)
    ar.ar_qdq_mxfp4_backward(torch.from_numpy(g).cuda(), W.cuda(), Vd, ad, None, again)
    assert torch.equal(da, again)
    assert ar.ar_get_device_status() == ar.AR_OK


def _product(ar, A, codes, scales, workspace=False):
    T, N, K = A.shape[0], codes.shape[0], A.shape[1]
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ar.ar_mxfp4_gemm_workspace(T, N, K), dtype=torch.uint8, device="cuda") if workspace else None
    ar.ar_mxfp4_gemm(A, codes, scales, out, ws)
    return out


def _check_product(out, A, codes, scales):
    w = torch.from_numpy(L.mxfp4_values(codes.cpu().numpy(), scales.cpu().numpy())).cuda()
    a = A.double()
    ref, mag = a @ w.t(), a.abs() @ w.abs().t()
    tol = 2.0 ** -8 * ref.abs() + (A.shape[1] / 16 + 32) * 2.0 ** -22 * mag
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), out[bad][:4], ref[bad][:4])


def _packed(ar, N, K, seed, spread=4):
    W, V, a = _inputs(N, K, seed, spread)
    _, codes, scales = _qdq(ar, W, V, a)
    return codes, scales


def _acts(T, K, seed):
    A = np.random.default_rng(seed).normal(size=(T, K)).astype(np.float32)
    A[:, ::max(1, K // 8)] *= 50
    return torch.from_numpy(A).bfloat16().cuda()


@pytest.mark.parametrize("N,K", [(1, 32), (8, 64), (129, 96), (300, 256), (264, 1056), (1000, 4096), (40, 8224), (2400, 512)])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 17, 64, 130])
def test_product(ar, N, K, T):
    codes, scales = _packed(ar, N, K, N + K)
    A = _acts(T, K, T)
    _check_product(_product(ar, A, codes, scales), A, codes, scales)
    assert ar.ar_get_device_status() == ar.AR_OK


@pytest.mark.parametrize("T,N,K", [(2048, 264, 96), (2100, 256, 1056), (2048, 129, 256), (2051, 1024, 512), (2048, 64, 8224)])
def test_product_with_workspace(ar, T, N, K):
    codes, scales = _packed(ar, N, K, N + K)
    A = _acts(T, K, T)
    out = _product(ar, A, codes, scales, workspace=True)
    assert ("expand_mxfp4_kernel" in ar.ar_last_kernels()) == (N % 8 == 0 and K <= 8192)
    _check_product(out, A, codes, scales)
    _check_product(_product(ar, A, codes, scales), A, codes, scales)


@pytest.mark.parametrize("T", [1, 8, 40])
def test_product_far_scales_and_nan_rows(ar, T):
    """Scales over the whole range that fp32 sums hold, and a row whose scale is NaN."""
    rng = np.random.default_rng(T)
    N, K = 48, 256
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(40, 214, (N, 1), dtype=np.uint8) + rng.integers(0, 3, (N, K // 32), dtype=np.uint8)).cuda()
    A = _acts(T, K, 3)
    _check_product(_product(ar, A, codes, scales), A, codes, scales)
    scales[5, 2] = 255
    out = _product(ar, A, codes, scales)
    assert out[:, 5].isnan().all() and not out[:, :5].isnan().any() and not out[:, 6:].isnan().any()


@pytest.mark.parametrize("T", [1, 2, 6, 200])
def test_product_activation_range(ar, T):
    """Tokens whose activations differ by 2^200, and whose own values span far more than fp16's range."""
    N, K = 64, 512
    codes, scales = _packed(ar, N, K, 9, spread=0)
    A = _acts(T, K, 11).double()
    A *= torch.exp2(torch.arange(T, device="cuda").double().mul(37).remainder(160) - 80)[:, None]
    A[:, 1::2] *= 2.0 ** -12
    A = A.bfloat16()
    _check_product(_product(ar, A, codes, scales), A, codes, scales)


def test_product_on_another_stream_and_in_a_graph(ar):
    codes, scales = _packed(ar, 640, 1024, 1)
    A = _acts(4, 1024, 2)
    want = _product(ar, A, codes, scales)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = _product(ar, A, codes, scales)
    st.synchronize()
    assert torch.equal(want, got)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ar.ar_mxfp4_gemm(A, codes, scales, out)
    A.copy_(_acts(4, 1024, 3))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _product(ar, A, codes, scales))


@pytest.mark.parametrize("N,K,M", [(64, 96, 40), (136, 512, 200)])
def test_tune_step(ar, N, K, M):
    """One step: its gradients are the backward of its own G^T X, its update follows their signs exactly, the loss is the
    forward's (2^-7: fp32 sums of bf16 products against 64 bits, and G's bf16 rounding does not enter it)."""
    W, V, a = _inputs(N, K, N)
    Wd, Vd, ad = W.cuda(), torch.from_numpy(V).cuda(), torch.from_numpy(a).cuda()
    X = _acts(M, K, 4)
    Y = torch.empty(M, N, device="cuda")
    ar.ar_linear_forward(X, Wd, Y)
    cfg = ar.ar_qconfig_default()
    loss = torch.empty(1, device="cuda")
    dV, da = torch.empty(N, K, device="cuda"), torch.empty(N, K // 32, device="cuda")
    ws = torch.empty(ar.ar_tune_step_mxfp4_workspace(M, N, K, 1), dtype=torch.uint8, device="cuda")
    V0, a0 = Vd.clone(), ad.clone()
    ar.ar_tune_step_mxfp4(Wd, Vd, ad, X, Y, cfg, 1, loss, ws, dV, da)
    ref = L.mxfp4_qdq(W.double().numpy(), V, a)
    R = X.double() @ torch.from_numpy(ref["W_hat"]).cuda().t() - X.double() @ Wd.double().t()
    assert loss.item() == pytest.approx((R * R).mean().item(), rel=2.0 ** -7)
    # G is bf16 (2^-8 relative an element): the gradients agree with the exact ones to that in norm
    rv, ra, _ = L.mxfp4_backward((2 * R / (M * N)).t().cpu().numpy() @ X.double().cpu().numpy(), W.double().numpy(), V, a)
    for got, want in ((dV, rv), (da, ra)):
        assert np.linalg.norm(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.linalg.norm(want)
    lr = np.float32(cfg.lr)
    assert torch.equal(Vd, (V0 - lr * torch.sign(dV)).clamp(-0.5, 0.5))
    assert torch.equal(ad, (a0 - lr * torch.sign(da)).clamp(0.5, 1.0))
    # n steps in one call are n calls
    for _ in range(2):
        ar.ar_tune_step_mxfp4(Wd, Vd, ad, X, Y, cfg, 1, loss, ws)
    ws3 = torch.empty(ar.ar_tune_step_mxfp4_workspace(M, N, K, 3), dtype=torch.uint8, device="cuda")
    losses = torch.empty(3, device="cuda")
    ar.ar_tune_step_mxfp4(Wd, V0, a0, X, Y, cfg, 3, losses, ws3)
    assert torch.equal(V0, Vd) and torch.equal(a0, ad) and losses[2] == loss[0]
    before = Vd.clone()
    ar.ar_tune_step_mxfp4(Wd, Vd, ad, X, Y, cfg, 0, loss, ws)
    assert torch.equal(before, Vd)
    assert ar.ar_get_device_status() == ar.AR_OK


def test_full_size_rows(ar):
    """64 sampled rows of the 8192 x 28672 layer, quantized and multiplied."""
    d = synth.make_linear(64, 28672, 1, seed=3)
    W = torch.from_numpy(d["W"].view(np.int16)).view(torch.bfloat16).cuda().repeat(128, 1)
    codes = torch.empty(8192, 14336, dtype=torch.uint8, device="cuda")
    scales = torch.empty(8192, 896, dtype=torch.uint8, device="cuda")
    ar.ar_qdq_mxfp4(W, None, None, None, codes, scales)
    ref = L.mxfp4_qdq(W[:64].double().cpu().numpy())
    assert np.array_equal(codes[:64].cpu().numpy(), L.pack_fp4(ref["codes"]))
    assert torch.equal(codes[:64].repeat(128, 1), codes) and torch.equal(scales[:64].repeat(128, 1), scales)
    for T in (1, 7, 16, 256):
        A = _acts(T, 28672, T)
        out = _product(ar, A, codes, scales)
        _check_product(out[:, :64], A, codes[:64], scales[:64])
        _check_product(out[:, -64:], A, codes[:64], scales[:64])


@pytest.mark.parametrize("K", [256, 1056])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 40])
def test_product_large_scales(ar, T, K):
    """Scale codes up to 252, the largest of finite weights, in some rows, with activations that keep the result finite; a row
    whose product is not finite, and one whose scale is NaN next to large ones, do not touch the others."""
    rng = np.random.default_rng(T + K)
    N = 50
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(214, 253, (N, K // 32), dtype=np.uint8))
    scales[::3] = torch.from_numpy(rng.integers(100, 130, (len(range(0, N, 3)), K // 32), dtype=np.uint8))
    scales[7] = 252
    scales = scales.cuda()
    A = (_acts(T, K, 3).double() * 2.0 ** -30).bfloat16()
    _check_product(_product(ar, A, codes, scales), A, codes, scales)
    one = torch.zeros_like(A)
    one[:, 5] = 1.0  # one product a result: exact
    want = torch.from_numpy(L.mxfp4_values(codes.cpu().numpy(), scales.cpu().numpy())[:, 5]).cuda()
    assert torch.equal(_product(ar, one, codes, scales).double(), want.expand(T, N))
    scales[4, 1] = 255
    big = one * 64.0
    got = _product(ar, big, codes, scales).double()
    assert got[:, 4].isnan().all()
    keep = [n for n in range(N) if n != 4]
    want = (64.0 * want).bfloat16().double()  # infinite where it leaves the range
    assert torch.equal(got[:, keep], want[keep].expand(T, N - 1)) and want.isinf().any()
    assert ar.ar_get_device_status() == ar.AR_OK


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9])
@pytest.mark.parametrize("K", [256, 800])
def test_product_scales_that_make_up_for_activations(ar, T, K):
    """Blocks whose activations lie far below the others' (2^-16 to 2^-60 of the largest) and whose weights' scales are as much
    larger: each block counts as much as the others.  A token whose activations are all alike next to it, and blocks of
    zeros."""
    rng = np.random.default_rng(T + K)
    N = 40
    down = rng.permutation(np.linspace(0, 60, K // 32).round().astype(int))
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(np.broadcast_to(down + 120, (N, K // 32)).astype(np.uint8).copy())
    scales[N // 2:] = 127
    scales = scales.cuda()
    A = rng.normal(size=(T, K)) * np.repeat(2.0 ** -down.astype(float), 32)[None]
    A[:, :32] = 0
    if T > 2:
        A[1] = rng.normal(size=K)
    A = torch.from_numpy(A).bfloat16().cuda()
    _check_product(_product(ar, A, codes, scales), A, codes, scales)
    # without the largest block the others still come out to the product's own rounding
    A[:, torch.from_numpy(np.repeat(down == 0, 32))] = 0
    _check_product(_product(ar, A, codes, scales), A, codes, scales)
    assert ar.ar_get_device_status() == ar.AR_OK
