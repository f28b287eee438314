"""Refusals of the MXFP4 and cache entry points: every call fails host-side validation (fake pointers, no GPU)."""
import ctypes
import os

import pytest
import torch

import post_weight_quantization_autoround_b200 as ar

pytestmark = pytest.mark.skipif(not os.path.exists(ar.library_path), reason="libautoround.so not built")

P = 0x100000
BAD, NO, WS = ar.AR_ERR_INVALID_ARG, ar.AR_ERR_UNSUPPORTED, ar.AR_ERR_WORKSPACE


def qdq(W=P, V=P, a=P, N=8, K=64, out=P, codes=P, scales=P):
    return ar.lib().ar_qdq_mxfp4(W, V, a, N, K, out, codes, scales, None)


def bwd(g=P, W=P, V=P, a=P, N=8, K=64, dV=P, da=P):
    return ar.lib().ar_qdq_mxfp4_backward(g, W, V, a, N, K, dV, da, None)


def gemm(A=P, T=4, codes=P, scales=P, N=8, K=64, out=P, ws=None, n=0):
    return ar.lib().ar_mxfp4_gemm(A, T, codes, scales, N, K, out, ws, n, None)


@pytest.mark.parametrize("kw,status", [(dict(N=0), BAD), (dict(K=48), BAD), (dict(W=None), BAD), (dict(W=P + 8), BAD),
                                       (dict(V=P + 4), BAD), (dict(a=P + 2), BAD), (dict(out=P + 2), BAD),
                                       (dict(out=None, codes=None, scales=None), BAD), (dict(N=1 << 40), NO)])
def test_qdq_refusals(kw, status):
    assert qdq(**kw) == status and ar.ar_last_error()


@pytest.mark.parametrize("kw,status", [(dict(g=None), BAD), (dict(K=33), BAD), (dict(dV=None, da=None), BAD),
                                       (dict(dV=P + 4), BAD), (dict(da=P + 1), BAD), (dict(W=P + 2), BAD)])
def test_backward_refusals(kw, status):
    assert bwd(**kw) == status and ar.ar_last_error()


@pytest.mark.parametrize("kw,status", [(dict(T=0), BAD), (dict(T=1 << 31), NO), (dict(K=16), BAD), (dict(N=0), BAD),
                                       (dict(A=P + 2), BAD), (dict(out=None), BAD), (dict(scales=P + 8), BAD),
                                       (dict(T=4096, ws=P, n=100), WS), (dict(T=4096, ws=P + 16, n=1 << 30), BAD)])
def test_gemm_refusals(kw, status):
    assert gemm(**kw) == status and ar.ar_last_error()


def test_gemm_workspace():
    assert ar.ar_mxfp4_gemm_workspace(4096, 1024, 256) >= 1024 * 256 * 2
    assert 0 < ar.ar_mxfp4_gemm_workspace(1, 1024, 256) < 4096
    for bad in ((0, 8, 64), (1, 0, 64), (1, 8, 40)):
        with pytest.raises(ar.ARError):
            ar.ar_mxfp4_gemm_workspace(*bad)


def test_tune_step_refusals():
    cfg = ar.ar_qconfig_default()

    def call(W=P, N=64, K=64, M=64, loss=P, ws=P, n=1 << 40, steps=1, cfg=cfg):
        return ar.lib().ar_tune_step_mxfp4(W, P, P, N, K, P, M, P, ctypes.byref(cfg), steps, loss, None, None, ws, n, None)

    assert call(W=None) == BAD and call(K=48) == BAD and call(N=60) == BAD and call(M=3) == BAD and call(steps=-1) == BAD
    assert call(n=10) == WS and call(ws=P + 16) == BAD and call(loss=P + 2) == BAD
    assert call(cfg=ar.ar_qconfig_default(lr=float("nan"))) == BAD
    assert ar.ar_tune_step_mxfp4_workspace(64, 64, 64, 3) > 64 * 64 * 6
    with pytest.raises(ar.ARError):
        ar.ar_tune_step_mxfp4_workspace(64, 64, 48, 3)


def cfg8(**kw):
    d = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10, max_pages=4)
    d.update(kw)
    return ar.Kv8Cfg(**d)


def append(c=None, qkv=P, T=4, cu=P, lens=P, table=P, S=2, max_new=2, base=10000.0, k=P, v=P, ks=P, vs=P, q=P):
    return ar.lib().ar_kv8_append(ctypes.byref(c or cfg8()), qkv, T, cu, lens, table, S, max_new, base, k, v, ks, vs, q, None)


def attend(c=None, q=P, T=4, cu=P, lens=P, table=P, S=2, max_new=2, scale=0.0, k=P, v=P, ks=P, vs=P, out=P, lse=None, ws=P,
           n=1 << 30):
    return ar.lib().ar_attention_kv8(ctypes.byref(c or cfg8()), q, T, cu, lens, table, S, max_new, scale, k, v, ks, vs, out,
                                     lse, ws, n, None)


@pytest.mark.parametrize("kw,status", [(dict(n_heads=0), BAD), (dict(n_heads=7), BAD), (dict(n_kv_heads=0), BAD),
                                       (dict(head_dim=96), NO), (dict(page_size=8), NO), (dict(page_size=48), NO),
                                       (dict(n_pages=0), BAD), (dict(max_pages=0), BAD), (dict(n_pages=1 << 31), NO),
                                       (dict(max_pages=1 << 30), NO), (dict(n_heads=1 << 20), NO)])
def test_cache_description_refusals(kw, status):
    for call in (append, attend):
        assert call(cfg8(**kw)) == status and ar.ar_last_error()


@pytest.mark.parametrize("kw,status", [(dict(T=0), BAD), (dict(S=0), BAD), (dict(S=4097), NO), (dict(max_new=0), BAD),
                                       (dict(max_new=5), BAD), (dict(T=1 << 30, max_new=1), NO), (dict(cu=None), BAD),
                                       (dict(lens=P + 2), BAD), (dict(table=None), BAD), (dict(k=P + 8), BAD), (dict(v=None), BAD),
                                       (dict(ks=None), BAD), (dict(vs=None), BAD), (dict(q=P + 2), BAD)])
def test_cache_argument_refusals(kw, status):
    for call in (append, attend):
        assert call(**kw) == status and ar.ar_last_error()


def test_append_and_attention_refusals():
    assert append(qkv=P + 2) == BAD
    for base in (0.5, -1.0, float("nan"), float("inf")):
        assert append(base=base) == BAD
    assert attend(out=P + 4) == BAD and attend(lse=P + 2) == BAD and attend(ws=None) == WS and attend(n=100) == WS
    assert attend(ws=P + 16) == BAD
    for scale in (-1.0, float("nan"), float("inf")):
        assert attend(scale=scale) == BAD
    # 2^31 units of work or more
    assert attend(cfg8(max_pages=(1 << 30) // 16, n_heads=64, n_kv_heads=64), T=1 << 20, max_new=1) == NO


def test_attention_workspace():
    args = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10, max_pages=4)
    one = ar.ar_attention_kv8_workspace(4, 4, 1, **args)
    many = ar.ar_attention_kv8_workspace(400, 4, 100, **args)
    assert 0 < one < many
    with pytest.raises(ar.ARError):
        ar.ar_attention_kv8_workspace(4, 4, 1, **dict(args, head_dim=80))


def test_attention_limit_of_steps():
    """2^31 steps bound what runs on mma.sync; the call and its workspace query agree."""
    def check(T, S, max_new, refused, **kw):
        d = dict(n_heads=64, n_kv_heads=8, head_dim=64, page_size=128, n_pages=1000, max_pages=1024)
        d.update(kw)
        got = attend(cfg8(**d), T=T, S=S, max_new=max_new, ws=None)
        size = ar.lib().ar_attention_kv8_workspace(ctypes.byref(cfg8(**d)), T, S, max_new)
        assert (got, size > 0) == ((NO, False) if refused else (WS, True)), (got, size, ar.ar_last_error())

    check(65536, 1, 65536, False)
    check(1 << 20, 64, 1, False, max_pages=1 << 13)  # rows behind the last sequence are no work
    check(131072, 1, 131072, True)
    check(4096, 4096, 1, True, head_dim=128, max_pages=1 << 23)


class _OnDevice(torch.Tensor):
    """A tensor that says it lies on a CUDA device of the given number."""
    def get_device(self):
        return self.number


def test_workspace_on_another_device_is_refused():
    w = torch.empty(64, dtype=torch.float32).as_subclass(_OnDevice)
    w.number = 1
    assert ar._space(w, 1) == (w.data_ptr(), 256) and ar._space(None, 0) == (None, 0)
    with pytest.raises(ar.ARError):
        ar._space(w, 0)
    with pytest.raises(ar.ARError):
        ar._space(torch.empty(64), 0)  # host memory
    strided = w[::2]
    strided.number = 1
    with pytest.raises(ar.ARError):
        ar._space(strided, 1)


def test_entry_points_check_their_workspace(monkeypatch):
    """Each of the three binds its workspace through that check."""
    monkeypatch.setattr(ar, "_typed", lambda *a: P)
    monkeypatch.setattr(ar, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    w = torch.empty(1 << 20, dtype=torch.uint8).as_subclass(_OnDevice)
    w.number = 1
    bf, u8, i32, f32 = (lambda *s, t=t: torch.empty(s, dtype=t) for t in (torch.bfloat16, torch.uint8, torch.int32, torch.float32))
    calls = [lambda: ar.ar_mxfp4_gemm(bf(4, 64), u8(8, 32), u8(8, 2), bf(4, 8), w),
             lambda: ar.ar_tune_step_mxfp4(bf(8, 64), f32(8, 64), f32(8, 2), bf(8, 64), f32(8, 8), ar.ar_qconfig_default(), 1, f32(1), w),
             lambda: ar.ar_attention_kv8(bf(1, 128), i32(2), i32(1), i32(1, 1), u8(1, 1, 16, 128), u8(1, 1, 16, 128), u8(1, 1), u8(1, 1),
                                         bf(1, 128), 1, w)]
    for call in calls:
        with pytest.raises(ar.ARError, match="workspace"):
            call()
