"""The paged 8-bit cache on the GPU against the 64-bit oracle.

Append: values go from bf16 to E4M3 with an exact power-of-two scale, so their codes are equal.  Keys pass the
rotation in fp32 (two products and a sum: 3 * 2^-24, cosine and sine another 2 * 2^-24 each, of |a| + |b|, taken as
2^-21), so a key's code may be the neighbour where the exact value lies that near a border: the value read back is
within half a step (2^-4 relative, 2^-10 of the scale for subnormal codes) plus that.

Attention: P is f16 (2^-11 relative half a step, 2^-25 absolute where it is subnormal), the exponent carries fp32
errors of z: sums over d / 16 steps and the scaling, at most 16 * 2^-23 of the largest sum of magnitudes, times ln 2
by the exponential (2^-22 more); the output rounds to bf16 (2^-8)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import lowbit_oracle as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ar():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_autoround_b200 as m
    return m


class Cache:
    """A batch's cache: random valid codes everywhere or, with garbage, arbitrary bytes (NaN codes among them) past the
    sequences' ends; a table of pages in random order, -1 past the last one."""

    def __init__(self, lens, n_heads, n_kv, d, page, seed, garbage=True, spread=3, max_pages=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.n_heads, self.n_kv, self.d, self.page = rng, list(lens), n_heads, n_kv, d, page
        used = [-(-n // page) for n in lens]
        width = max_pages or max(1, max(used))
        total = sum(used) + 3
        order = rng.permutation(total)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        shape = (total, n_kv, page, d)
        self.k, self.v = (L.e4m3_codes(rng.normal(0, 100, shape)) for _ in range(2))
        self.ks, self.vs = (rng.integers(120 - spread, 121 + spread, (total, n_kv)).astype(np.uint8) for _ in range(2))
        if garbage:
            free = np.ones((total, page), bool)
            for s, n in enumerate(lens):
                for j in range(n):
                    free[self.table[s, j // page], j % page] = False
            for x in (self.k, self.v):
                x.transpose(0, 2, 1, 3)[free] = rng.integers(0, 256, (free.sum(), n_kv, d), dtype=np.uint8)
                x.transpose(0, 2, 1, 3)[free, :, ::3] = 0x7F

    def gpu(self):
        return [torch.from_numpy(x.copy()).cuda() for x in (self.k, self.v, self.ks, self.vs)]


def _index(news, lens):
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda(), torch.tensor(list(lens), dtype=torch.int32, device="cuda")


def _workspace(ar, c, T, max_new):
    n = ar.ar_attention_kv8_workspace(T, len(c.lens), max_new, c.n_heads, c.n_kv, c.d, c.page, c.k.shape[0], c.table.shape[1])
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _attend(ar, c, q, cu, lens, max_new, gpu=None, rows=None, lse=None, ws=None, scale=0.0):
    k, v, ks, vs = gpu or c.gpu()
    out = torch.full_like(q, 7.0)
    ws = _workspace(ar, c, q.shape[0], max_new) if ws is None else ws
    ar.ar_attention_kv8(q, cu, lens, torch.from_numpy(c.table).cuda(), k, v, ks, vs, out, max_new, ws, lse=lse, sm_scale=scale)
    return out


def _check(c, q, cu, out, lse=None, scale=None):
    T = cu[-1]
    ref, rl, mag, units, zmag = L.kv8_attention(q[:T].double().cpu().numpy(), cu, c.lens, c.table, c.k, c.v, c.ks, c.vs, c.n_heads, scale)
    got = out[:T].double().cpu().numpy().reshape(ref.shape)
    zerr = (16 * 2.0 ** -23 * zmag + 2.0 ** -21)[..., None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * zerr) * mag + 2.0 ** -25 * units + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:4], ref[bad][:4], tol[bad][:4])
    if lse is not None:
        l = lse[:T].double().cpu().numpy()
        assert np.array_equal(np.isinf(l), np.isinf(rl))
        f = np.isfinite(rl)
        assert (np.abs(l[f] - rl[f]) <= zerr[..., 0][f] + 2.0 ** -21 * (2 + np.abs(rl[f]))).all()


SHAPES = [(8, 8, 128), (8, 1, 128), (10, 2, 64), (14, 2, 128), (16, 1, 128), (32, 1, 64), (40, 1, 128), (5, 5, 64)]


@pytest.mark.parametrize("n_heads,n_kv,d", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_one_token(ar, n_heads, n_kv, d, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 200, 513]
    c = Cache(lens, n_heads, n_kv, d, page, n_heads + page)
    cu, cud, ld = _index([1] * len(lens), lens)
    q = torch.from_numpy(c.rng.normal(size=(len(lens), n_heads * d)).astype(np.float32)).bfloat16().cuda()
    lse = torch.empty(len(lens), n_heads, device="cuda")
    out = _attend(ar, c, q, cud, ld, 1, lse=lse)
    _check(c, q, cu, out, lse)
    assert ar.ar_get_device_status() == ar.AR_OK and "attn_kv8_kernel" in ar.ar_last_kernels()


@pytest.mark.parametrize("n_heads,n_kv,d,page", [(8, 2, 128, 16), (14, 2, 64, 64), (4, 4, 128, 128), (8, 1, 64, 32)])
def test_attention_ragged_chunks(ar, n_heads, n_kv, d, page):
    """Several new tokens a sequence, none, a whole prompt, more than the cache holds (rows that see no key), an empty
    sequence; rows behind the last one stay as they were."""
    news = [3, 0, 40, 1, 9, 5, 0, 33, 1]
    lens = [130, 77, 40, 500, 4, 260, 0, 300, 0]
    c = Cache(lens, n_heads, n_kv, d, page, d + page)
    cu, cud, ld = _index(news, lens)
    T = cu[-1] + 5
    q = torch.from_numpy(c.rng.normal(size=(T, n_heads * d)).astype(np.float32)).bfloat16().cuda()
    lse = torch.full((T, n_heads), 3.0, device="cuda")
    out = _attend(ar, c, q, cud, ld, 40, lse=lse)
    _check(c, q, cu, out, lse)
    empty = slice(cu[4], cu[4] + 5)  # nine new tokens, four keys
    assert not out[empty].any() and lse[empty].isneginf().all() and not out[cu[8]].any()
    assert (out[cu[-1]:] == 7.0).all() and (lse[cu[-1]:] == 3.0).all()
    assert ar.ar_get_device_status() == ar.AR_OK


@pytest.mark.parametrize("n_heads,n_kv,d,lens", [(1, 1, 128, [40001]), (8, 1, 64, [20000, 5, 9000]), (16, 1, 128, [17000]),
                                                 (32, 1, 128, [9001, 1])])
def test_attention_split_over_blocks(ar, n_heads, n_kv, d, lens):
    """Few rows over a long axis: row tiles that many blocks share; twice the same answer, and in a graph whose lengths
    change between replays."""
    c = Cache(lens, n_heads, n_kv, d, 64, 5, max_pages=700)
    cu, cud, ld = _index([1] * len(lens), lens)
    q = torch.from_numpy(c.rng.normal(size=(len(lens), n_heads * d)).astype(np.float32)).bfloat16().cuda()
    gpu = c.gpu()
    out = _attend(ar, c, q, cud, ld, 1, gpu)
    _check(c, q, cu, out)
    assert torch.equal(out, _attend(ar, c, q, cud, ld, 1, gpu))
    ws, got, table = _workspace(ar, c, len(lens), 1), torch.empty_like(q), torch.from_numpy(c.table).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ar.ar_attention_kv8(q, cud, ld, table, *gpu, got, 1, ws)
    g.replay()
    assert torch.equal(out, got)
    c.lens[0] //= 3
    ld[0] = c.lens[0]
    g.replay()
    torch.cuda.synchronize()
    _check(c, q, cu, got)


@pytest.mark.parametrize("n_heads,n_kv,page,news,lens", [
    (64, 8, 16, [200, 0, 129, 1, 97], [1000, 50, 129, 700, 97]),
    (40, 8, 64, [300, 300], [300, 811]),
    (32, 32, 128, [700], [1301]),
    (21, 3, 32, [900, 33, 600, 5], [890, 1, 613, 3]),  # rows that see no key, an odd group
    (148, 4, 128, [130, 7], [4500, 4200]),
])
def test_attention_prompts(ar, n_heads, n_kv, page, news, lens):
    """Rows enough for the tcgen05 kernel, ragged, with page tables that end and garbage past the sequences' ends."""
    c = Cache(lens, n_heads, n_kv, 128, page, n_heads)
    cu, cud, ld = _index(news, lens)
    T = cu[-1] + 3
    q = torch.from_numpy(c.rng.normal(size=(T, n_heads * 128)).astype(np.float32)).bfloat16().cuda()
    lse = torch.full((T, n_heads), 3.0, device="cuda")
    gpu = c.gpu()
    out = _attend(ar, c, q, cud, ld, max(news), gpu, lse=lse)
    assert "attn_kv8_tc_kernel" in ar.ar_last_kernels() and ar.ar_get_device_status() == ar.AR_OK
    _check(c, q, cu, out, lse)
    assert (out[cu[-1]:] == 7.0).all() and (lse[cu[-1]:] == 3.0).all()
    assert torch.equal(out, _attend(ar, c, q, cud, ld, max(news), gpu))


def test_attention_prompts_growing_scores_and_scales(ar):
    """Maxima that grow from block to block (the sums in tensor memory are rescaled often), and value scales 2^20 apart."""
    lens, news = [1500], [640]
    c = Cache(lens, 32, 8, 128, 16, 9)
    c.vs[:] = c.rng.integers(100, 121, c.vs.shape)
    for j in range(lens[0]):
        c.ks[c.table[0, j // 16]] = 112 + j // 150
    cu, cud, ld = _index(news, lens)
    q = torch.from_numpy(c.rng.normal(size=(640, 32 * 128)).astype(np.float32)).bfloat16().cuda()
    lse = torch.empty(640, 32, device="cuda")
    out = _attend(ar, c, q, cud, ld, 640, lse=lse)
    assert "attn_kv8_tc_kernel" in ar.ar_last_kernels()
    _check(c, q, cu, out, lse)
    # a page that is not in the pool, a sequence with more tokens than said
    c.table[0, 3] = c.k.shape[0]
    _attend(ar, c, q, cud, ld, 640)
    assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG
    out = _attend(ar, c, q, cud, ld, 639)
    assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG and (out == 7.0).all()


def test_attention_prompts_next_to_single_tokens(ar):
    """Sequences of a few rows run on mma.sync, long and short, the others of the same call on tcgen05."""
    news, lens = [200, 1, 1, 129, 1, 3, 0, 4, 1, 40], [900, 5000, 1, 129, 64, 700, 50, 300, 0, 9]
    c = Cache(lens, 64, 8, 128, 32, 5)
    cu, cud, ld = _index(news, lens)
    T = cu[-1] + 2
    q = torch.from_numpy(c.rng.normal(size=(T, 64 * 128)).astype(np.float32)).bfloat16().cuda()
    lse = torch.full((T, 64), 3.0, device="cuda")
    gpu = c.gpu()
    out = _attend(ar, c, q, cud, ld, 200, gpu, lse=lse)
    kernels = ar.ar_last_kernels().split(";")
    assert "attn_kv8_tc_kernel" in kernels and "attn_kv8_kernel" in kernels and ar.ar_get_device_status() == ar.AR_OK
    _check(c, q, cu, out, lse)
    assert (out[cu[-1]:] == 7.0).all() and (lse[cu[-1]:] == 3.0).all()
    assert torch.equal(out, _attend(ar, c, q, cud, ld, 200, gpu))
    # a sequence that does not fit is left as it was by both kernels
    cu[5] = cu[4] - 1
    out2 = _attend(ar, c, q, torch.from_numpy(cu).cuda(), ld, 200, gpu)
    assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG and torch.equal(out2[:cu[4] - 1], out[:cu[4] - 1])


@pytest.mark.parametrize("page", [16, 128])
def test_attention_prompts_of_one_tile(ar, page):
    """Up to 128 rows a sequence and head: one tile, whose blocks two groups share by turns; lengths around whole blocks,
    odd and even counts of them, maxima that grow, rows that see no key; a query that is not finite stays in its row."""
    lens = [16, 17, 128, 129, 255, 256, 257, 384, 385, 1000, 5, 1300, 513]
    news = [16, 15, 16, 1, 16, 7, 16, 16, 9, 16, 16, 16, 0]
    c = Cache(lens, 96, 12, 128, page, page)
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            c.ks[c.table[s, i]] = 114 + min(13, i * page // 60 + s % 2)
    cu, cud, ld = _index(news, lens)
    T = cu[-1] + 2
    q = torch.from_numpy(c.rng.normal(size=(T, 96 * 128)).astype(np.float32)).bfloat16().cuda()
    lse = torch.full((T, 96), 3.0, device="cuda")
    gpu = c.gpu()
    out = _attend(ar, c, q, cud, ld, 16, gpu, lse=lse)
    assert "attn_kv8_tc_kernel" in ar.ar_last_kernels() and ar.ar_get_device_status() == ar.AR_OK
    _check(c, q, cu, out, lse)
    assert (out[cu[-1]:] == 7.0).all() and (lse[cu[-1]:] == 3.0).all()
    rows = [(cu[9] + 3, 40, "nan"), (cu[11], 0, "inf"), (cu[4] + 15, 95, "-inf")]
    for t, h, x in rows:
        q[t, h * 128 + 5] = float(x)
    got = _attend(ar, c, q, cud, ld, 16, gpu)
    for t, h, x in rows:
        assert not torch.equal(got[t, h * 128:(h + 1) * 128], out[t, h * 128:(h + 1) * 128])
        got[t, h * 128:(h + 1) * 128] = out[t, h * 128:(h + 1) * 128]
    assert torch.equal(got, out)


@pytest.mark.parametrize("n_heads,n_kv,d", [(8, 8, 128), (64, 4, 64), (24, 1, 128)])
def test_attention_many_short_sequences(ar, n_heads, n_kv, d):
    """Many items to a block, most of them too short to give every warp a step, some in two pieces."""
    rng = np.random.default_rng(n_heads)
    lens = [int(x) for x in rng.choice([1, 3, 20, 40, 200, 300, 700], 700, p=[.3, .2, .2, .1, .1, .05, .05])]
    c = Cache(lens, n_heads, n_kv, d, 16, 3)
    cu, cud, ld = _index([1] * len(lens), lens)
    q = torch.from_numpy(c.rng.normal(size=(len(lens), n_heads * d)).astype(np.float32)).bfloat16().cuda()
    out = _attend(ar, c, q, cud, ld, 1)
    assert ar.ar_get_device_status() == ar.AR_OK
    _check(c, q, cu, out)


def test_attention_scales_that_differ_widely(ar):
    """Value scales 2^20 apart between pages, key scales that make some scores large: the weights' f16 rounding stays
    relative to the largest contribution."""
    lens = [400, 90]
    c = Cache(lens, 8, 2, 128, 16, 8)
    c.vs[:] = c.rng.integers(100, 121, c.vs.shape)
    c.ks[:] = c.rng.integers(116, 121, c.ks.shape)
    cu, cud, ld = _index([1, 1], lens)
    q = torch.from_numpy(c.rng.normal(size=(2, 1024)).astype(np.float32)).bfloat16().cuda()
    _check(c, q, cu, _attend(ar, c, q, cud, ld, 1))
    # queries far from 1, and zero
    for f in (2.0 ** -60, 0.0):
        qs = (q.double() * f).bfloat16()
        _check(c, qs, cu, _attend(ar, c, qs, cud, ld, 1))
    qs = (q.double() * 2.0 ** 60).bfloat16()
    _check(c, qs, cu, _attend(ar, c, qs, cud, ld, 1, scale=2.0 ** -64), scale=2.0 ** -64)


def test_attention_non_finite_query_stays_in_its_row(ar):
    lens = [60, 70]
    c = Cache(lens, 8, 1, 128, 32, 2)
    cu, cud, ld = _index([1, 1], lens)
    q = torch.from_numpy(c.rng.normal(size=(2, 1024)).astype(np.float32)).bfloat16().cuda()
    want = _attend(ar, c, q, cud, ld, 1)
    q[0, 130] = float("nan")
    got = _attend(ar, c, q, cud, ld, 1)
    assert got[0, 128:256].isnan().all()
    got[0, 128:256] = want[0, 128:256]
    assert torch.equal(got, want)


def test_attention_bad_indices_are_skipped(ar):
    """Page numbers outside the pool, bounds outside the arrays: raised, and the other sequences come out right."""
    lens = [100, 100, 100]
    c = Cache(lens, 8, 2, 64, 16, 4)
    cu, cud, ld = _index([1, 1, 1], lens)
    q = torch.from_numpy(c.rng.normal(size=(3, 512)).astype(np.float32)).bfloat16().cuda()
    want = _attend(ar, c, q, cud, ld, 1)
    good = c.table.copy()
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table = good.copy()
        c.table[1, 2] = bad
        got = _attend(ar, c, q, cud, ld, 1)
        assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    c.table = good
    for bad in (-5, 7 * 16 + 1, 2 ** 31 - 1):
        ld[1] = bad
        got = _attend(ar, c, q, cud, ld, 1)
        assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and (got[1] == 7.0).all()
    ld[1] = 100
    two = torch.tensor([0, 0, 2, 3], dtype=torch.int32, device="cuda")  # the second sequence has more than max_new
    got = _attend(ar, c, q, two, ld, 1)
    assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG
    assert torch.equal(got[2], want[2]) and (got[:2] == 7.0).all()
    for bad in (-1, 9, 2 ** 31 - 1):
        cud[3] = bad
        got = _attend(ar, c, q, cud, ld, 1)
        assert ar.ar_get_device_status() == ar.AR_ERR_INVALID_ARG
        assert torch.equal(got[:2], want[:2]) and (got[2] == 7.0).all()


def _check_keys(c, gpu, keys, qkv):
    """Keys: their scales equal, their values within half a code's step of the exact rotation."""
    k, ks = gpu[0].cpu().numpy(), gpu[2].cpu().numpy()
    for ph, h, at, new in keys:
        scale = 2.0 ** (int(ks[ph, h]) - 127)
        got = L.e4m3_values(k[ph, h, at:at + len(new)]) * scale
        err = 2.0 ** -21 * np.abs(new).max(1, keepdims=True) * 2
        assert (np.abs(got - new) <= np.maximum(2.0 ** -4 * np.abs(new), 2.0 ** -10 * scale) * (1 + 2.0 ** -20) + err).all()


@pytest.mark.parametrize("n_heads,n_kv,d", [(6, 6, 128), (8, 2, 64), (14, 2, 128), (5, 1, 64)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append(ar, n_heads, n_kv, d, page):
    """From one token to several pages a sequence, pages begun before (whose scale grows, or does not), none, far
    positions; bytes that belong to no new or older token stay."""
    news = [1, 1, 0, 3, page, page + 1, 2 * page + 7, 1, 1, 5]
    lens = [1, page + 3, 9, 3, page, 3 * page, 4 * page + 1, page, 6 * page + 2, 5 + page - 2]
    c = Cache(lens, n_heads, n_kv, d, page, d + page)
    cu, cud, ld = _index(news, lens)
    T = cu[-1] + 2
    qkv = c.rng.normal(size=(T, (n_heads + 2 * n_kv) * d)) * 3
    qkv[cu[1]:cu[2]] *= 2.0 ** -9  # older tokens keep the larger scale
    qkv[cu[8]:cu[9]] *= 2.0 ** 13  # older tokens are re-coded
    qkv = torch.from_numpy(qkv.astype(np.float32)).bfloat16().cuda()
    gpu = c.gpu()
    q_out = torch.full((T, n_heads * d), 7.0, dtype=torch.bfloat16, device="cuda")
    ar.ar_kv8_append(qkv, cud, ld, torch.from_numpy(c.table).cuda(), *gpu, q_out, 2 * page + 7)
    assert ar.ar_get_device_status() == ar.AR_OK, ar.ar_last_error()
    before = c.k.copy()
    rq, keys = L.kv8_append(qkv.double().cpu().numpy()[:cu[-1]], cu, lens, c.table, c.k, c.v, c.ks, c.vs, n_heads)
    got = q_out[:cu[-1]].double().cpu().numpy().reshape(rq.shape)
    assert (np.abs(got - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -21 * np.abs(rq).max(2, keepdims=True) * 2).all()
    assert (q_out[cu[-1]:] == 7.0).all()
    assert np.array_equal(gpu[1].cpu().numpy(), c.v) and np.array_equal(gpu[3].cpu().numpy(), c.vs)
    assert np.array_equal(gpu[2].cpu().numpy(), c.ks)
    _check_keys(c, gpu, keys, qkv)
    k = gpu[0].cpu().numpy()
    new = np.zeros(k.shape, bool)
    for ph, h, at, rows in keys:
        new[ph, h, at:at + len(rows)] = True
    assert np.array_equal(k[~new], c.k[~new])  # untouched, or re-coded the same
    assert (before[~new] != c.k[~new]).any() and (k[new] != c.k[new]).mean() < 1e-3


def test_append_far_positions(ar):
    """A position past 10^6: the angle keeps its fraction of a turn."""
    page, d = 128, 128
    lens = [1_000_001, 777_777]
    n_pages = 4
    table = np.zeros((2, -(-lens[0] // page)), np.int32)
    table[0, (lens[0] - 1) // page], table[1, (lens[1] - 1) // page] = 1, 2
    k, v = (np.zeros((n_pages, 1, page, d), np.uint8) for _ in range(2))
    ks, vs = (np.full((n_pages, 1), 27, np.uint8) for _ in range(2))
    cu, cud, ld = _index([1, 1], lens)
    qkv = torch.from_numpy(np.random.default_rng(0).normal(size=(2, 3 * d)).astype(np.float32)).bfloat16().cuda()
    gpu = [torch.from_numpy(x.copy()).cuda() for x in (k, v, ks, vs)]
    q_out = torch.empty(2, d, dtype=torch.bfloat16, device="cuda")
    ar.ar_kv8_append(qkv, cud, ld, torch.from_numpy(table).cuda(), *gpu, q_out, 1, rope_base=500000.0)
    rq, keys = L.kv8_append(qkv.double().cpu().numpy(), cu, lens, table, k, v, ks, vs, 1, base=500000.0)
    got = q_out.double().cpu().numpy().reshape(rq.shape)
    assert (np.abs(got - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -20 * np.abs(rq).max(2, keepdims=True)).all()
    _check_keys(None, gpu, keys, qkv)


def test_append_non_finite_and_zero(ar):
    c = Cache([20, 20], 2, 1, 64, 16, 1)
    cu, cud, ld = _index([4, 4], [20, 20])
    qkv = torch.from_numpy(c.rng.normal(size=(8, 4 * 64)).astype(np.float32)).bfloat16().cuda()
    qkv[0, 192], qkv[1, 193], qkv[2, 194] = float("nan"), float("inf"), -float("inf")  # values of the first sequence
    qkv[4:, 128:] = 0.0  # keys and values of the second
    gpu = c.gpu()
    q_out = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
    ar.ar_kv8_append(qkv, cud, ld, torch.from_numpy(c.table).cuda(), *gpu, q_out, 4)
    assert ar.ar_get_device_status() == ar.AR_ERR_NONFINITE
    v = gpu[1][c.table[0, 1], 0].cpu().numpy()
    assert v[0, 0] == 0 and v[1, 1] == 0x7E and v[2, 2] == 0xFE
    finite = qkv[:4, 192:].double().cpu().numpy()
    finite[~np.isfinite(finite)] = 0
    assert gpu[3][c.table[0, 1], 0].item() == L.exponent_for(np.abs(finite).max()) + 127
    z = c.table[1, 1]
    # zeros of either sign: a rotation gives 0 * c - 0 * s
    assert not (gpu[0][z, 0, :4] & 0x7F).any() and not (gpu[1][z, 0, :4] & 0x7F).any() and gpu[2][z, 0] == 27 and gpu[3][z, 0] == 27


def test_append_bad_indices_are_skipped(ar):
    lens = [40, 40, 40]
    c = Cache(lens, 4, 2, 64, 16, 6)
    cu, cud, ld = _index([2, 2, 2], lens)
    qkv = torch.from_numpy(c.rng.normal(size=(6, 8 * 64)).astype(np.float32)).bfloat16().cuda()

    def run(table=c.table, cu_=cud, ld_=ld, max_new=2):
        gpu = c.gpu()
        q = torch.full((6, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        ar.ar_kv8_append(qkv, cu_, ld_, torch.from_numpy(table).cuda(), *gpu, q, max_new)
        return gpu, q, ar.ar_get_device_status()

    want, wq, st = run()
    assert st == ar.AR_OK
    page1 = c.table[1, 2]
    others = [p for p in range(c.k.shape[0]) if p != page1]

    def same_but_second(got, q, st):
        assert st == ar.AR_ERR_INVALID_ARG
        for a, b, orig in zip(got, want, (c.k, c.v, c.ks, c.vs)):
            assert torch.equal(a[others], b[others]) and np.array_equal(a[page1].cpu().numpy(), orig[page1])
        assert torch.equal(q[:2], wq[:2]) and torch.equal(q[4:], wq[4:])

    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c.table.copy()
        t[1, 2] = bad
        same_but_second(*run(table=t))
    for bad in (1, 3 * 16 + 1, -3, 2 ** 31 - 1):
        l2 = ld.clone()
        l2[1] = bad
        got, q, st = run(ld_=l2)
        same_but_second(got, q, st)
        assert (q[2:4] == 7.0).all()
    for bad in (7, -1, 2 ** 31 - 1):
        c2 = cud.clone()
        c2[3] = bad
        got, q, st = run(cu_=c2)
        assert st == ar.AR_ERR_INVALID_ARG and torch.equal(q[:4], wq[:4]) and (q[4:] == 7.0).all()
    assert run(max_new=1)[2] == ar.AR_ERR_INVALID_ARG  # every sequence has two


def test_two_calls_at_once(ar):
    """Two streams, a workspace each."""
    cs = [Cache([900, 33], 8, 2, 128, 32, s) for s in (1, 2)]
    cu, cud, ld = _index([1, 1], [900, 33])
    qs = [torch.from_numpy(c.rng.normal(size=(2, 1024)).astype(np.float32)).bfloat16().cuda() for c in cs]
    gpus = [c.gpu() for c in cs]
    want = [_attend(ar, c, q, cud, ld, 1, g) for c, q, g in zip(cs, qs, gpus)]
    ws = [_workspace(ar, c, 2, 1) for c in cs]
    tables = [torch.from_numpy(c.table).cuda() for c in cs]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            ar.ar_attention_kv8(qs[i], cud, ld, tables[i], *gpus[i], outs[i], 1, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_a_decode_step_of_the_operators_together(ar):
    """Norm, MXFP4 projection, append, attention, MXFP4 projection: a prompt in two pieces and then token by token gives
    what the whole prompt at once gives.  Both runs quantize the same keys and values; a page's scale may have grown in
    steps in one of them, which re-codes exactly unless a code is subnormal, so they agree to E4M3's smallest steps;
    measured against the outputs' size that is far below the 2^-5 allowed here (bf16 steps of four roundings in a row
    are 2^-6)."""
    H, n_heads, n_kv, d, page, L_ = 512, 8, 2, 64, 16, 45
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(L_, H, device="cuda", generator=g).bfloat16()
    gamma = torch.ones(H, device="cuda")

    def packed(n, k):
        w = (torch.randn(n, k, device="cuda", generator=g) * 0.05).bfloat16()
        codes, scales = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda"), torch.empty(n, k // 32, dtype=torch.uint8, device="cuda")
        ar.ar_qdq_mxfp4(w, codes=codes, scales=scales)
        return codes, scales

    wqkv, wo = packed((n_heads + 2 * n_kv) * d, H), packed(H, n_heads * d)

    def run(pieces):
        pages = -(-L_ // page)
        k, v = (torch.full((pages, n_kv, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.full((pages, n_kv), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
        table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, -1)
        outs, at = [], 0
        for n in pieces:
            r = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
            ar.ar_rmsnorm(x[at:at + n].contiguous(), gamma, r)
            qkv = torch.empty(n, (n_heads + 2 * n_kv) * d, dtype=torch.bfloat16, device="cuda")
            ar.ar_mxfp4_gemm(r, *wqkv, qkv)
            cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            at += n
            lens = torch.tensor([at], dtype=torch.int32, device="cuda")
            q, o = torch.empty(n, n_heads * d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, n_heads * d, dtype=torch.bfloat16, device="cuda")
            ar.ar_kv8_append(qkv, cu, lens, table, k, v, ks, vs, q, n)
            ws = torch.empty(ar.ar_attention_kv8_workspace(n, 1, n, n_heads, n_kv, d, page, pages, pages), dtype=torch.uint8, device="cuda")
            ar.ar_attention_kv8(q, cu, lens, table, k, v, ks, vs, o, n, ws)
            y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
            ar.ar_mxfp4_gemm(o, *wo, y)
            outs.append(y)
        assert ar.ar_get_device_status() == ar.AR_OK
        return torch.cat(outs).double(), (k, v, ks, vs)

    whole, ca = run([L_])
    steps, cb = run([20, 17] + [1] * 8)
    assert (whole[-1] - steps[-1]).norm() <= 2.0 ** -5 * whole[-1].norm()
    for a, b in zip(ca[2:], cb[2:]):
        assert torch.equal(a, b)  # the scales end where the whole prompt put them


@pytest.mark.parametrize("n_heads,n_new", [(4, 1), (64, 300)])
def test_pool_past_32_bits(ar, n_heads, n_new):
    """A pool of more than 2^32 bytes whose last pages hold the sequence: the same codes and outputs as from a small pool,
    for the decode kernel and for the prompts' one."""
    n_kv, d, page, length = 2, 128, 128, 700
    pages = -(-length // page)
    rng = np.random.default_rng(n_heads)
    cu, cud, ld = _index([n_new], [length])
    qkv = torch.from_numpy(rng.normal(size=(n_new, (n_heads + 2 * n_kv) * d)).astype(np.float32)).bfloat16().cuda()
    small = Cache([length], n_heads, n_kv, d, page, 3, garbage=False).gpu()
    big = 140_000
    table = np.arange(pages, dtype=np.int32)[None]
    results = []
    for total in (small[0].shape[0], big):
        base = 0 if total != big else big - pages
        if total == big:
            pool = [torch.empty((total, *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in small]
            for x, y in zip(pool, small):
                x[base:] = y[:pages]
            assert pool[0].numel() > 2 ** 32
        else:
            pool = [x.clone() for x in small]
        t = torch.from_numpy(table + base).cuda()
        q, out = (torch.empty(n_new, n_heads * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ar.ar_kv8_append(qkv, cud, ld, t, *pool, q, n_new)
        ws = torch.empty(ar.ar_attention_kv8_workspace(n_new, 1, n_new, n_heads, n_kv, d, page, total, pages), dtype=torch.uint8, device="cuda")
        ar.ar_attention_kv8(q, cud, ld, t, *pool, out, n_new, ws)
        assert ("attn_kv8_tc_kernel" in ar.ar_last_kernels()) == (n_new > 1) and ar.ar_get_device_status() == ar.AR_OK
        results.append([x[base:base + pages].clone() for x in pool] + [q, out])
        del pool
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_decode_loop_in_a_graph(ar):
    """One captured append and attention, replayed for every token while the lengths grow, against calls made one by one;
    the graph runs on a stream of its own."""
    n_heads, n_kv, d, page, start, steps = 8, 2, 128, 16, 13, 40
    pages = -(-(start + steps) // page) + 1
    rng = np.random.default_rng(0)
    c = Cache([start, 2 * page], n_heads, n_kv, d, page, 7, max_pages=pages + 2)
    total = c.k.shape[0] + 2 * pages
    gpu = [torch.cat([x, torch.zeros(2 * pages, *x.shape[1:], dtype=x.dtype, device="cuda")]) for x in c.gpu()]
    table = c.table.copy()
    nxt = c.k.shape[0]
    for s in range(2):
        for i in range(table.shape[1]):
            if table[s, i] < 0:
                table[s, i] = nxt
                nxt = nxt + 1 if nxt + 1 < total else nxt
    table = torch.from_numpy(table).cuda()
    tokens = [torch.from_numpy(rng.normal(size=(2, (n_heads + 2 * n_kv) * d)).astype(np.float32)).bfloat16().cuda() for _ in range(steps)]
    cu, cud, _ = _index([1, 1], [start, 2 * page])

    def buffers():
        return dict(pool=[x.clone() for x in gpu], lens=torch.tensor([start, 2 * page], dtype=torch.int32, device="cuda"),
                    q=torch.empty(2, n_heads * d, dtype=torch.bfloat16, device="cuda"),
                    out=torch.empty(2, n_heads * d, dtype=torch.bfloat16, device="cuda"), qkv=torch.empty_like(tokens[0]),
                    ws=torch.empty(ar.ar_attention_kv8_workspace(2, 2, 1, n_heads, n_kv, d, page, total, table.shape[1]), dtype=torch.uint8, device="cuda"))

    def step(b):
        b["lens"] += 1
        ar.ar_kv8_append(b["qkv"], cud, b["lens"], table, *b["pool"], b["q"], 1)
        ar.ar_attention_kv8(b["q"], cud, b["lens"], table, *b["pool"], b["out"], 1, b["ws"])

    one, two = buffers(), buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(two)
    st = torch.cuda.Stream()
    for x in tokens:
        one["qkv"].copy_(x)
        two["qkv"].copy_(x)
        step(one)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(one["out"], two["out"])
    assert ar.ar_get_device_status() == ar.AR_OK and one["lens"].tolist() == [start + steps, 2 * page + steps]
    for a, b in zip(one["pool"], two["pool"]):
        assert torch.equal(a, b)


def test_binding_refusals(ar):
    c = Cache([20], 4, 2, 64, 16, 1)
    cu, cud, ld = _index([1], [20])
    k, v, ks, vs = c.gpu()
    t = torch.from_numpy(c.table).cuda()
    q = torch.zeros(1, 256, dtype=torch.bfloat16, device="cuda")
    ws = _workspace(ar, c, 1, 1)
    good = dict(q=q, cu_seqlens=cud, seq_lens=ld, page_table=t, k_pages=k, v_pages=v, k_scales=ks, v_scales=vs, out=torch.empty_like(q), max_new=1, workspace=ws)
    ar.ar_attention_kv8(**good)
    wide = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda")
    for name, bad in (("q", q.float()), ("out", wide), ("out", wide[:, ::2]), ("cu_seqlens", cud.long()), ("seq_lens", ld.cpu()),
                      ("v_pages", v[:-1]), ("k_scales", ks.int()), ("page_table", t.cpu()), ("seq_lens", ld.repeat(2)), ("workspace", ws[:16])):
        with pytest.raises(ar.ARError):
            ar.ar_attention_kv8(**{**good, name: bad})
    qkv = torch.zeros(1, 8 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ar.ARError):
        ar.ar_kv8_append(qkv, cud, ld, t, k, v, ks, vs, q[:, ::2], 1)
    with pytest.raises(ar.ARError):
        ar.ar_kv8_append(qkv[:, :500], cud, ld, t, k, v, ks, vs, q, 1)
    W = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((W.float(), None, None, W), (W, W, None, W), (W, None, None, W.t()), (W, None, W.float(), W), (W.cpu(), None, None, W)):
        with pytest.raises(ar.ARError):
            ar.ar_qdq_mxfp4(*args)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8, device="cuda"), torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    A = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    for out in (torch.empty(3, 8, device="cuda"), torch.empty(8, 3, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ar.ARError):
            ar.ar_mxfp4_gemm(A, codes, scales, out)
    with pytest.raises(ar.ARError):
        ar.ar_mxfp4_gemm(A, codes[:, :16], scales, torch.empty(3, 8, dtype=torch.bfloat16, device="cuda"))
    assert ar.ar_get_device_status() == ar.AR_OK


def _reference64(c, q, n_new, shift):
    """Outputs and log-sum-exps of a batch of one sequence in 64 bits on the GPU, and the tolerance: an output's bf16 half step; the
    exponent's error (as in _check) of every weight; a weight's f16 half step, 2^-11 of it or 2^-25 below f16's normal range, with
    the row's largest weight (times its value scale) at 2^shift."""
    n, d, group = c.lens[0], c.d, c.n_heads // c.n_kv
    at = np.arange(n)
    pg = c.table[0, at // c.page]
    out, tol = (torch.empty(n_new, c.n_heads, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.empty(n_new, c.n_heads, dtype=torch.float64, device="cuda")
    x = q[:n_new].double().view(n_new, c.n_heads, d)
    late = torch.ones(n_new, n, dtype=torch.bool, device="cuda").triu(n - n_new + 1)
    for h in range(c.n_kv):
        key = torch.from_numpy(L.e4m3_values(c.k[pg, h, at % c.page]) * np.ldexp(1.0, c.ks[pg, h].astype(int) - 127)[:, None]).cuda()
        code = torch.from_numpy(L.e4m3_values(c.v[pg, h, at % c.page])).cuda()
        ev = torch.from_numpy(c.vs[pg, h].astype(np.float64) - 127).cuda()
        value = code * torch.exp2(ev)[:, None]
        for i in range(h * group, (h + 1) * group):
            z = (x[:, i] @ key.t() * d ** -0.5).masked_fill(late, -torch.inf)
            zerr = 16 * 2.0 ** -23 * (x[:, i].abs() @ key.abs().t()).amax(1) * d ** -0.5 + 2.0 ** -21
            lse[:, i] = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[:, i, None])
            out[:, i] = p @ value
            u = z / np.log(2) + ev
            top = u.amax(1, keepdim=True)
            half = torch.clamp(torch.exp2(u - top + shift) * 2.0 ** -11, min=2.0 ** -25).masked_fill(late, 0.0)
            unit = torch.exp2(top - shift - lse[:, i, None] / np.log(2))
            tol[:, i] = 2.0 ** -8 * out[:, i].abs() + 2 * zerr[:, None] * (p @ value.abs()) + (half @ code.abs()) * unit
    return out, lse, tol


def _sink(n, page, raised, n_heads, n_kv, d, n_new, weight):
    """A cache and queries whose first key takes `weight` of every row and has the value zero, before n - 1 keys of ordinary scores:
    they make the output.  raised: the first page's value scale is so many powers of two above the others'."""
    c = Cache([1], n_heads, n_kv, d, page, n_heads)
    pages, rng = -(-n // page), np.random.default_rng(n + n_heads)
    g = torch.Generator().manual_seed(n + n_heads)

    def codes(mean, sd):
        return torch.randn(pages, n_kv, page, d, generator=g).mul_(sd).add_(mean).to(torch.float8_e4m3fn).view(torch.uint8).numpy()

    c.lens, c.table = [n], rng.permutation(pages).astype(np.int32)[None]
    c.k, c.v = codes(0, 16), codes(64, 32)
    c.k[..., 0] = 0
    c.ks, c.vs = (np.full((pages, n_kv), 127 - e, np.uint8) for e in (4, 6))
    first = c.table[0, 0]
    c.k[first, :, 0] = L.e4m3_codes(np.eye(d)[0] * 416)  # 26, the others' dimension 0 is zero
    c.v[first, :, 0] = 0
    if raised:
        c.vs[first] += raised
        c.v[first] = 0
    q = rng.normal(size=(n_new, n_heads, d))
    q[:, :, 0] = np.log(n * np.exp(0.5) * weight / (1 - weight)) * d ** 0.5 / 26
    return c, torch.from_numpy(q.reshape(n_new, n_heads * d).astype(np.float32)).bfloat16().cuda()


def _check_sink(c, q, n_new, out, lse, shift):
    ref, rl, tol = _reference64(c, q, n_new, shift)
    err = (out.double().view(-1, *ref.shape[1:]) - ref).abs()
    assert (err <= tol).all(), ((err / tol).max().item(), (err / ref.abs()).max().item())
    assert (tol <= 2.0 ** -6 * ref.abs()).all()  # what the test allows is little next to the output
    assert ((lse.double() - rl).abs() <= 2.0 ** -14 * rl.abs()).all()


@pytest.mark.parametrize("weight", [0.99, 0.999])
@pytest.mark.parametrize("n,page,raised", [(32000, 64, 0), (131000, 128, 0), (32000, 16, 6)])
@pytest.mark.parametrize("n_heads,n_kv,d,n_new", [(8, 1, 128, 1), (4, 2, 64, 2), (24, 1, 128, 1), (64, 1, 128, 96)])
def test_attention_sink(ar, n_heads, n_kv, d, n_new, n, page, raised, weight):
    # raised by more, weights fall below what f16 holds to a bf16 step: by 2^4 earlier on tcgen05
    c, q = _sink(n, page, min(raised, 2) if n_new == 96 else raised, n_heads, n_kv, d, n_new, weight)
    cu, cud, ld = _index([n_new], [n])
    lse = torch.empty(n_new, n_heads, device="cuda")
    out = _attend(ar, c, q, cud, ld, n_new, lse=lse)
    tc = "attn_kv8_tc_kernel" in ar.ar_last_kernels()
    assert tc == (n_new == 96) and ar.ar_get_device_status() == ar.AR_OK
    _check_sink(c, q, n_new, out, lse, 11 if tc else 15)


@pytest.mark.parametrize("weight", [0.99, 0.999])
def test_attention_sink_of_a_batch(ar, weight):
    """The same cache read by so many sequences that a warp runs through nearly all of an item's keys."""
    n, S = 32000, 450
    c, q = _sink(n, 64, 0, 8, 4, 128, 1, weight)
    cu, cud, ld = _index([1] * S, [n] * S)
    lse = torch.empty(S, 8, device="cuda")
    one = c.table
    c.table, c.lens = np.repeat(one, S, 0), [n] * S
    out = _attend(ar, c, q.repeat(S, 1), cud, ld, 1, lse=lse)
    assert ar.ar_get_device_status() == ar.AR_OK
    c.table, c.lens = one, [n]
    _check_sink(c, q, 1, out, lse, 15)


@pytest.mark.parametrize("T,S,max_new,max_pages", [
    (131072, 1, 131072, 1024),  # a prompt of 131072 tokens
    (16384, 1, 16384, 1 << 13),  # a piece of a prompt, a page table of 2^20 tokens
    (32768, 4, 20000, 1 << 13),
    (16384 + 63, 64, 16384, 1 << 13),  # next to 63 single tokens
])
def test_attention_steps_do_not_bound_prompts(ar, T, S, max_new, max_pages):
    """The limit of mma.sync's list of steps is not a limit of what runs on tcgen05: the sizes pass the checks (the workspace's,
    which follows, refuses the call: nothing runs)."""
    assert ar.ar_attention_kv8_workspace(T, S, max_new, 64, 8, 128, 128, 1000, max_pages) > 0
    cfg, p = ar.Kv8Cfg(64, 8, 128, 128, 1000, max_pages), 0x100000
    st = ar.lib().ar_attention_kv8(ctypes.byref(cfg), p, T, p, p, p, S, max_new, 0.0, p, p, p, p, p, None, None, 0, None)
    assert st == ar.AR_ERR_WORKSPACE, ar.ar_last_error()


def test_attention_long_prompt(ar):
    """A whole prompt whose row tiles times the page table's width pass 2^31, on tcgen05; sampled rows of it."""
    n, n_heads, n_kv, d, page = 32768, 64, 8, 128, 128
    c = Cache([n], n_heads, n_kv, d, page, 2, garbage=False, max_pages=(1 << 20) // page)
    cu, cud, ld = _index([n], [n])
    q = torch.randn(n, n_heads * d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    out = _attend(ar, c, q, cud, ld, n)
    assert ar.ar_last_kernels() == "attn_kv8_tc_kernel" and ar.ar_get_device_status() == ar.AR_OK
    for t in (0, 1, 127, 128, 4095, 20001, n - 1):
        c.lens = [t + 1]
        ref, _, tol = _reference64(c, q[t:t + 1], 1, 11)
        assert ((out[t].double().view_as(ref) - ref).abs() <= tol).all()


@pytest.mark.parametrize("n_heads,n_kv,d,n_new,lens", [(8, 1, 128, 1, [60, 70]), (8, 2, 64, 1, [30000, 9]), (64, 8, 128, 200, [400, 333])])
def test_attention_lse_of_a_nan_row(ar, n_heads, n_kv, d, n_new, lens):
    """Rows without keys have a log-sum-exp of -inf; a row whose query is NaN has NaN, in one warp's item, in one that blocks
    share, and on tcgen05."""
    c = Cache(lens, n_heads, n_kv, d, 32, 2)
    cu, cud, ld = _index([n_new] * 2, lens)
    q = torch.from_numpy(c.rng.normal(size=(2 * n_new, n_heads * d)).astype(np.float32)).bfloat16().cuda()
    want = torch.empty(2 * n_new, n_heads, device="cuda")
    _attend(ar, c, q, cud, ld, n_new, lse=want)
    rows = [(0, 1), (n_new, n_heads - 1), (2 * n_new - 1, 0)]
    for t, h in rows:
        q[t, h * d + 7] = float("nan")
    lse = torch.empty_like(want)
    out = _attend(ar, c, q, cud, ld, n_new, lse=lse)
    for t, h in rows:
        assert lse[t, h].isnan() and out[t, h * d:(h + 1) * d].isnan().all()
        lse[t, h] = want[t, h]
    assert torch.equal(lse, want)


@pytest.mark.parametrize("top", [-4, 12, 45, 90, 115])
@pytest.mark.parametrize("order", ["zeros first", "zeros last", "between"])
@pytest.mark.parametrize("n_heads,n_kv,d,n_new,n,page", [(8, 2, 128, 1, 70, 16), (4, 2, 64, 1, 300, 32), (24, 1, 128, 1, 9000, 16), (32, 1, 64, 2, 500, 64),
                                                         (64, 2, 128, 160, 700, 16), (64, 4, 128, 2, 600, 128)])
def test_attention_pages_of_zeros_next_to_large_values(ar, n_heads, n_kv, d, n_new, n, page, order, top):
    """Pages of zero values, whose scale is the smallest there is, in front of, behind and between pages of large ones: their
    keys count in the row sum."""
    c = Cache([n], n_heads, n_kv, d, page, n + top)
    pages = -(-n // page)
    zero = {"zeros first": lambda i: i < pages // 2, "zeros last": lambda i: i >= pages // 2, "between": lambda i: i % 3 == 1}[order]
    c.ks[:] = 127 - 7
    for i in range(pages):
        pg = c.table[0, i]
        c.vs[pg] = 127 - 100 if zero(i) else 127 + top - i % 2
        if zero(i):
            c.v[pg] = 0
        else:
            c.v[pg] = L.e4m3_codes(c.rng.uniform(1, 16, c.v[pg].shape))
    if n % page:
        c.v[c.table[0, pages - 1], :, n % page:] = 0x7F
    q = torch.from_numpy(c.rng.normal(size=(n_new, n_heads * d)).astype(np.float32)).bfloat16().cuda()
    q[0] = 0  # all keys alike
    cu, cud, ld = _index([n_new], [n])
    lse = torch.empty(n_new, n_heads, device="cuda")
    out = _attend(ar, c, q, cud, ld, n_new, lse=lse)
    assert ("attn_kv8_tc_kernel" in ar.ar_last_kernels()) == (n_new == 160) and ar.ar_get_device_status() == ar.AR_OK
    ref, rl, tol = _reference64(c, q, n_new, 11 if n_new == 160 else 15)
    got = out.double().view_as(ref)
    assert ((got - ref).abs() <= tol).all(), (((got - ref).abs() / tol).max().item(), got[0, 0, :3], ref[0, 0, :3])
    assert ((lse.double() - rl).abs() <= 2.0 ** -14 * (1 + rl.abs())).all()
