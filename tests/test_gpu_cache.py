"""GPU parity of the 4-bit key/value cache through the ABI against plain forms in 64 bits (tests/cache_forms.py).

Block tables and slots, codes and scales are whole numbers and compared exactly; attention and the merge within the
bounds derived at cache_forms.tolerances and below.
"""
import math
import os

import numpy as np
import pytest
import torch

import block_sparse_video_gather_b200 as vsa
from block_sparse_video_gather_b200 import build as vsa_build
from tests import cache_forms as F

pytestmark = pytest.mark.gpu

TDT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    vsa_build.build()
    vsa.lib()


@pytest.fixture(autouse=True)
def _status():
    assert vsa.get_status() == vsa.VSA_OK
    yield
    assert vsa.get_status() == vsa.VSA_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# Block tables and slots
# ---------------------------------------------------------------------------


def _run_tables(kv, new, page, n_free, start, max_pages, max_tokens, seed=0):
    rng = np.random.default_rng(seed)
    R = len(kv)
    free = rng.permutation(n_free + 7)[:n_free].astype(np.int32) if n_free else np.zeros(0, np.int32)
    table = rng.integers(0, 5000, (R, max_pages)).astype(np.int32)
    guard = 8
    slots = torch.full((max_tokens + guard,), -77, dtype=torch.int32, device="cuda")
    t = i32(table)
    buf = i32(np.append(free, [9]))  # never an empty tensor
    out = vsa.cache_tables(i32(kv), i32(new), page, buf[:n_free], i32([start]), t,
                           slots[:max_tokens])
    torch.cuda.synchronize()
    want = F.tables(np.asarray(kv), np.asarray(new), page, free, start, table,
                    max_tokens)
    got = [x.cpu().numpy() for x in out] + [slots.cpu().numpy(), t.cpu().numpy()]
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    assert got[2][0] == want[3]
    np.testing.assert_array_equal(got[3][:max_tokens], want[2])
    assert np.all(got[3][max_tokens:] == -77)
    np.testing.assert_array_equal(got[4], want[4])
    return want[5]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("R", [1, 2, 33, 513, 4096])
def test_tables(page, R):
    rng = np.random.default_rng(R * page)
    kv, new = rng.integers(0, 4 * page, R), rng.integers(0, 3 * page, R)
    kv[rng.random(R) < 0.3] //= page
    kv[rng.random(R) < 0.2] *= 0
    kv[rng.random(R) < 0.2] = 2 * page  # pages that are just full
    new[rng.random(R) < 0.3] = 0
    new[rng.random(R) < 0.2] = page
    tokens = int(new.sum())
    assert _run_tables(kv, new, page, 3 * R + 4 * R, 5, 12, tokens + 5) == []


def test_tables_of_one_long_request_and_of_none_new():
    assert _run_tables([0], [32760], 64, 600, 0, 512, 32760) == []
    assert _run_tables([16], [16], 16, 3, 2, 2, 16) == []
    assert _run_tables([100, 0, 3], [0, 0, 0], 16, 4, 4, 7, 0) == []
    assert _run_tables([100, 0, 3], [0, 0, 0], 16, 4, 4, 7, 3) == []


@pytest.mark.parametrize("kv,new,n_free,start,max_pages,max_tokens,refused", [
    ([5, -1, 40], [3, 4, 5], 20, 0, 8, 20, [1]),                 # a negative length
    ([5, 6, 40], [3, -4, 5], 20, 0, 8, 20, [1]),
    ([5, 120, 40], [3, 9, 5], 20, 0, 8, 20, [1]),                # past its row of the table
    ([15, 15, 15, 16], [2, 2, 1, 2], 13, 10, 8, 20, []),         # the last pages
    ([15, 15, 15, 16, 1], [2, 2, 1, 2, 60], 12, 10, 8, 80, [3, 4]),  # no page left for the fourth; the third needs none
    ([15, 15, 15, 16, 1], [2, 60, 1, 2, 2], 12, 10, 8, 80, [1, 3]),  # a large one is refused, and each later one with need
    ([5, 5, 5], [3, 9, 5], 20, 0, 8, 11, [1, 2]),                # tokens past the batch
    ([5, 5, 5], [3, 9, 0], 20, 0, 8, 11, [1, 2]),
    ([5, 5], [3, 2000000000], 20, 0, 8, 11, [1]),
    ([5, 5], [3, 30], 20, 21, 8, 40, [1]),                       # a stack pointer past the stack
    ([2147483647, 5], [2147483647, 3], 20, 0, 8, 20, [0, 1]),
])
def test_tables_refuse_what_does_not_fit(kv, new, n_free, start, max_pages, max_tokens, refused):
    got = _run_tables(kv, new, 16, n_free, start, max_pages, max_tokens)
    assert got == refused
    assert vsa.get_status() == (vsa.VSA_ERR_CAPACITY if refused else vsa.VSA_OK)


@pytest.mark.parametrize("R", [1, 7, 700])
def test_release_gives_pages_back(R):
    rng = np.random.default_rng(R)
    page, max_pages = 16, 9
    kv = rng.integers(0, max_pages * page + 1, R)
    used = -(-kv // page)
    n = int(used.sum()) + 6
    free = rng.permutation(n).astype(np.int32)
    table = np.full((R, max_pages), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :used[r]] = free[at:at + used[r]]
        at += used[r]
    drop = rng.random(R) < 0.5
    drop[0] = True
    want_kv = np.where(drop, 0, kv)
    back = np.concatenate([table[r, :used[r]] for r in range(R) if drop[r]] + [np.zeros(0, np.int32)])
    d_kv, d_free, d_start = i32(kv), i32(free), i32([at])
    vsa.cache_release(torch.from_numpy(drop).cuda(), page, d_kv, i32(table), d_free, d_start)
    np.testing.assert_array_equal(d_kv.cpu().numpy(), want_kv)
    assert int(d_start) == at - len(back)
    got = d_free.cpu().numpy()
    np.testing.assert_array_equal(got[at - len(back):at], back)
    np.testing.assert_array_equal(got[at:], free[at:])
    np.testing.assert_array_equal(got[:at - len(back)], free[:at - len(back)])


def test_release_refuses_more_pages_than_are_out():
    kv, free, start = i32([40, 3]), i32(np.arange(9)), i32([2])
    vsa.cache_release(i32([1, 1]).to(torch.uint8), 16, kv, i32([[1, 2, 3], [4, 5, 6]]), free, start)
    assert kv.tolist() == [40, 3] and start.tolist() == [2] and free.tolist() == list(range(9))
    assert vsa.get_status() == vsa.VSA_ERR_CAPACITY


# ---------------------------------------------------------------------------
# Append and read back
# ---------------------------------------------------------------------------


def _tokens(rng, T, H, dtype, kind="normal"):
    x = rng.standard_normal((T, 2, H, 128)).astype(np.float32)
    if kind == "wide":
        x *= np.exp2(rng.integers(-24, 12, (T, 2, H, 1)))
        x[..., :16] = 0
        x[..., 16:32] *= 2.0**-20
    x = torch.from_numpy(x).to(TDT[dtype])
    return x[:, 0], x[:, 1]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,page,kind", [(1, 1, 16, "normal"), (5, 3, 32, "wide"), (33, 12, 16, "normal"),
                                           (100, 5, 64, "wide"), (300, 2, 256, "normal"), (17, 24, 128, "wide")])
def test_append_and_read(T, H, page, kind, dtype):
    rng = np.random.default_rng(T)
    n = -(-T // page) + 2
    k, v = _tokens(rng, T, H, dtype, kind)
    slots = rng.permutation(n * page)[:T]
    slots[rng.random(T) < 0.1] = -1
    before = rng.integers(0, 256, (n, H, page // 16, F.REC)).astype(np.uint8)
    pages = torch.from_numpy(before).cuda()
    # a slice of a wider row, as out of a fused projection
    wide = torch.zeros((T, 3, H, 128), dtype=TDT[dtype], device="cuda")
    wide[:, 1], wide[:, 2] = k.cuda(), v.cuda()
    vsa.cache_append(wide[:, 1], wide[:, 2], i32(slots), pages)
    want = before.copy()
    F.put(want, slots, f64(k), f64(v))
    np.testing.assert_array_equal(pages.cpu().numpy(), want)  # every other byte as it was
    ko = torch.full((T, H, 128), 7.0, dtype=TDT[dtype], device="cuda")
    vo = ko.clone()
    vsa.cache_read(i32(slots), pages, k_out=ko, v_out=vo)
    wk, wv = np.full((2, T, H, 128), 7.0)
    wk[slots >= 0], wv[slots >= 0] = F.get(want, slots[slots >= 0])
    np.testing.assert_array_equal(f64(ko), wk)
    np.testing.assert_array_equal(f64(vo), wv)


def test_append_saturates_and_stores_no_nan():
    x = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    x[0, 0, 0], x[0, 0, 16], x[0, 0, 32], x[0, 0, 33] = float("inf"), float("nan"), 1e30, -1.0
    pages = vsa.cache_pages(1, 1, 16).fill_(0xFF)
    vsa.cache_append(x.cuda(), x.cuda(), i32([3]), pages)
    k, v = vsa.cache_read(i32([3]), pages)
    for y in (k, v):
        y = f64(y)[0, 0]
        assert y[0] == 2688 and y[32] == 2688 and np.all(np.isfinite(y)) and np.all(y[48:] == 0)


def test_append_and_read_out_of_range_slots():
    pages = torch.zeros((2, 2, 1, F.REC), dtype=torch.uint8, device="cuda")
    k = torch.ones((3, 2, 128), dtype=torch.float16, device="cuda")
    slots = i32([32, 31, 2147483647])
    vsa.cache_append(k, k, slots, pages)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    want = np.zeros((2, 2, 1, F.REC), np.uint8)
    F.put(want, [-1, 31, -1], f64(k), f64(k))
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    ko, vo = vsa.cache_read(slots, pages, torch.float16)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    wk, _ = F.get(want, [31])
    for y in (f64(ko), f64(vo)):
        np.testing.assert_array_equal(y[1], wk[0])
        assert not y[0].any() and not y[2].any()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------


class Batch:
    """A batch of requests with n[r] new tokens over kv[r] cached ones, in shuffled pages whose other bytes are 0xFF
    (scales of NaN)."""

    def __init__(self, n, kv, Hq, Hkv, page, dtype, seed=0, q_scale=1.0, spare=3, pad_rows=0, extra_pages=2):
        rng = np.random.default_rng(seed)
        R = len(n)
        self.n, self.kv, self.Hq, self.Hkv, self.page, self.dtype = n, kv, Hq, Hkv, page, dtype
        per = [-(-L // page) for L in kv]
        self.M = max(per + [1]) + extra_pages
        order = rng.permutation(sum(per) + spare)
        self.table = np.full((R, self.M), -5, np.int32)  # entries past the last page are not read
        at = 0
        for r in range(R):
            self.table[r, :per[r]] = order[at:at + per[r]]
            at += per[r]
        self.pages = torch.full((sum(per) + spare, Hkv, page // 16, F.REC), 255, dtype=torch.uint8, device="cuda")
        slots = np.concatenate([self.table[r, np.arange(kv[r]) // page].astype(np.int64) * page
                                + np.arange(kv[r]) % page for r in range(R)] + [np.zeros(0, np.int64)])
        T = int(sum(kv))
        x = torch.from_numpy(rng.standard_normal((max(T, 1), 2, Hkv, 128)).astype(np.float32)).to(TDT[dtype]).cuda()
        x[:, 0] += x[:1, 0]  # keys with a common part
        if T:
            vsa.cache_append(x[:T, 0], x[:T, 1], i32(slots), self.pages)
        kc, ks = F.quantise(f64(x[:T, 0]))
        vc, vs = F.quantise(f64(x[:T, 1]))
        k, v = F.values(kc, ks), F.values(vc, vs)
        cut = np.cumsum([0] + list(kv))
        self.k = [k[cut[r]:cut[r + 1]] for r in range(R)]
        self.v = [v[cut[r]:cut[r + 1]] for r in range(R)]
        self.cu = np.cumsum([0] + list(n))
        self.T = int(self.cu[-1]) + pad_rows
        q = rng.standard_normal((max(self.T, 1), 3, Hq, 128)).astype(np.float32) * q_scale
        self.qkv = torch.from_numpy(q).to(TDT[dtype]).cuda()
        self.q = self.qkv[:self.T, 0]  # strided
        self.ws = vsa.cache_workspace(max(list(n) + [1]), Hq, Hkv)

    def run(self, causal, max_q=None, ws=None):
        o = torch.full((self.T, self.Hq, 128), 3.0, dtype=TDT[self.dtype], device="cuda")
        lse = torch.full((self.T, self.Hq), 3.0, device="cuda")
        vsa.cache_attn(self.q, i32(self.cu), i32(self.kv), i32(self.table), self.pages, max_q or max(list(self.n) + [1]),
                       self.ws if ws is None else ws, causal=causal, o_out=o, lse_out=lse)
        torch.cuda.synchronize()
        return o, lse

    def check(self, o, lse, causal, live=None, heads=None):
        o, lse, q = f64(o), f64(lse), f64(self.q)
        for r in range(len(self.n)):
            a, b = self.cu[r], self.cu[r + 1]
            n, L = self.n[r], self.kv[r]
            limit = np.arange(n) + L - n + 1 if causal else np.full(n, L)
            for h in heads if heads is not None else range(self.Hq):
                g = h // (self.Hq // self.Hkv)
                k, v = self.k[r][:, g], self.v[r][:, g]
                eo, el, spread, reach = F.attention(q[a:b, h], k, v, limit, None if live is None else live[r])
                to, tl = F.tolerances(eo, el, spread, reach, L, np.abs(v).max(initial=0.0), self.dtype)
                inf = np.isinf(el)
                np.testing.assert_array_equal(np.isneginf(lse[a:b, h]), inf)
                assert np.all(o[a:b, h][inf] == 0)
                assert np.all(np.abs(o[a:b, h] - eo) <= to), (r, h, np.max(np.abs(o[a:b, h] - eo) - to))
                assert np.all(np.abs(lse[a:b, h] - el)[~inf] <= tl[~inf]), (r, h, np.abs(lse[a:b, h] - el)[~inf].max())
        # rows outside every request are left as they were
        assert np.all(o[self.cu[-1]:] == 3.0) and np.all(lse[self.cu[-1]:] == 3.0)


SHAPES = [
    # n, kv, Hq, Hkv, page
    ([1], [1], 1, 1, 16),
    ([1], [17], 2, 1, 16),
    ([1], [777], 12, 12, 64),
    ([1, 1, 1], [0, 33, 300], 4, 2, 16),
    ([1] * 9, [1, 15, 16, 17, 255, 256, 257, 1000, 31], 8, 1, 32),
    ([3, 0, 1, 5], [40, 50, 1, 500], 6, 3, 16),
    ([2, 4], [2, 4], 24, 2, 128),
    ([8, 7], [100, 2000], 3, 3, 256),
    ([16, 1, 33], [900, 64, 33], 4, 4, 64),
    ([5, 2], [3, 300], 8, 2, 16),       # more new tokens than cached ones: rows that see nothing when causal
    ([64], [640], 5, 1, 16),
    ([130], [1000], 2, 2, 64),
    ([257, 3, 128], [700, 400, 128], 4, 2, 32),
    ([1000], [1000], 3, 1, 16),
    ([300], [129], 2, 1, 64),           # causal rows that see nothing, over more than one tile
    ([90, 40, 1], [2048, 1, 0], 12, 4, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{len(s[0])}x{max(s[0])}on{max(s[1])}h{s[2]}-{s[3]}p{s[4]}" for s in SHAPES])
def test_attention(shape, causal, dtype):
    b = Batch(*shape, dtype, pad_rows=2)
    o, lse = b.run(causal)
    b.check(o, lse, causal)
    # a bound on the new tokens that is not the largest only changes the kernel
    o2, lse2 = b.run(causal, max_q=1)
    b.check(o2, lse2, causal)
    # the same call again: the same bits, and the workspace is ready for it
    o3, lse3 = b.run(causal)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_attention_of_fewer_tokens_than_the_bound():
    """The bound on the new tokens selects the kernel; one request, and several, with far fewer than it says."""
    for n, kv in (([1], [500]), ([3], [2]), ([1, 30, 0], [500, 40, 7])):
        b = Batch(n, kv, 6, 2, 32, "bf16")
        b.ws = vsa.cache_workspace(2000, 6, 2)
        b.check(*b.run(True, max_q=2000), True)


@pytest.mark.parametrize("n,kv,Hq,Hkv,page", [([1], [30011], 2, 1, 256), ([1, 2], [9000, 20000], 8, 2, 16),
                                              ([200], [12345], 2, 1, 64), ([3], [16000], 4, 4, 64),
                                              ([40, 1, 513], [5000, 9000, 4097], 2, 1, 32)])
def test_attention_over_long_caches(n, kv, Hq, Hkv, page):
    b = Batch(n, kv, Hq, Hkv, page, "bf16", seed=5)
    b.check(*b.run(True), True)
    b.check(*b.run(False), False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,kv", [([1] * 50, [0, 1, 40, 90] * 12 + [7, 16]), ([60, 2, 0, 1] * 11, [60, 130, 5, 0] * 11),
                                  ([100], [0]), ([70, 70], [0, 33])])
def test_attention_of_many_requests_and_of_empty_ones(n, kv, causal):
    """More requests than a warp has lanes, on either kernel and on both, and requests without a cached token."""
    b = Batch(n, kv, 2, 1, 16, "f16", pad_rows=1)
    b.check(*b.run(causal), causal)


def test_attention_of_the_most_requests():
    R = 4096
    rng = np.random.default_rng(9)
    b = Batch([1] * R, list(rng.integers(0, 40, R)), 1, 1, 16, "bf16")
    b.check(*b.run(True), True)
    n = [1] * R
    n[7], n[4095] = 70, 50
    b = Batch(n, list(np.maximum(n, rng.integers(0, 40, R))), 1, 1, 16, "bf16")
    b.check(*b.run(True), True)


@pytest.mark.parametrize("n", [1, 64])
def test_attention_after_a_workspace_that_was_not_zero(n):
    """Counters that were not zero join an item early or not at all -- wrong rows, no hang -- and once the workspace
    is zeroed again the results are right."""
    b = Batch([n], [6000], 1, 1, 64, "bf16")
    good = b.run(False)
    b.ws.view(torch.int32)[:1024] = 5
    b.run(False)
    b.ws.zero_()
    o, lse = b.run(False)
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_of_every_scale(dtype):
    """Blocks whose largest value makes each of E4M3's scales, and values at the borders between codes."""
    x = np.zeros((127, 1, 128), np.float32)
    steps = np.array([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6], np.float32)
    for b in range(127):
        x[b, 0, 0:15] = steps * F.E4M3[b]
        x[b, 0, 16:31] = -steps * F.E4M3[b]
        x[b, 0, 32:128] = np.random.default_rng(b).uniform(-6, 6, 96) * F.E4M3[b]
    k = torch.from_numpy(x).to(TDT[dtype]).cuda()
    pages = torch.zeros((8, 1, 1, F.REC), dtype=torch.uint8, device="cuda")
    vsa.cache_append(k, -k, i32(np.arange(127)), pages)
    want = np.zeros((8, 1, 1, F.REC), np.uint8)
    F.put(want, np.arange(127), f64(k), f64(-k))
    np.testing.assert_array_equal(pages.cpu().numpy(), want)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 3e4])
@pytest.mark.parametrize("n", [1, 100])
def test_attention_of_small_and_large_queries(scale, n):
    b = Batch([n], [300], 2, 1, 16, "bf16", q_scale=scale)
    b.check(*b.run(False), False)


@pytest.mark.parametrize("n", [1, 70])
def test_attention_of_queries_that_are_not_finite(n):
    """A query row with an infinity or a NaN gives NaN in its own row only."""
    b = Batch([n, 2], [100, 50], 2, 1, 16, "bf16")
    clean = b.run(False)[0]
    b.q[0, 0, 5] = float("inf")
    b.q[n, 1, 6] = float("nan")
    o, lse = b.run(False)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(o[n, 1]).all()
    keep = torch.ones(o.shape[:2], dtype=torch.bool)
    keep[0, 0] = keep[n, 1] = False
    assert torch.equal(o[keep.cuda()], clean[keep.cuda()])


@pytest.mark.parametrize("n", [1, 5, 200])
def test_attention_leaves_bad_pages_out(n):
    b = Batch([n, n], [200, 333], 4, 2, 32, "f16")
    b.table[0, 2], b.table[1, 0], b.table[1, 10] = -1, b.pages.shape[0], 2147483647
    o, lse = b.run(False)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    live = [np.ones(200, bool), np.ones(333, bool)]
    live[0][64:96] = False
    live[1][:32] = live[1][320:] = False
    b.check(o, lse, False, live)


@pytest.mark.parametrize("n", [1, 100])
def test_attention_of_a_request_whose_pages_are_all_bad(n):
    b = Batch([n, 1], [60, 20], 2, 2, 16, "bf16")
    b.table[0] = -1
    o, lse = b.run(True)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    b.check(o, lse, True, [np.zeros(60, bool), np.ones(20, bool)])


def test_attention_cuts_lengths_and_offsets():
    b = Batch([2, 3], [64, 32], 2, 1, 16, "bf16", extra_pages=0)
    good = b.run(False)
    b.kv[0] = 10**6  # past the table's four pages
    o, lse = b.run(False)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    b.kv[0] = 64
    b.cu = np.array([0, 2, 99])  # past the batch
    o, lse = b.run(False)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    assert torch.equal(o, good[0])
    b.cu = np.array([0, 2, 1])  # not ascending: the second request has no token
    o, lse = b.run(False)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    assert torch.equal(o[:2], good[0][:2]) and float(o[2:].float().min()) == 3.0
    b.kv[1] = -7
    b.cu = np.array([0, 2, 5])
    o, lse = b.run(False)
    assert vsa.get_status() == vsa.VSA_ERR_BAD_INDEX
    assert torch.equal(o[:2], good[0][:2]) and float(o[2:].float().abs().max()) == 0.0
    assert torch.isneginf(lse[2:]).all()


@pytest.mark.parametrize("n", [[1] * 40, [150, 1, 30]])
def test_attention_captured_and_replayed_with_other_lengths(n):
    """Two graphs that share a workspace, replayed in turn with lengths changed in place."""
    R = len(n)
    b = Batch(n, [300] * R, 4, 2, 32, "bf16")
    cu, kv, table = i32(b.cu), i32(b.kv), i32(b.table)
    outs = [(torch.empty((b.T, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((b.T, 4), device="cuda"))
            for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    for causal, (o, lse) in zip((True, False), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            vsa.cache_attn(b.q, cu, kv, table, b.pages, max(n), b.ws, causal=causal, o_out=o, lse_out=lse)
        graphs.append(g)
    rng = np.random.default_rng(1)
    for _ in range(3):
        b.kv = [int(x) for x in rng.integers(150, 301, R)]
        k, v = b.k, b.v
        b.k, b.v = [x[:L] for x, L in zip(k, b.kv)], [x[:L] for x, L in zip(v, b.kv)]
        kv.copy_(i32(b.kv))
        for causal, g, (o, lse) in zip((True, False), graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            b.check(o, lse, causal, heads=[0, 3])
        b.k, b.v = k, v


def test_attention_on_two_streams_with_a_workspace_each():
    big = Batch([1] * 20, [3000] * 20, 8, 2, 64, "bf16")
    b = Batch([130], [2000], 8, 2, 64, "bf16", seed=3)
    want = [x.run(True) for x in (big, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, (x, s) in enumerate(zip((big, b), streams)):
            with torch.cuda.stream(s):
                got[i].append(vsa.cache_attn(x.q, i32(x.cu), i32(x.kv), i32(x.table), x.pages, max(x.n), x.ws))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_empty_calls():
    b = Batch([1], [5], 2, 1, 16, "bf16")
    o, lse = vsa.cache_attn(b.q[:0], i32([0, 0]), i32([5]), i32(b.table), b.pages, 1, b.ws)
    assert o.shape == (0, 2, 128) and lse.shape == (0, 2)
    vsa.cache_append(b.q[:0, :1], b.q[:0, :1], i32([]), b.pages)


def test_a_record_past_the_32_bit_offset():
    """Pages of more than 2^32 bytes: the last page's tokens are found."""
    Hkv, page = 24, 256
    n = (1 << 32) // (Hkv * page * 144) + 2
    pages = vsa.cache_pages(n, Hkv, page)
    k = torch.randn((300, Hkv, 128), device="cuda").to(torch.bfloat16)
    table = i32([[n - 1, 0]])
    slots = torch.cat([torch.arange((n - 1) * page, n * page), torch.arange(44)]).int().cuda()
    vsa.cache_append(k, k, slots, pages)
    rk, rv = vsa.cache_read(slots, pages)
    np.testing.assert_array_equal(f64(rk), F.values(*F.quantise(f64(k))))
    for m in (1, 129):
        q = torch.randn((m, Hkv, 128), device="cuda").to(torch.bfloat16)
        o, lse = vsa.cache_attn(q, i32([0, m]), i32([300]), table, pages, m, vsa.cache_workspace(m, Hkv, Hkv), causal=False)
        for h in (0, 23):
            v = f64(rk[:, h])
            eo, el, spread, reach = F.attention(f64(q[:, h]), v, v, [300] * m)
            to, tl = F.tolerances(eo, el, spread, reach, 300, np.abs(v).max(), "bf16")
            assert np.all(np.abs(f64(o[:, h]) - eo) <= to) and np.all(np.abs(f64(lse[:, h]) - el) <= tl)


# ---------------------------------------------------------------------------
# The merge
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("grid,block,prefix,B,H", [((4, 8, 8), (4, 8, 8), 0, 1, 1), ((5, 9, 11), (4, 8, 8), 0, 2, 3),
                                                   ((4, 8, 12), (4, 4, 4), 70, 1, 2)])
def test_untile_merge(grid, block, prefix, B, H, dtype):
    """One weight is off by a few fp32 roundings (exp, sum, quotient: below 2^-20), the sum by as much, then o is
    rounded once; lse is off by expf and logf, below 2^-20 (1 + |lse|)."""
    rng = np.random.default_rng(3)
    plan = vsa.Plan(*grid, block=block, n_prefix=prefix)
    past = torch.from_numpy(rng.standard_normal((B, plan.S, H, 128)).astype(np.float32)).to(TDT[dtype]).cuda()
    fine = torch.from_numpy(rng.standard_normal((B, plan.S, H, 128)).astype(np.float32)).to(TDT[dtype]).cuda()
    l1, l2 = (torch.from_numpy(rng.normal(3, 20, (B, plan.S, H)).astype(np.float32)).cuda() for _ in range(2))
    l1[torch.rand(l1.shape, device="cuda") < 0.2] = -np.inf
    l2[torch.rand(l2.shape, device="cuda") < 0.2] = -np.inf
    l1[:, :40] = l2[:, :40] + 0.5
    past[torch.isneginf(l2)] = float("nan")  # not used
    ot = vsa.tile(plan, fine)
    lt = vsa.tile(plan, l1.to(torch.float16)[..., None].expand(-1, -1, -1, 128).contiguous())[..., 0].float()
    l1 = l1.to(torch.float16).float()  # what the tiling above carried
    o, lse = vsa.untile_merge(plan, ot, lt.contiguous(), past, l2)
    a, b = f64(l1), f64(l2)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.maximum(a, b)
        el = np.where(np.isneginf(m), -np.inf, m + np.log(np.exp(a - m) + np.exp(b - m)))
        w1, w2 = (np.where(np.isneginf(x), 0.0, np.exp(x - el)) for x in (a, b))
    p = np.where(np.isneginf(b)[..., None], 0.0, f64(past))
    f = f64(fine)
    eo = w1[..., None] * f + w2[..., None] * p
    slack = 2.0**-20 * (w1[..., None] * np.abs(f) + w2[..., None] * np.abs(p))
    half = 2.0**-8 if dtype == "bf16" else 2.0**-11
    assert np.all(np.abs(f64(o) - eo) <= slack + half * (np.abs(eo) + slack) + 2.0**-25)
    got = f64(lse)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(el))
    fin = ~np.isneginf(el)
    assert np.all(np.abs(got - el)[fin] <= 2.0**-20 * (1 + np.abs(el[fin])))
    # in place, and without the lse
    o2, lse2 = past.clone(), l2.clone()
    vsa.untile_merge(plan, ot, lt.contiguous(), o2, lse2, out=o2, lse_out=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chunks_of_a_video(dtype):
    """Three chunks: each attends to itself with every block selected and to the cached chunks before it; the result
    is dense attention over the current chunk's keys and the earlier ones' quantised keys."""
    rng = np.random.default_rng(11)
    plan, B, H = vsa.Plan(4, 9, 10), 2, 3
    fwd = vsa.Forward(plan, B, H, plan.NB, dtype=TDT[dtype])
    cache = vsa.KVCache(num_pages=64, Hq=H, max_requests=B, max_len=3 * plan.S, page_tokens=64, max_q=plan.S)
    past = [[np.zeros((0, H, 128))] * 2 for _ in range(B)]
    for chunk in range(3):
        q, k, v = (torch.from_numpy(rng.standard_normal((B, plan.S, H, 128)).astype(np.float32)).to(TDT[dtype]).cuda()
                   for _ in range(3))
        o, lse = fwd(q, k, v, past=cache.attend_chunk(q))
        slots = cache.reserve(i32([plan.S] * B), B * plan.S)
        cache.append(k.view(-1, H, 128), v.view(-1, H, 128))
        assert cache.kv_len.tolist() == [(chunk + 1) * plan.S] * B
        rk, rv = (f64(x).reshape(B, plan.S, H, 128) for x in vsa.cache_read(slots, cache.pages, TDT[dtype]))
        for b in range(B):
            for h in range(H):
                ks = np.concatenate([past[b][0][:, h], f64(k[b, :, h])])
                vs = np.concatenate([past[b][1][:, h], f64(v[b, :, h])])
                eo, el, spread, reach = F.attention(f64(q[b, :, h]), ks, vs, [len(ks)] * plan.S)
                to, tl = F.tolerances(eo, el, spread, reach, len(ks), np.abs(vs).max(), dtype)
                # each part is rounded to its type before the merge, and bf16 numerators to 2^-8 of themselves (both
                # at most `half` of the spread), and the weights come from two lse: 2 tl more
                half = 2.0**-8 if dtype == "bf16" else 2.0**-11
                to = to + (2 * half + 2 * tl[:, None]) * spread
                assert np.all(np.abs(f64(o[b, :, h]) - eo) <= to)
                assert np.all(np.abs(f64(lse[b, :, h]) - el) <= 2 * tl)
            past[b] = [np.concatenate([past[b][0], rk[b]]), np.concatenate([past[b][1], rv[b]])]
    with pytest.raises(ValueError, match="max_q"):
        vsa.KVCache(num_pages=4, Hq=H, max_requests=B).attend_chunk(q)
    with pytest.raises(ValueError, match="past"):
        vsa.Forward(plan, B, H, 2, gated=True, dtype=TDT[dtype])(q, k, v, gate=q, past=cache.attend_chunk(q))


def test_steps_of_a_serving_loop():
    """Prompts in, tokens one at a time from a captured step, a request out, its pages used again."""
    rng = np.random.default_rng(2)
    R, Hq, Hkv = 3, 4, 2
    cache = vsa.KVCache(num_pages=20, Hq=Hq, Hkv=Hkv, max_requests=R, max_len=160, page_tokens=16, max_q=40)
    kept = [np.zeros((2, 0, Hkv, 128)) for _ in range(R)]

    def rand(T, H):
        return torch.from_numpy(rng.standard_normal((T, H, 128)).astype(np.float32)).to(torch.bfloat16).cuda()

    def step(new, q, k, v, go):
        o, lse = go()
        cu = np.cumsum([0] + new)
        kq, vq = (F.values(*F.quantise(f64(x))) for x in (k, v))
        for r in range(R):
            a, b = cu[r], cu[r + 1]
            kept[r] = np.concatenate([kept[r], np.stack([kq[a:b], vq[a:b]])], 1)
            L, n = kept[r].shape[1], new[r]
            for h in range(Hq):
                kk, vv = kept[r][:, :, h // 2]
                eo, el, spread, reach = F.attention(f64(q[a:b, h]), kk, vv, np.arange(n) + L - n + 1)
                to, tl = F.tolerances(eo, el, spread, reach, L, np.abs(vv).max(initial=0.0), "bf16")
                assert np.all(np.abs(f64(o[a:b, h]) - eo) <= to)
                assert np.all(np.abs(f64(lse[a:b, h]) - el) <= tl)
        assert cache.kv_len.tolist() == [x.shape[1] for x in kept]

    def eager(new, q, k, v):
        def go():
            cache.reserve(i32(new), q.shape[0])
            cache.append(k, v)
            return cache.attend(q)
        step(new, q, k, v, go)

    eager([40, 17, 0], rand(60, Hq), rand(60, Hkv), rand(60, Hkv))  # three rows of padding
    q, k, v, one = rand(R, Hq), rand(R, Hkv), rand(R, Hkv), i32([1] * R)
    o, lse = torch.empty_like(q), torch.empty((R, Hq), device="cuda")
    cache.reserve(i32([0] * R), R)  # makes the step's slots outside the capture
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cache.reserve(one, R)
        cache.append(k, v)
        cache.attend(q, o_out=o, lse_out=lse)

    def replay():
        g.replay()
        return o, lse

    for i in range(20):
        for x, H in ((q, Hq), (k, Hkv), (v, Hkv)):
            x.copy_(rand(R, H))
        step([1] * R, q, k, v, replay)
    cache.release(i32([1, 0, 0]).bool())
    kept[0] = kept[0][:, :0]
    used = sum(-(-x.shape[1] // 16) for x in kept)
    assert int(cache.free_start) == used
    eager([33, 1, 2], rand(36, Hq), rand(36, Hkv), rand(36, Hkv))
    pages = np.concatenate([cache.table[r, :-(-kept[r].shape[1] // 16)].cpu().numpy() for r in range(R)])
    assert len(set(pages.tolist())) == len(pages)


# ---------------------------------------------------------------------------
# One dominant key before a long tail
# ---------------------------------------------------------------------------


def _attend_shared(q, kv, page, pages, table, ws_q):
    """Requests of the rows of q [R, n, Hq, 128] over the same cached tokens."""
    R, n, Hq = q.shape[:3]
    ws = vsa.cache_workspace(ws_q, Hq, pages.shape[1])
    return vsa.cache_attn(q.reshape(R * n, Hq, 128), i32(np.arange(R + 1) * n), i32([kv] * R), table, pages, ws_q, ws,
                          causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("where", [0, 1500, 29999])
@pytest.mark.parametrize("R,n,Hq", [(2368, 1, 1), (1184, 1, 16), (1, 256, 148)],
                         ids=["one row", "16 rows", "256-row tiles"])
def test_attention_of_a_dominant_key_and_its_tail(R, n, Hq, where, dtype):
    """One key of score 17.5 and value 0, all others of score 0 and value 6: each weighs 2^-25.2 of the first, together
    they are the whole output.  As many items as warps (or CTAs), so that the workers that hold the dominant key hold
    most of an item's tail too.

    A numerator is off by 2^-11 of itself, or by 2^-32 of the largest where fp16 holds it as a subnormal (the largest
    is between 2^7 and 2^15, the subnormal half step 2^-25); the other terms are those of cache_forms.tolerances."""
    L, page = 30000, 64
    k = torch.zeros((L, 1, 128), dtype=TDT[dtype])
    v = torch.full((L, 1, 128), 6.0, dtype=TDT[dtype])
    k[where, 0, 0], v[where] = 6.0, 0.0
    n_pages = -(-L // page)
    pages = vsa.cache_pages(n_pages, 1, page)
    vsa.cache_append(k.cuda(), v.cuda(), i32(np.arange(L)), pages)
    table = i32(np.tile(np.arange(n_pages), (R, 1)))
    q = torch.zeros((R, n, Hq, 128), dtype=TDT[dtype], device="cuda")
    q[..., 0] = 33.0
    o, lse = _attend_shared(q, L, page, pages, table, n)
    eo, el, spread, reach = F.attention(f64(q[0, 0, :1]), f64(k[:, 0]), f64(v[:, 0]), [L])
    assert 2.0**-26 < math.exp(-33 * 6 / math.sqrt(128)) < 2.0**-25
    score = 2.0**-17 * reach[0] + 2.0**-22 * (1 + abs(el[0]))
    sums = L * 2.0**-24 + 2.0**-20
    to = (2.0**-11 + 2 * score + 2 * sums) * spread[0] + L * 2.0**-32 * 6
    to = to + (2.0**-8 if dtype == "bf16" else 2.0**-11) * (eo[0] + to) + 2.0**-25
    assert np.all(to < eo[0] / 20)  # a lost tail would show
    err = (o.double() - torch.from_numpy(eo[0]).cuda()).abs().amax((0, 1)).cpu().numpy()
    assert np.all(err <= to), (err.max(), to.max(), eo[0].max())
    assert float((lse.double() - el[0]).abs().max()) <= score + sums


@pytest.mark.parametrize("R,n,Hq", [(1, 1, 2), (1, 1, 16), (1, 130, 2)], ids=["one row", "16 rows", "256-row tiles"])
@pytest.mark.parametrize("up", [7.9, 8.1, 15.9])
def test_attention_of_scores_that_climb(up, R, n, Hq):
    """Scores that rise by steps, `up` binary orders in all: numerators against the first keys' maximum reach 2^up,
    on either side of where the maximum in use is taken anew."""
    L, page, Hkv = 640, 16, 1
    k = torch.zeros((L, Hkv, 128), dtype=torch.float16)
    k[:, 0, 0] = torch.from_numpy(F.E2M1[np.arange(L) * 8 // L])
    k[:, 0, 1] = 6.0
    v = torch.from_numpy(np.random.default_rng(0).standard_normal((L, Hkv, 128))).to(torch.float16)
    pages = vsa.cache_pages(L // page, Hkv, page)
    vsa.cache_append(k.cuda(), v.cuda(), i32(np.arange(L)), pages)
    q = torch.zeros((R, n, Hq, 128), dtype=torch.float16, device="cuda")
    q[..., 0] = up * math.log(2) * math.sqrt(128) / 6
    q[..., 1] = 30.0
    table = i32(np.tile(np.arange(L // page), (R, 1)))
    o, lse = _attend_shared(q, L, page, pages, table, n)
    vv = F.values(*F.quantise(f64(v)))[:, 0]
    eo, el, spread, reach = F.attention(f64(q[0, 0, :1]), f64(k[:, 0]), vv, [L])
    to, tl = F.tolerances(eo, el, spread, reach, L, np.abs(vv).max(), "f16")
    assert np.all(np.abs(f64(o) - eo[0]) <= to[0])
    assert np.all(np.abs(f64(lse) - el[0]) <= tl[0])


# ---------------------------------------------------------------------------
# The longest request
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("n", [1, 66])
def test_attention_over_the_most_tokens_a_table_row_holds(n):
    """2^31 - 16 positions, all in one page of 16 tokens: the output is that over the page, the lse more by the log of
    how often it occurs.  A worker adds fewer than 2^20 products of 16 keys one after another (2^27 of them, 148 workers
    and more), each sum truncated at 2^-23 of itself: 2^-3; denominators gather fewer terms."""
    M = (1 << 27) - 1
    x = torch.from_numpy(np.random.default_rng(4).standard_normal((16, 2, 1, 128)).astype(np.float32)).bfloat16().cuda()
    pages = vsa.cache_pages(1, 1, 16)
    vsa.cache_append(x[:, 0], x[:, 1], i32(np.arange(16)), pages)
    k, v = (F.values(*F.quantise(f64(y)))[:, 0] for y in (x[:, 0], x[:, 1]))
    q = torch.from_numpy(np.random.default_rng(5).standard_normal((n, 1, 128)).astype(np.float32)).bfloat16().cuda()
    table = torch.zeros((1, M), dtype=torch.int32, device="cuda")
    o, lse = vsa.cache_attn(q, i32([0, n]), i32([16 * M]), table, pages, n, vsa.cache_workspace(n, 1, 1), causal=False)
    eo, el, spread, _ = F.attention(f64(q[:, 0]), k, v, [16] * n)
    assert np.all(np.abs(f64(lse[:, 0]) - el - math.log(M)) <= 2.0**-3)
    assert np.all(np.abs(f64(o[:, 0]) - eo) <= 2.0**-3 * spread + 2.0**-8 * np.abs(eo))


# ---------------------------------------------------------------------------
# The merge of what is not a number
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("which", ["fine", "past"])
def test_untile_merge_of_nan(which):
    """A NaN in one lse is a NaN in the result, whether or not the other side has a key."""
    plan = vsa.Plan(4, 8, 8)
    ot = torch.ones((1, 1, 256, 128), dtype=torch.bfloat16, device="cuda")
    past = torch.ones((1, 256, 1, 128), dtype=torch.bfloat16, device="cuda")
    lt, lp = torch.zeros((1, 1, 256), device="cuda"), torch.zeros((1, 256, 1), device="cuda")
    own, other = (lt, lp) if which == "fine" else (lp, lt)
    own.view(-1)[:] = float("nan")
    other.view(-1)[::2] = -np.inf
    o, lse = vsa.untile_merge(plan, ot, lt, past, lp)
    assert torch.isnan(lse).all() and torch.isnan(o).all()


# ---------------------------------------------------------------------------
# A wait that runs out
# ---------------------------------------------------------------------------


def test_a_wait_that_runs_out_is_reported_and_leaves_the_context_usable(tmp_path, monkeypatch):
    """The attention for few rows in a build whose longest wait is nothing: its loading warp gives up as soon as no
    stage is free, the copies under way land, the call ends and reports VSA_ERR_TIMEOUT.  The normal build then gives
    its results with the workspace zeroed."""
    if not os.path.exists(vsa_build.NVCC):
        pytest.skip("needs nvcc")
    b = Batch([1] * 4, [20000] * 4, 8, 8, 64, "bf16")
    good = b.run(False)
    variant = vsa_build.build(lib=str(tmp_path / "libvsa_nowait.so"), defines=("VSA_CACHE_WAIT_NS=0",))
    with monkeypatch.context() as m:
        m.setattr(vsa, "_lib", None)
        m.setattr(vsa, "LIB_PATH", variant)
        b.run(False)
        assert vsa.get_status() == vsa.VSA_ERR_TIMEOUT
        assert vsa.get_status() == vsa.VSA_OK  # read and cleared
    b.ws.zero_()
    o, lse = b.run(False)
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


# ---------------------------------------------------------------------------
# KVCache and Forward(past=)
# ---------------------------------------------------------------------------


def test_reserves_of_many_sizes_keep_no_memory():
    cache = vsa.KVCache(num_pages=4, Hq=1, page_tokens=16)
    none = i32([0])
    cache.reserve(none, 4000)
    before = torch.cuda.memory_allocated()
    for tokens in range(4001, 4201):
        cache.reserve(none, tokens)
    assert torch.cuda.memory_allocated() - before <= 1 << 16


def test_slots_of_a_reserve_are_its_callers():
    cache = vsa.KVCache(num_pages=4, Hq=1, page_tokens=16)
    first = cache.reserve(i32([3]), 3)
    second = cache.reserve(i32([3]), 3)
    assert first.tolist() != second.tolist()
    assert vsa.cache_read(first, cache.pages)[0].shape == (3, 1, 128)
    page = int(cache.table[0, 0])
    assert [s - 16 * page for s in first.tolist()] == [0, 1, 2] and [s - 16 * page for s in second.tolist()] == [3, 4, 5]


def test_a_captured_append_follows_the_reserves_outside():
    """reserve outside the capture, append inside: each replay writes at the slots of the last reserve of that size,
    whatever was reserved and allocated between."""
    cache = vsa.KVCache(num_pages=8, Hq=1, page_tokens=16)
    k = torch.zeros((2, 1, 128), dtype=torch.bfloat16, device="cuda")
    cache.reserve(i32([2]), 2)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cache.append(k, k)
    g.replay()
    for i in range(1, 5):
        cache.reserve(i32([1]), 1)
        cache.append(k[:1], k[:1])
        slots = cache.reserve(i32([2]), 2)
        del slots
        junk = [torch.full((2,), -1, dtype=torch.int32, device="cuda") for _ in range(50)]
        k.fill_(6.0 * i)
        g.replay()
        at = cache.kv_len.item()
        last = i32([int(cache.table[0, p // 16]) * 16 + p % 16 for p in (at - 2, at - 1)])
        assert bool((vsa.cache_read(last, cache.pages)[0] == 6.0 * i).all())
        del junk


@pytest.mark.parametrize("n,kv", [([2, 1], [40, 20]), ([100], [300]), ([100, 2], [300, 40])],
                         ids=["few rows", "many", "both"])
def test_rows_outside_every_request_in_tensors_made_here(n, kv):
    """Rows before and behind the requests of a result that the call makes itself: o = 0, lse = -inf; in a tensor that
    the caller gives they stay."""
    b = Batch(n, kv, 4, 2, 16, "bf16", pad_rows=8)
    T, first, behind = b.T, 3, 3 + sum(n)
    want = b.run(True)
    q = torch.cat([b.q[:first], b.q[:T - first]])
    args = (q, i32(b.cu + first), i32(kv), i32(b.table), b.pages, max(n), b.ws)
    for keep in ((), ("o_out",), ("lse_out",)):
        junk = [torch.full((T, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((T, 4), float("nan"), device="cuda")]
        given = dict(o_out=junk[0].clone().fill_(7.0), lse_out=junk[1].clone().fill_(7.0))
        given = {name: given[name] for name in keep}
        del junk
        o, lse = vsa.cache_attn(*args, **given)
        assert torch.equal(o[first:behind], want[0][:sum(n)]) and torch.equal(lse[first:behind], want[1][:sum(n)])
        for x, name, value in ((o, "o_out", 0.0), (lse, "lse_out", -np.inf)):
            outside = torch.cat([x[:first], x[behind:]])
            assert outside.shape[0] == T - sum(n) and bool((outside == (7.0 if name in keep else value)).all())


def test_rows_of_a_request_that_was_refused():
    """A request that reserve refuses keeps its length; its rows of the batch see what its last tokens see."""
    cache = vsa.KVCache(num_pages=3, Hq=1, max_requests=2, page_tokens=16, max_q=8)
    x = torch.randn((40, 1, 128), device="cuda").bfloat16()
    cache.reserve(i32([16, 10]), 26)
    cache.append(x[:26], x[:26])
    cache.reserve(i32([17, 6]), 23)  # two pages where one is left; none
    assert vsa.get_status() == vsa.VSA_ERR_CAPACITY
    cache.append(x[:23], x[:23])
    assert cache.kv_len.tolist() == [16, 16] and cache.cu.tolist() == [0, 17, 23]
    assert bool((cache.slots[:17] == -1).all()) and bool((cache.slots[17:] >= 0).all())
    q = torch.randn((23, 1, 128), device="cuda").bfloat16()
    o, lse = cache.attend(q)
    kv, cu = i32([16, 16]), i32([0, 17, 23])
    o2, lse2 = vsa.cache_attn(q, cu, kv, cache.table, cache.pages, 8, vsa.cache_workspace(8, 1, 1))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert not o[0].any() and bool(torch.isneginf(lse[0]).all())  # 17 rows over 16 tokens: the first sees none


def _chunk(plan, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((1, plan.S, H, 128), generator=g, device="cuda").bfloat16() for _ in range(3)]


def test_forward_refuses_a_past_before_it_launches_anything():
    plan, H = vsa.Plan(4, 8, 8), 1
    q, k, v = _chunk(plan, H, 3)
    past = (torch.zeros_like(q), torch.zeros((1, plan.S, H), device="cuda"))
    fwd, gated = vsa.Forward(plan, 1, H, 1), vsa.Forward(plan, 1, H, 1, gated=True)
    for f in (fwd, gated):
        f.ot.fill_(7.0)
    with pytest.raises(ValueError, match="past"):
        gated(q, k, v, gate=q, past=past)
    for bad in ((past[0][:, :-1], past[1]), (past[0], past[1][:, :-1]), (past[0].half(), past[1]),
                (past[0], past[1].double()), (past[0].cpu(), past[1])):
        with pytest.raises(ValueError):
            fwd(q, k, v, past=bad)
    torch.cuda.synchronize()
    assert bool((fwd.ot == 7.0).all()) and bool((gated.ot == 7.0).all())


FORMS = {"256": (dict(T=4, Hg=9, Wg=10), {}, {}), "nvfp4": (dict(T=4, Hg=9, Wg=10), {}, dict(nvfp4=True)),
         "64": (dict(T=4, Hg=8, Wg=12), dict(block=(4, 4, 4), n_prefix=70), dict(prefix_dense=True)),
         "64 nvfp4": (dict(T=4, Hg=8, Wg=12), dict(block=(4, 4, 4), n_prefix=70), dict(prefix_dense=True, nvfp4=True))}


@pytest.mark.parametrize("form", FORMS)
def test_forward_with_a_past_in_each_form(form):
    """fwd(past=) is the fine stage's result merged with the past, eager and as Forward.graph captures it."""
    grid, layout, kind = FORMS[form]
    plan, H = vsa.Plan(*grid.values(), **layout), 2
    q, k, v = _chunk(plan, H, 1)
    past = (torch.randn_like(q), torch.randn((1, plan.S, H), device="cuda") + 4)
    plain = vsa.Forward(plan, 1, H, 2, **kind)
    plain(q, k, v)
    o_fine = vsa.untile(plan, plain.ot)
    l_fine = vsa.untile(plan, plain.lse[..., None].expand(-1, -1, -1, 128).to(torch.bfloat16).contiguous())[..., 0]
    want = vsa.untile_merge(plan, plain.ot, plain.lse, *past)
    w = torch.sigmoid(past[1] - l_fine.float())[..., None]  # weight of the past; l_fine is rounded to 8 bits
    near = (1 - w) * o_fine.float() + w * past[0].float()
    assert float((want[0].float() - near).abs().max()) <= 2.0**-5 * float(past[0].abs().max())
    fwd = vsa.Forward(plan, 1, H, 2, **kind)
    o, lse = fwd(q, k, v, past=past)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = fwd.graph(q, k, v, past=past)
    q2, k2, v2 = _chunk(plan, H, 2)
    for a, b in zip((q, k, v), (q2, k2, v2)):
        a.copy_(b)
    past[1].add_(1.5)
    g.replay()
    plain(q, k, v)
    want = vsa.untile_merge(plan, plain.ot, plain.lse, *past)
    assert torch.equal(fwd.o, want[0]) and torch.equal(fwd.lse_all, want[1])


def test_a_captured_step_of_a_video():
    """attend_chunk, Forward(past=), reserve and append of one chunk in a graph, replayed chunk after chunk, give the
    bits of the eager calls."""
    plan, H = vsa.Plan(4, 9, 10), 2

    def new():
        return vsa.Forward(plan, 1, H, 2), vsa.KVCache(num_pages=40, Hq=H, max_len=4 * plan.S, max_q=plan.S)

    def step(fwd, cache, q, k, v, n):
        o, lse = fwd(q, k, v, past=cache.attend_chunk(q))
        cache.reserve(n, plan.S)
        cache.append(k[0], v[0])
        return o, lse

    (fe, ce), (fg, cg) = new(), new()
    n = i32([plan.S])
    q, k, v = _chunk(plan, H, 0)
    step(*new(), q, k, v, n)  # one-time set-up
    fg(q, k, v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, lg = step(fg, cg, q, k, v, n)
    for chunk in range(4):
        for a, b in zip((q, k, v), _chunk(plan, H, 10 + chunk)):
            a.copy_(b)
        g.replay()
        oe, le = step(fe, ce, q, k, v, n)
        assert torch.equal(og, oe) and torch.equal(lg, le)
        assert torch.equal(cg.kv_len, ce.kv_len) and torch.equal(cg.table, ce.table)
    pos = torch.arange(4 * plan.S, device="cuda")
    slots = (ce.table[0, pos // 64] * 64 + pos % 64).int()
    for a, b in zip(vsa.cache_read(slots, cg.pages), vsa.cache_read(slots, ce.pages)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_of_the_smallest_blocks(dtype):
    """A block whose largest magnitude is 6 x 2^-10 or less has no scale and is stored as zeros; the next larger value
    of either type has one."""
    edge = 6 * 2.0**-10
    up = edge + 2.0**-8 * torch.finfo(TDT[dtype]).eps
    x = torch.zeros((2, 1, 128), dtype=TDT[dtype])
    x[0], x[1] = edge, up
    pages = vsa.cache_pages(1, 1, 16).fill_(0xA5)
    vsa.cache_append(x.cuda(), -x.cuda(), i32([0, 1]), pages)
    k, v = vsa.cache_read(i32([0, 1]), pages, TDT[dtype])
    assert not f64(k)[0].any() and not f64(v)[0].any()
    assert np.all(f64(k)[1] == 6 * 2.0**-9 * 0.5) and np.all(f64(v)[1] == -6 * 2.0**-9 * 0.5)
