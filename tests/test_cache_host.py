"""Host-side checks of the 4-bit key/value cache's calls: refusals (no kernel is launched: every rejected call
returns before any CUDA call), sizes, and the plain forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_video_gather_b200 as vsa
from block_sparse_video_gather_b200 import build as vsa_build
from tests import cache_forms as F

FAKE = 0x100000  # an aligned, non-null address; never dereferenced


@pytest.fixture(scope="module")
def L():
    vsa_build.build()
    return vsa.lib()


A, M = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 8)  # aligned / misaligned
B = ctypes.c_void_p(FAKE + 4096)
INV, UNS = vsa.VSA_ERR_INVALID_ARG, vsa.VSA_ERR_UNSUPPORTED


def _calls(L):
    """name -> (call, good arguments, {argument position: [(bad value, code)]})."""
    ptr = [(None, INV), (M, INV)]
    page = [(0, UNS), (8, UNS), (48, UNS), (512, UNS)]
    heads = [(0, INV), (-1, INV), (65536, UNS)]
    dtype = [(2, INV), (-1, INV)]
    size = [(64, UNS), (256, UNS)]
    num_pages = [(0, INV), (1 << 28, UNS)]  # 2^28 pages of 64 tokens are 2^34 slots
    R = [(0, INV), (4097, UNS)]
    return {
        "vsa_cache_tables": (
            [A, A, 3, 64, A, 10, A, A, 8, B, A, A, 100, B, None],
            {0: ptr, 1: ptr, 2: R, 3: page, 4: ptr, 5: [(-1, INV)], 6: ptr, 7: ptr,
             8: [(0, INV), (1 << 28, UNS)], 9: ptr + [(A, INV)], 10: ptr, 11: ptr, 12: [(-1, INV)],
             13: ptr + [(A, INV)]}),
        "vsa_cache_release": (
            [A, 3, 64, A, A, 8, A, 10, A, None],
            {0: ptr, 1: R, 2: page, 3: ptr, 4: ptr, 5: [(0, INV), (1 << 28, UNS)], 6: ptr, 7: [(-1, INV)], 8: ptr}),
        "vsa_cache_append_nvfp4": (
            [0, A, A, 256, 256, A, 3, 2, 128, A, 4, 64, None],
            {0: dtype, 1: ptr, 2: ptr, 3: [(255, INV), (248, INV), (260, INV)], 4: [(0, INV), (257, INV)], 5: ptr,
             6: [(-1, INV)], 7: heads, 8: size, 9: ptr, 10: num_pages, 11: page}),
        "vsa_cache_read_nvfp4": (
            [0, A, 3, 2, 128, A, 4, 64, A, A, None],
            {0: dtype, 1: ptr, 2: [(-1, INV)], 3: heads, 4: size, 5: ptr, 6: num_pages, 7: page, 8: ptr, 9: ptr}),
        "vsa_cache_attn_nvfp4": (
            [0, A, 512, A, A, 3, 9, 5, 4, 2, 128, A, 4, 64, A, 8, 1, A, A, A, None],
            {0: dtype, 1: ptr, 2: [(504, INV), (513, INV)], 3: ptr, 4: ptr, 5: R, 6: [(-1, INV), (1 << 30, UNS)],
             7: [(0, INV)], 8: [(0, INV), (3, INV)], 9: heads + [(3, INV)], 10: size, 11: ptr, 12: num_pages,
             13: page, 14: ptr, 15: [(0, INV), (1 << 28, UNS)], 17: ptr, 18: ptr, 19: ptr}),
    }


@pytest.mark.parametrize("name", ["vsa_cache_tables", "vsa_cache_release", "vsa_cache_append_nvfp4",
                                  "vsa_cache_read_nvfp4", "vsa_cache_attn_nvfp4"])
def test_calls_refuse_invalid_arguments(L, name):
    good, bad = _calls(L)[name]
    for pos, values in bad.items():
        for value, code in values:
            args = list(good)
            args[pos] = value
            assert getattr(L, name)(*args) == code, (name, pos, value)


def test_untile_merge_refuses_invalid_arguments(L):
    h = vsa.Plan(4, 8, 8).handle
    good = [h, 0, A, A, A, A, 1, 2, 128, A, A, None]
    for pos, values in {0: [(None, INV)], 1: [(2, INV)], 2: [(None, INV), (M, INV)], 3: [(None, INV), (M, INV)],
                        4: [(None, INV), (M, INV)], 5: [(None, INV), (M, INV)], 6: [(0, INV), (40000, UNS)],
                        7: [(0, INV)], 8: [(64, UNS)], 9: [(None, INV), (M, INV)], 10: [(M, INV)]}.items():
        for value, code in values:
            args = list(good)
            args[pos] = value
            assert L.vsa_untile_merge(*args) == code, (pos, value)


def test_sizes(L):
    n = ctypes.c_size_t(0)
    assert L.vsa_cache_page_bytes(12, 128, 64, ctypes.byref(n)) == vsa.VSA_OK and n.value == 12 * 64 * 144
    assert L.vsa_cache_page_bytes(12, 128, 64, None) == INV
    assert L.vsa_cache_page_bytes(12, 64, 64, ctypes.byref(n)) == UNS
    assert L.vsa_cache_page_bytes(12, 128, 24, ctypes.byref(n)) == UNS
    for args, code in (((12, 12, 1), vsa.VSA_OK), ((12, 5, 1), INV), ((12, 12, 0), INV), ((0, 12, 1), INV)):
        assert L.vsa_cache_attn_workspace(*args, ctypes.byref(n)) == code
    assert L.vsa_cache_attn_workspace(12, 12, 1, None) == INV
    assert b"cache" in L.vsa_strerror(vsa.VSA_ERR_CAPACITY)


def test_binding_refuses_wrong_tensors(L):
    pages = torch.empty((2, 3, 4, 2304), dtype=torch.uint8)
    k = torch.zeros((5, 3, 128), dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vsa.cache_append(k, k, slots, pages)
    with pytest.raises(ValueError, match="one type"):
        vsa.cache_append(k, k.half(), slots, pages)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        vsa.cache_append(k.float(), k.float(), slots, pages)
    with pytest.raises(ValueError, match="one type"):
        vsa.cache_append(k[:, :2], k[:, :2], slots, pages)
    with pytest.raises(ValueError, match="slots"):
        vsa.cache_append(k, k, slots[:4], pages)
    with pytest.raises(ValueError, match="pages"):
        vsa.cache_append(k, k, slots, pages[..., :2000])
    with pytest.raises(ValueError, match="k_out"):
        vsa.cache_read(slots, pages, k_out=k[:4], v_out=k)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vsa.cache_attn(k, i, i[:3], i.view(1, 4).expand(3, 4), pages, 1, torch.zeros(1 << 20))
    with pytest.raises(ValueError, match="block_table"):
        vsa.cache_tables(i, i, 64, i, i, i, i)


def test_plain_forms_round_to_nearest_even_and_invert():
    x = np.array([0, 0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.0])
    assert F.nearest_even(x, F.E2M1).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 37, 3, 128))
    pages = np.full((3, 3, 2, F.REC), 0xA5, dtype=np.uint8)
    slots = rng.permutation(96)[:37]
    F.put(pages, slots, k, v)
    gk, gv = F.get(pages, slots)
    np.testing.assert_array_equal(gk, F.values(*F.quantise(k)))
    np.testing.assert_array_equal(gv, F.values(*F.quantise(v)))
    # a value times its block's scale is off by at most half of E2M1's widest step
    assert np.all(np.abs(gk - k) <= np.abs(k).reshape(37, 3, 8, 16).max(-1).repeat(16, -1).reshape(k.shape) / 6 * 1.07)


def test_plain_attention_of_a_row_without_keys():
    o, lse, _, _ = F.attention(np.ones((2, 128)), np.ones((3, 128)), np.ones((3, 128)), [0, 2])
    assert np.all(o[0] == 0) and lse[0] == -np.inf and np.allclose(o[1], 1)


def test_the_filling_attention_refuses_what_the_other_does(L):
    good, bad = _calls(L)["vsa_cache_attn_nvfp4"]
    at = lambda pos: pos + (pos >= 17)  # `fill` comes after `causal`
    cases = [(at(pos), value, code) for pos, values in bad.items() for value, code in values]
    for pos, value, code in cases + [(17, -1, INV), (17, 4, INV)]:
        args = good[:17] + [3] + good[17:]
        args[pos] = value
        assert L.vsa_cache_attn_nvfp4_fill(*args) == code, (pos, value)


def test_release_refuses_wrong_shapes(L):
    kv, table, one = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32), torch.ones(3).bool()
    good = dict(drop=one, kv_len=kv, block_table=table, free_pages=kv, free_start=kv[:1])
    for name, value, match in (("kv_len", kv.view(3, 1), r"\[R\]"), ("kv_len", table, r"\[R\]"),
                               ("kv_len", kv[0], r"\[R\]"), ("drop", one[:2], r"\[R\]"),
                               ("block_table", table[:2], r"\[R\]"), ("block_table", kv, r"\[R\]"),
                               ("free_start", kv[:0], "free_start")):
        with pytest.raises(ValueError, match=match):
            vsa.cache_release(page_tokens=16, **{**good, name: value})
    with pytest.raises(ValueError, match="CUDA"):
        vsa.cache_release(page_tokens=16, **good)
