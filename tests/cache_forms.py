"""Plain forms of the 4-bit key/value cache in 64 bits (numpy, CPU), written from the format's definition: codes and
scales of a token, the 2304-byte record of 16 tokens, block tables, attention, and the tolerances that go with it."""
from __future__ import annotations

import math

import numpy as np

D = 128
REC = 2304
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
# E4M3 without its NaN (bias 7, 3 mantissa bits)
E4M3 = np.array([(b & 7) / 8 * 2.0**-6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def nearest_even(x, levels):
    """Index of the level nearest to x >= 0; a tie goes to the even index; beyond the last: the last."""
    hi = np.clip(np.searchsorted(levels, x), 1, len(levels) - 1)
    lo = hi - 1
    d = (x - levels[lo]) - (levels[hi] - x)
    up = (d > 0) | ((d == 0) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x):
    """x [..., 128] -> (codes 0..15 [..., 128], scale bytes [..., 8]); quotients rounded to fp32 as defined."""
    f = x.astype(np.float64).reshape(*x.shape[:-1], 8, 16)
    amax = np.abs(f).max(-1)
    sb = nearest_even((amax / 6).astype(np.float32).astype(np.float64), E4M3)
    s = E4M3[sb]
    inv = np.where(s == 0, 0.0, 1 / np.where(s == 0, 1.0, s)).astype(np.float32).astype(np.float64)
    y = (f * inv[..., None]).astype(np.float32).astype(np.float64)
    c = nearest_even(np.abs(y), E2M1) + 8 * np.signbit(y)
    return c.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def values(codes, sb):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return (v.reshape(*codes.shape[:-1], 8, 16) * E4M3[sb][..., None]).reshape(codes.shape)


def put(pages, slots, k, v):
    """Writes tokens k, v [T, H, 128] at their slots of pages [n, H, page / 16, 2304]; negative slots are skipped."""
    page = pages.shape[2] * 16
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        p = s % 16
        for h in range(pages.shape[1]):
            rec = pages[s // page, h, s % page // 16]
            rec[p * 64:p * 64 + 64] = kc[t, h, 0::2] | (kc[t, h, 1::2] << 4)
            rec[1024 + p * 64:1024 + p * 64 + 64] = vc[t, h, 0::2] | (vc[t, h, 1::2] << 4)
            rec[2048 + p * 8:2048 + p * 8 + 8] = ks[t, h]
            for g in range(8):
                rec[2176 + g * 16 + (p % 4) * 4 + p // 4] = vs[t, h, g]


def get(pages, slots):
    """(k, v) [T, H, 128] in 64 bits."""
    page = pages.shape[2] * 16
    s = np.asarray(slots)
    rec = pages[s // page, :, s % page // 16]  # [T, H, 2304]
    p = (s % 16)[:, None, None]
    j, g = np.arange(64)[None, None], np.arange(8)[None, None]

    def one(at, sc):
        b = np.take_along_axis(rec, at + p * 64 + j + np.zeros((1, rec.shape[1], 1), dtype=np.int64), -1)
        sb = np.take_along_axis(rec, sc + np.zeros((1, rec.shape[1], 1), dtype=np.int64), -1)
        c = np.empty((*b.shape[:2], D), dtype=np.uint8)
        c[..., 0::2], c[..., 1::2] = b & 15, b >> 4
        return values(c, sb)

    return one(0, 2048 + p * 8 + g), one(1024, 2176 + g * 16 + (p % 4) * 4 + p // 4)


def tables(kv_len, new_len, page, free, start, table, max_tokens):
    """Request after request: (kv_out, cu, slots, next, table, refused)."""
    R, max_pages = table.shape
    table = table.copy()
    kv_out, cu, slots = kv_len.copy(), np.zeros(R + 1, np.int64), np.full(max_tokens, -1, np.int64)
    at, take, short, refused = 0, start, False, []
    for r in range(R):
        n, L = int(new_len[r]), int(kv_len[r])
        cu[r] = min(at, max_tokens)
        first = at
        at += max(n, 0)
        ok = n >= 0 and L >= 0 and L + n <= max_pages * page and at <= max_tokens
        need = -(-(L + n) // page) - -(-L // page) if ok else 0
        if ok and need > 0:
            short = short or take + need > len(free)
            ok = not short
        if not ok:
            refused.append(r)
            continue
        had = -(-L // page)
        table[r, had:had + need] = free[take:take + need]
        take += need
        kv_out[r] = L + n
        for i in range(n):
            pos = L + i
            slots[first + i] = int(table[r, pos // page]) * page + pos % page
    cu[R] = min(at, max_tokens)
    return kv_out, cu, slots, take, table, refused


def attention(q, k, v, limit, live=None):
    """q [n, 128], k, v [L, 128] in 64 bits, query i over keys j < limit[i] with live[j].  Returns (o, lse, spread,
    reach): spread_i = sum_j p_ij |v_j|, reach_i = max_j sum_d |q_id k_jd| / sqrt(128), what the tolerances go by."""
    n, L = q.shape[0], k.shape[0]
    see = np.arange(L)[None] < np.asarray(limit)[:, None]
    if live is not None:
        see = see & live[None]
    x = np.where(see, (q @ k.T) / math.sqrt(D), -np.inf)
    m = x.max(-1, initial=-np.inf)
    p = np.exp(x - np.where(np.isinf(m), 0.0, m)[:, None])
    z = p.sum(-1)
    p = p / np.where(z == 0, 1.0, z)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(z == 0, -np.inf, np.where(np.isinf(m), 0.0, m) + np.log(z))
    reach = ((np.abs(q) @ np.abs(k).T) * see).max(-1, initial=0.0) / math.sqrt(D)
    return p @ v, lse, p @ np.abs(v), reach


def tolerances(o, lse, spread, reach, L, vmax, dtype):
    """Bounds on |o - exact| (per element) and |lse - exact| (per row).

    The products are exact in fp32; a score is a sum of 128 of them, off by at most 127 * 2^-24 * reach, taken as
    2^-17 * reach, and scaled with one rounding more.  A softmax weight is off by that and by exp2's 2^-22; its
    numerator is rounded to fp16, 2^-11 of itself, or 2^-25 where it is below 2^-14 of the largest (the
    denominator is at least 1): twice the score's error, for numerator and denominator.  A sum over L keys in fp32
    gathers at most L * 2^-24 of the sum of magnitudes, whatever the order, and the rescales 2^-20.  Last, o is
    rounded to its type: half a step (fp16 below its normal range: 2^-25)."""
    half = 2.0**-8 if dtype == "bf16" else 2.0**-11
    score = 2.0**-17 * reach + 2.0**-22 * (1 + np.abs(np.where(np.isinf(lse), 0.0, lse)))
    sums = L * 2.0**-24 + 2.0**-20
    weight = (2.0**-11 + 2 * score + 2 * sums)[:, None]
    to = weight * spread + L * 2.0**-25 * vmax
    to = to + half * (np.abs(o) + to) + (2.0**-25 if dtype == "f16" else 0.0)
    return to, score + sums
