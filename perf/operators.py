"""Workloads of the 4-bit key/value cache operators, in plain torch and through this package.

Four operators: the block tables and slot map of a batch of requests, the cache's writer (read back through its
reader), attention over the cache, and the merge of that attention with the sparse fine stage's output.  `run`
computes them with elementary torch operations in 32 bits, or with the package's calls where `own` is set.

The cache holds keys and values as NVFP4: 4-bit E2M1 codes with one E4M3 scale for each 16 channels of a token's
head.  Pages are [num_pages, H_kv, page_tokens / 16, 2304] bytes; a record of 2304 bytes holds 16 tokens: 16 x 64
bytes of key codes, 16 x 64 of value codes (channel 2j in the low nibble of byte j), 16 x 8 key scales, and 128
value scales, the one of token t and channel block g at byte g * 16 + (t % 4) * 4 + t // 4.
"""
import math

import torch

own = False

D = 128
RECORD = 2304
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoding step of a few requests: one new token each
        {"name": "tables 8 requests", "op": "tables", "R": 8, "page": 64, "max_pages": 512, "new": 1, "old": 30000},
        # admission of a large batch of prompts of mixed length
        {"name": "tables 4096 requests", "op": "tables", "R": 4096, "page": 16, "max_pages": 160, "new": 500,
         "old": 2000},
        # the new tokens of a decoding step, 24 heads
        {"name": "append 33 tokens", "op": "append", "T": 33, "H": 24, "page": 16, "dtype": "f16"},
        # one whole clip of (31, 22, 40) latent tokens, 24 heads, as slices of a fused projection
        {"name": "append 27280 tokens", "op": "append", "T": 27280, "H": 24, "page": 64, "dtype": "bf16"},
        # a single token against a short context: latency
        {"name": "attend 1x1 on 777", "op": "attend", "R": 1, "n": 1, "L": 777, "Hq": 12, "Hkv": 12, "page": 64,
         "causal": True, "dtype": "bf16"},
        # a decoding batch of ragged contexts, four query heads to a key head, small pages
        {"name": "attend 32x1 on 8000", "op": "attend", "R": 32, "n": 1, "L": 8000, "Hq": 32, "Hkv": 8, "page": 16,
         "causal": True, "dtype": "f16"},
        # a single token against a long clip of (81, 30, 52) latent tokens
        {"name": "attend 1x1 on 126360", "op": "attend", "R": 1, "n": 1, "L": 126360, "Hq": 12, "Hkv": 12,
         "page": 256, "causal": True, "dtype": "bf16"},
        # a few drafted tokens of several requests checked together
        {"name": "attend 9x5 on 3001", "op": "attend", "R": 9, "n": 5, "L": 3001, "Hq": 24, "Hkv": 3, "page": 32,
         "causal": True, "dtype": "bf16"},
        # a chunk of (4, 30, 52) latent tokens against the cached (21, 30, 52) of the clip so far, 12 heads
        {"name": "attend 1x6240 on 32760", "op": "attend", "R": 1, "n": 6240, "L": 32760, "Hq": 12, "Hkv": 12,
         "page": 64, "causal": False, "dtype": "bf16"},
        # prompts read in pieces, causal, grouped heads, ragged
        {"name": "attend 4x1023 on 5000", "op": "attend", "R": 4, "n": 1023, "L": 5000, "Hq": 16, "Hkv": 4,
         "page": 16, "causal": True, "dtype": "f16"},
        # the merge for a small latent grid
        {"name": "merge 3x15x26", "op": "merge", "B": 2, "H": 12, "T": 3, "Hg": 15, "Wg": 26, "dtype": "f16"},
        # the merge for a clip of (21, 30, 52) latent tokens, 12 heads
        {"name": "merge 21x30x52", "op": "merge", "B": 1, "H": 12, "T": 21, "Hg": 30, "Wg": 52, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "attend", "merge"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    if op == "tables":
        old, new = _log_int(rng, 1, 30000), _log_int(rng, 1, 600)
        return {"op": op, "R": _log_int(rng, 1, 4096), "page": page, "max_pages": (old + new) // page + 1 + rng.randint(0, 9),
                "new": new, "old": old}
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, 27000), "H": rng.choice([1, 3, 8, 12, 24]), "page": page,
                "dtype": dtype}
    if op == "merge":
        return {"op": op, "B": rng.randint(1, 2), "H": rng.choice([1, 5, 12]), "T": _log_int(rng, 1, 10),
                "Hg": _log_int(rng, 3, 30), "Wg": _log_int(rng, 3, 52), "dtype": dtype}
    Hkv = rng.choice([1, 2, 3, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    if rng.random() < 0.6:  # one or a few new tokens of each request
        R, n = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7])
        L = _log_int(rng, max(n, 16), max(64, min(100000, 1500000 // (R * Hkv))))
    else:
        R, n = rng.randint(1, 5), _log_int(rng, 17, 4000)
        L = _log_int(rng, n, max(n + 1, min(30000, int(1.5e9 / (R * n * Hkv * group)))))
    return {"op": op, "R": R, "n": n, "L": L, "Hq": Hkv * group, "Hkv": Hkv, "page": page,
            "causal": rng.random() < 0.6, "dtype": dtype}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ragged(R, lo, hi, step):
    """R lengths spread over lo .. hi, the largest among them."""
    return [hi - (r * step) % (hi - lo + 1) for r in range(R)]


def _lengths(case):
    """New and cached tokens of the requests of a case of `attend`: ragged, up to n and L."""
    q = _ragged(case["R"], max(1, (case["n"] + 1) // 2), case["n"], 7)
    kv = _ragged(case["R"], max(1, case["L"] // 4), case["L"], 1237)
    if case["causal"]:
        kv = [max(a, b) for a, b in zip(q, kv)]  # the new tokens are in the cache
    return q, kv


def _tokens(g, T, H, dtype):
    """Keys and values as slices of a fused projection's output [T, 3, H, D]: normal values about each channel's own
    level, as after a projection."""
    x = torch.randn((T, 3, H, D), generator=g, device="cuda", dtype=torch.float32)
    x += torch.randn((1, 3, H, D), generator=g, device="cuda") * 0.5
    x = x.to(dtype)
    return x[:, 1], x[:, 2]


def _quantise(x):
    """[..., 128] 16-bit -> (codes in 0..15 as uint8 [..., 128], scale bytes uint8 [..., 8]).

    scale = E4M3(amax / 6), code = E2M1(x * (1 / scale)): each step rounded to fp32, then to the format, to nearest,
    ties to even."""
    f = x.float().unflatten(-1, (8, 16))
    amax = f.abs().amax(-1)
    scale = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)  # a division, not * (1 / 6)
    s = scale.float()
    inv = torch.where(s == 0, torch.zeros_like(s), 1 / s)
    y = f * inv[..., None]
    a = y.abs()
    # rounding borders of 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.signbit(y).to(torch.uint8) * 8
    return code.flatten(-2), scale.view(torch.uint8)


_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _levels(device, dtype):
    return torch.tensor(_LEVELS, device=device, dtype=dtype)


def _records(kc, ks, vc, vs):
    """Codes [N, 16, H, 128] and scales [N, 16, H, 8] of N groups of 16 tokens -> records [N, H, 2304]."""
    N, _, H, _ = kc.shape
    k = (kc[..., 0::2] | (kc[..., 1::2] << 4)).transpose(1, 2).reshape(N, H, 1024)
    v = (vc[..., 0::2] | (vc[..., 1::2] << 4)).transpose(1, 2).reshape(N, H, 1024)
    ks = ks.transpose(1, 2).reshape(N, H, 128)
    vs = vs.permute(0, 2, 3, 1).reshape(N, H, 8, 4, 4).transpose(3, 4).reshape(N, H, 128)
    return torch.cat([k, v, ks, vs], -1)


def _slot_bytes(slots, H, page):
    """Byte offsets in the pages of the tokens' records: [T, H], and the tokens' places in them: [T, 1]."""
    s = slots.long()[:, None]
    h = torch.arange(H, device=slots.device)[None]
    return (((s // page) * H + h) * (page // 16) + s % page // 16) * RECORD, s % 16


def _put(pages, slots, kc, ks, vc, vs):
    """Writes the tokens' codes and scales into their records."""
    H, page = pages.shape[1], pages.shape[2] * 16
    base, t = _slot_bytes(slots, H, page)
    flat = pages.view(-1)
    j, g = torch.arange(64, device=slots.device), torch.arange(8, device=slots.device)
    flat[(base + t * 64)[..., None] + j] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    flat[(base + 1024 + t * 64)[..., None] + j] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    flat[(base + 2048 + t * 8)[..., None] + g] = ks
    flat[(base + 2176 + t % 4 * 4 + t // 4)[..., None] + g * 16] = vs


def _values(codes, scales, dtype=torch.float32):
    """Packed codes [..., 64] and scale bytes [..., 8] -> the values [..., 128] they stand for (exact in fp32)."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.view(torch.float8_e4m3fn).to(dtype)
    return (_levels(codes.device, dtype)[c].unflatten(-1, (8, 16)) * s[..., None]).flatten(-2)


def _get(pages, slots):
    """Keys and values of the tokens at `slots`, fp32 [T, H, 128] each."""
    H, page = pages.shape[1], pages.shape[2] * 16
    base, t = _slot_bytes(slots, H, page)
    flat = pages.view(-1)
    j, g = torch.arange(64, device=slots.device), torch.arange(8, device=slots.device)
    k = _values(flat[(base + t * 64)[..., None] + j], flat[(base + 2048 + t * 8)[..., None] + g])
    v = _values(flat[(base + 1024 + t * 64)[..., None] + j], flat[(base + 2176 + t % 4 * 4 + t // 4)[..., None] + g * 16])
    return k, v


def _cache(g, num_pages, H, page, dtype):
    """Pages filled with quantised tokens, a slice of pages at a time."""
    pages = torch.empty((num_pages, H, page // 16, RECORD), dtype=torch.uint8, device="cuda")
    groups = num_pages * (page // 16)
    step = max(1, (1 << 25) // (16 * H * D * 3) // (page // 16)) * (page // 16)
    for at in range(0, groups, step):
        n = min(step, groups - at)
        k, v = _tokens(g, n * 16, H, dtype)
        (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
        rec = _records(*(x.reshape(n, 16, H, -1) for x in (kc, ks, vc, vs)))
        rec = rec.reshape(n // (page // 16), page // 16, H, RECORD).transpose(1, 2)
        pages[at // (page // 16):(at + n) // (page // 16)] = rec
    return pages


def prepare(case, seed):
    g = _gen(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "tables":
        R, P, M = case["R"], case["page"], case["max_pages"]
        # the lengths of a running batch; an empty request among them now and then
        kv = torch.tensor(_ragged(R, 0, case["old"], 1237), **i32)
        new = torch.tensor(_ragged(R, 0 if R > 8 else 1, case["new"], 7), **i32)
        kv, new = (x[torch.randperm(R, generator=g, device="cuda")] for x in (kv, new))
        had = (kv + P - 1) // P
        need = (kv + new + P - 1) // P - had
        total, used = int(need.sum()), int(had.sum())
        perm = torch.randperm(used + total + 16, generator=g, device="cuda").int()
        table = torch.full((R, M), -1, **i32)
        col = torch.arange(M, device="cuda")[None]
        table[col < had[:, None]] = perm[:used]
        tokens = int(new.sum())
        tokens += tokens % 3  # a padded batch now and then
        return {"case": case, "kv": kv, "new": new, "table": table, "free": perm, "tokens": tokens,
                "start": torch.tensor([used], **i32), "kv_out": torch.empty(R, **i32), "cu": torch.empty(R + 1, **i32),
                "slots": torch.empty(tokens, **i32), "next": torch.empty(1, **i32)}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "append":
        T, H, P = case["T"], case["H"], case["page"]
        k, v = _tokens(g, T, H, dtype)
        n = -(-T // P) + 3
        pages = torch.zeros((n, H, P // 16, RECORD), dtype=torch.uint8, device="cuda")
        order = torch.randperm(n, generator=g, device="cuda")
        at = torch.arange(T, device="cuda") + int(seed % P)  # the first page is partly full
        slots = (order[at // P] * P + at % P).int()
        return {"case": case, "k": k, "v": v, "pages": pages, "slots": slots,
                "ko": torch.empty((T, H, D), dtype=dtype, device="cuda"),
                "vo": torch.empty((T, H, D), dtype=dtype, device="cuda")}
    if case["op"] == "attend":
        R, P, Hq, Hkv = case["R"], case["page"], case["Hq"], case["Hkv"]
        order = torch.randperm(R, generator=g, device="cuda")
        q_len, kv_len = (torch.tensor(x, **i32)[order] for x in _lengths(case))
        M = -(-case["L"] // P)
        if case["causal"]:
            M = -(-max(case["L"], case["n"]) // P)
        had = (kv_len + P - 1) // P
        used = int(had.sum())
        pages = _cache(g, used + 2, Hkv, P, dtype)
        perm = torch.randperm(used + 2, generator=g, device="cuda").int()
        table = torch.zeros((R, M), **i32)
        table[torch.arange(M, device="cuda")[None] < had[:, None]] = perm[:used]
        T = int(q_len.sum())
        cu = torch.zeros(R + 1, **i32)
        cu[1:] = q_len.cumsum(0)
        q = torch.randn((T, Hq, D), generator=g, device="cuda").to(dtype)
        state = {"case": case, "q": q, "cu": cu, "kv_len": kv_len, "table": table, "pages": pages,
                 "o": torch.empty_like(q), "lse": torch.empty((T, Hq), dtype=torch.float32, device="cuda")}
        if own:
            import block_sparse_video_gather_b200 as vsa
            state["ws"] = vsa.cache_workspace(case["n"], Hq, Hkv)
        return state
    B, H, T, Hg, Wg = (case[k] for k in ("B", "H", "T", "Hg", "Wg"))
    slot, Sp = _grid_slots(T, Hg, Wg)
    S = T * Hg * Wg
    ot = torch.zeros((B, H, Sp, D), dtype=dtype, device="cuda")
    ot[:, :, slot] = torch.randn((B, H, S, D), generator=g, device="cuda").to(dtype)
    lse = torch.randn((B, H, Sp), generator=g, device="cuda") + 8
    past = torch.randn((B, S, H, D), generator=g, device="cuda").to(dtype)
    lse_past = torch.randn((B, S, H), generator=g, device="cuda") * 2 + 8
    # query blocks whose selection is empty, and tokens with no past
    lse.view(B, H, -1, 256)[:, :, 0] = torch.where(torch.rand((B, H, 1), generator=g, device="cuda") < 0.5, -math.inf,
                                                   lse.view(B, H, -1, 256)[:, :, 0])
    lse_past[torch.rand((B, S, H), generator=g, device="cuda") < 0.02] = -math.inf
    state = {"case": case, "ot": ot, "lse": lse, "past": past, "lse_past": lse_past, "slot": slot,
             "o": torch.empty_like(past), "lse_out": torch.empty_like(lse_past)}
    if own:
        import block_sparse_video_gather_b200 as vsa
        state["plan"] = vsa.Plan(T, Hg, Wg)
    return state


def _grid_slots(T, Hg, Wg):
    """Tiled row of each token of a (T, Hg, Wg) grid in (4, 8, 8) blocks, and the number of tiled rows."""
    s = torch.arange(T * Hg * Wg, device="cuda")
    t, y, x = s // (Hg * Wg), s // Wg % Hg, s % Wg
    nT, nH, nW = -(-T // 4), -(-Hg // 8), -(-Wg // 8)
    return (((t // 4) * nH + y // 8) * nW + x // 8) * 256 + (t % 4) * 64 + (y % 8) * 8 + x % 8, nT * nH * nW * 256


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import block_sparse_video_gather_b200 as vsa
    op = s["case"]["op"]
    if op == "tables":
        vsa.cache_tables(s["kv"], s["new"], s["case"]["page"], s["free"], s["start"], s["table"], s["slots"],
                         kv_len_out=s["kv_out"], cu_out=s["cu"], free_next_out=s["next"])
        return {"table": s["table"], "kv_len": s["kv_out"], "cu": s["cu"], "slots": s["slots"], "next": s["next"]}
    if op == "append":
        vsa.cache_append(s["k"], s["v"], s["slots"], s["pages"])
        return vsa.cache_read(s["slots"], s["pages"], s["k"].dtype, k_out=s["ko"], v_out=s["vo"])
    if op == "attend":
        return vsa.cache_attn(s["q"], s["cu"], s["kv_len"], s["table"], s["pages"], s["case"]["n"], s["ws"],
                              causal=s["case"]["causal"], o_out=s["o"], lse_out=s["lse"])
    return vsa.untile_merge(s["plan"], s["ot"], s["lse"], s["past"], s["lse_past"], out=s["o"], lse_out=s["lse_out"])


def _run_plain(s):
    op = s["case"]["op"]
    if op == "tables":
        return _tables(s)
    if op == "append":
        (kc, ks), (vc, vs) = _quantise(s["k"]), _quantise(s["v"])
        _put(s["pages"], s["slots"], kc, ks, vc, vs)
        k, v = _get(s["pages"], s["slots"])
        return k.to(s["k"].dtype), v.to(s["v"].dtype)
    if op == "attend":
        return _attend(s)
    return _merge(s)


def _tables(s):
    P, table = s["case"]["page"], s["table"]
    kv, new, device = s["kv"].long(), s["new"].long(), s["kv"].device
    had = (kv + P - 1) // P
    need = (kv + new + P - 1) // P - had
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=device)[None]
    j = col - had[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    take = s["start"].long() + first[:, None] + j
    table.copy_(torch.where(fresh, s["free"][take.clamp(0, s["free"].numel() - 1)], table))
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    i = torch.arange(s["tokens"], device=device)
    r = torch.searchsorted(cu, i, right=True) - 1
    real = r < kv.numel()
    r = r.clamp(max=kv.numel() - 1)
    pos = kv[r] + i - cu[r]
    page = table[r, (pos // P).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(real, page * P + pos % P, -1)
    return {"table": table, "kv_len": (kv + new).int(), "cu": cu.int(), "slots": slots.int(),
            "next": (s["start"] + need.sum()).int()}


def _attend(s):
    case, q, table, pages, kv_len = s["case"], s["q"], s["table"], s["pages"], s["kv_len"].long()
    P, Hkv = pages.shape[2] * 16, pages.shape[1]
    R, G, n = case["R"], case["Hq"] // Hkv, case["n"]
    L = table.shape[1] * P
    pos = torch.arange(L, device=q.device)
    slots = table.long()[:, pos // P] * P + pos % P
    k, v = _get(pages, slots.flatten())
    k = k.view(R, L, Hkv, D).transpose(1, 2)
    live = pos < kv_len[:, None]
    v = (v.view(R, L, Hkv, D) * live[..., None, None]).transpose(1, 2)
    q_len = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(n, device=q.device)
    token = (s["cu"][:-1, None] + i).clamp(max=q.shape[0] - 1)
    qp = q.float()[token].view(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D)
    x = torch.matmul(qp, k.transpose(-1, -2)).mul_(D ** -0.5)
    limit = (kv_len[:, None] - q_len[:, None] + i + 1) if case["causal"] else kv_len[:, None].expand(R, n)
    limit = limit.repeat_interleave(G, 1)
    x.masked_fill_((pos >= limit[..., None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z == 0, 1.0, z)
    lse = (m + z.log())[..., 0]
    o = o.view(R, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(R, n, Hkv * G, D)
    lse = lse.view(R, Hkv, n, G).permute(0, 2, 1, 3).reshape(R, n, Hkv * G)
    have = i < q_len[:, None]
    return o[have].to(q.dtype), lse[have]


def _merge(s):
    o1 = s["ot"].float()[:, :, s["slot"]].transpose(1, 2)
    l1 = s["lse"][:, :, s["slot"]].transpose(1, 2)
    l2 = s["lse_past"]
    m = torch.maximum(l1, l2)
    m0 = torch.where(m == -math.inf, 0.0, m)
    w1, w2 = (l1 - m0).exp(), (l2 - m0).exp()
    z = w1 + w2
    d = torch.where(z == 0, 1.0, z)
    o = o1 * (w1 / d)[..., None] + s["past"].float() * (w2 / d)[..., None]
    return o.to(s["past"].dtype), m0 + z.log()


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "tables":
        T = sum(_ragged(case["R"], 0 if case["R"] > 8 else 1, case["new"], 7))
        return {"bytes": 4 * (4 * case["R"] + T + 2 * (T // case["page"])), "flops": 0}
    if case["op"] == "append":
        return {"bytes": case["T"] * (case["H"] * (2 * 2 * 2 * D + 2 * 144) + 8), "flops": 0}
    if case["op"] == "merge":
        S = case["B"] * case["H"] * case["T"] * case["Hg"] * case["Wg"]
        return {"bytes": S * (3 * 2 * D + 12), "flops": S * 4 * D}
    q, kv = _lengths(case)
    pairs = sum(n * L - (n * (n - 1) // 2 if case["causal"] else 0) for n, L in zip(q, kv))
    return {"bytes": sum(kv) * case["Hkv"] * 144 + sum(q) * case["Hq"] * (4 * D + 4),
            "flops": 4 * D * case["Hq"] * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_quantised(s["k"]), _exact_quantised(s["v"])
    if case["op"] == "merge":
        S = s["past"].shape[1]
        o = torch.empty(s["past"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty((o.shape[0], S, o.shape[2]), dtype=torch.float64, device="cuda")
        for h in range(o.shape[2]):
            both = torch.stack([s["lse"].double()[:, h, s["slot"]], s["lse_past"].double()[:, :, h]], -1)
            lse[:, :, h] = torch.logsumexp(both, -1)
            w = torch.exp(both - lse[:, :, h, None]).nan_to_num(0.0)
            o[:, :, h] = s["ot"].double()[:, h, s["slot"]] * w[..., :1] + s["past"].double()[:, :, h] * w[..., 1:]
        return o, lse
    q, cu, kv = s["q"], s["cu"].tolist(), s["kv_len"].tolist()
    pairs = sum((cu[r + 1] - cu[r]) * kv[r] for r in range(case["R"])) * case["Hq"]
    if pairs > 4e9:
        return None
    P, Hkv = case["page"], case["Hkv"]
    G = case["Hq"] // Hkv
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    step = 1024
    for r in range(case["R"]):
        n, L = cu[r + 1] - cu[r], kv[r]
        kr, vr = _exact_tokens(s["pages"], s["table"][r], P, L)
        for h in range(case["Hq"]):
            for a in range(0, n, step):
                b = min(n, a + step)
                x = q[cu[r] + a:cu[r] + b, h].double() @ kr[:, h // G].T / math.sqrt(D)
                if case["causal"]:
                    last = L - n + torch.arange(a, b, device="cuda")[:, None]
                    x = torch.where(torch.arange(L, device="cuda")[None] <= last, x, -math.inf)
                lse[cu[r] + a:cu[r] + b, h] = torch.logsumexp(x, -1)
                o[cu[r] + a:cu[r] + b, h] = torch.softmax(x, -1).nan_to_num(0.0) @ vr[:, h // G]
    return o, lse


def _exact_tokens(pages, row, P, L):
    """Keys and values [L, Hkv, 128] of a request in 64 bits, from its pages as a whole."""
    rec = pages[row[:-(-L // P)].long()].transpose(1, 2).flatten(0, 1)  # [groups, Hkv, 2304]
    level = _levels("cuda", torch.float64)

    # E4M3: bias 7, three mantissa bits
    scale = torch.tensor([(b & 7) / 8 * 2.0 ** -6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7)
                          for b in range(127)], dtype=torch.float64, device="cuda")

    out = []
    for at, sc in ((0, rec[..., 2048:2176].unflatten(-1, (16, 8))),
                   (1024, rec[..., 2176:].unflatten(-1, (8, 4, 4)).permute(0, 1, 4, 3, 2).flatten(2, 3))):
        c = rec[..., at:at + 1024].unflatten(-1, (16, 64)).long()
        x = torch.empty((*c.shape[:-1], D), dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = level[c % 16], level[c // 16]
        x *= scale[sc.long()].repeat_interleave(16, -1)
        out.append(x.transpose(1, 2).flatten(0, 1)[:L])
    return out


def _exact_quantised(x):
    """The values that a token's codes stand for, by the format's definition: nearest of the levels, ties to the even
    code; the quotients are those of the definition, rounded to fp32."""
    f = x.double().unflatten(-1, (8, 16))
    a = (f.abs().amax(-1) / 6).float().double().clamp(max=448.0)
    # E4M3's step at a: an eighth of the power of two below it, and no less than 2^-9
    powers = torch.tensor([2.0 ** k for k in range(-6, 9)], dtype=torch.float64, device=x.device)
    step = powers[(torch.bucketize(a, powers, right=True) - 1).clamp(min=0)] / 8
    s = (torch.round(a / step) * step).clamp(max=448.0)
    inv = torch.where(s == 0, 0.0, (1 / s.clamp(min=2.0 ** -12))).float().double()
    y = (f * inv[..., None]).float().double()
    b = y.abs().clamp(max=6.0)
    step = torch.where(b < 2, 0.5, torch.where(b < 4, 1.0, 2.0))
    q = (torch.round(b / step) * step).clamp(max=6.0)
    return (torch.where(y < 0, -q, q) * s[..., None]).flatten(-2)
