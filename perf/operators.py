"""What is measured of the attention path around the W4A4 linears: per-head norms with the position
rotation, appending to a paged 4-bit cache, and attention over that cache.

``run`` makes one pass: with ``own`` false in plain torch operations, with ``own`` true through the
package's entry points.  Both work on the same state: bf16 rows of a stacked q/k/v projection, and a
cache whose bytes are laid out as include/macaq.h documents.

The cache of one (page, kv head), P tokens of D = 32 nb elements each, 17 P D / 16 bytes:
  K codes [P][4 c][nb b][4 bytes]       element 32 b + 8 c + j, j = 0..7, two per byte, even j low
  V codes [P/2][8 g][2 r][nb b][2 bytes]  token 2 p + r, element 32 b + 4 g + j, j = 0..3
  K scales [P][nb], V scales [P][nb]    E8M0
and what it holds are MXFP4 codes of FWHT32(x / sqrt(32)).
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
C0 = 0.1767766952966369  # 1 / sqrt(32), rounded to fp32 where it is used
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one step of eight running requests, heads of Qwen3-32B (64 query, 8 key heads, norms): latency
        dict(name="norm_rope_step", kind="norm_rope", T=8, Hq=64, Hk=8, D=128, R=128, norm=True, inter=False, pos=40000),
        # a prompt of the same model
        dict(name="norm_rope_prompt", kind="norm_rope", T=4096, Hq=64, Hk=8, D=128, R=128, norm=True, inter=False, pos=8192),
        # an odd number of rows, small heads, half of each head rotated, neighbouring pairs
        dict(name="norm_rope_partial", kind="norm_rope", T=1237, Hq=24, Hk=4, D=64, R=32, norm=False, inter=True, pos=4096),
        # one step of 64 running requests, heads of Llama-3-8B (32 / 8, no norms), each into its own page
        dict(name="append_step", kind="append", T=64, Hq=32, Hk=8, D=128, R=128, norm=False, inter=False, pos=8192, page=64, pad=3),
        # a prompt of Qwen3-32B into pages of 128
        dict(name="append_prompt", kind="append", T=4096, Hq=64, Hk=8, D=128, R=128, norm=True, inter=False, pos=8192, page=128, pad=0),
        # rows of many short prompts with padding between them, as many key as query heads, small pages
        dict(name="append_ragged", kind="append", T=777, Hq=20, Hk=20, D=64, R=64, norm=True, inter=False, pos=2048, page=16, pad=31),
        # a single request, a short context: latency
        dict(name="decode_one", kind="attend", B=1, nq=1, ctx=2047, even=True, Hq=64, Hk=8, D=128, page=128, window=0),
        # a running batch of unequal contexts, heads of Llama-3-8B
        dict(name="decode_batch", kind="attend", B=32, nq=1, ctx=8000, even=False, Hq=32, Hk=8, D=128, page=64, window=0),
        # long contexts, heads of Qwen3-32B: the cache's bytes
        dict(name="decode_long", kind="attend", B=16, nq=1, ctx=32768, even=True, Hq=64, Hk=8, D=128, page=128, window=0),
        # verifying four drafted tokens a request in a sliding window, small heads and pages
        dict(name="verify_window", kind="attend", B=24, nq=4, ctx=6001, even=False, Hq=16, Hk=2, D=64, page=16, window=1024),
        # a whole prompt
        dict(name="prompt", kind="attend", B=1, nq=8192, ctx=8192, even=True, Hq=32, Hk=8, D=128, page=128, window=0),
        # chunks of prompts behind prefixes of unequal length, heads of Qwen3-32B
        dict(name="prompt_chunks", kind="attend", B=5, nq=509, ctx=6000, even=False, Hq=64, Hk=8, D=128, page=32, window=0),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is spread evenly between lo and hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice((64, 128, 128))
    Hk = rng.choice((1, 2, 4, 8))
    Hq = Hk * rng.choice((1, 2, 4, 7, 8))
    kind = rng.choice(("norm_rope", "append", "attend", "attend", "prompt"))
    if kind in ("norm_rope", "append"):
        T = _spread(rng, 1, 4096)
        case = dict(kind=kind, T=T, Hq=Hq, Hk=Hk, D=D, R=rng.choice((D, D, D // 2)), norm=rng.random() < 0.6,
                    inter=rng.random() < 0.3, pos=_spread(rng, 256, 100000))
        if kind == "append":
            case.update(page=rng.choice((16, 32, 64, 128)), pad=rng.choice((0, T // 8)))
        return case
    window = rng.choice((0, 0, 0, _spread(rng, 16, 4096)))
    page, even = rng.choice((16, 32, 64, 128)), rng.random() < 0.3
    if kind == "attend":  # few queries a sequence
        B, ctx = _spread(rng, 1, 48), _spread(rng, 1, 8192)
        nq = rng.choice((1, 1, 1, 2, 5))
        return dict(kind="attend", B=B, nq=nq, ctx=max(ctx, nq), even=even, Hq=Hq, Hk=Hk, D=D, page=page, window=window)
    nq = _spread(rng, 16, 1024)
    return dict(kind="attend", B=rng.choice((1, 2, 3)), nq=nq, ctx=nq + rng.choice((0, _spread(rng, 1, 4096))), even=even,
                Hq=Hq, Hk=Hk, D=D, page=page, window=window)


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rope_table(P, R):
    """fp32 [P, R]: cos of the R/2 angles, then their sines; angles in 64 bits."""
    inv = 1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), 1).float()


def _rows(g, T, H, D):
    """bf16 [T, H D] of a projection: normal, a few channels of each head much larger."""
    x = torch.randn(T, H, D, generator=g, device="cuda")
    gain = torch.where(torch.rand(H, D, generator=g, device="cuda") < 0.02, 12.0, 1.0)
    return (x * gain).reshape(T, H * D).to(torch.bfloat16)


def _lengths(case, g):
    """Per sequence: the keys in the cache and the queries, which are the last of them."""
    B, ctx, nq = case["B"], case["ctx"], case["nq"]
    if case["even"]:
        kv = torch.full((B,), ctx, dtype=torch.int64, device="cuda")
        q = torch.full((B,), nq, dtype=torch.int64, device="cuda")
    else:
        lo = max(1, ctx // 8)
        kv = torch.randint(lo, ctx + 1, (B,), generator=g, device="cuda")
        kv[0] = ctx
        # the queries' lengths, and with them the shapes, are the case's own and not the seed's
        q = torch.full((B,), nq, dtype=torch.int64, device="cuda") if nq < 16 else \
            torch.randint(1, nq + 1, (B,), generator=_gen(nq), device="cuda")
        q[0] = nq
        kv = torch.maximum(kv, q)
    return kv.to(torch.int32), q.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    if case["kind"] != "attend":
        T, P = case["T"], case["pos"]
        st = dict(case=case, qkv=_rows(g, T, Hq + 2 * Hk, D), rope=_rope_table(P, case["R"]),
                  positions=torch.randint(0, P, (T,), generator=g, device="cuda"), wq=None, wk=None)
        if case["norm"]:
            st["wq"] = torch.rand(D, generator=g, device="cuda") + 0.5
            st["wk"] = torch.rand(D, generator=g, device="cuda") + 0.5
        if case["kind"] == "append":
            page = case["page"]
            pages = (T + page - 1) // page + 4
            st["cache"] = torch.zeros(pages, Hk, page * D * 17 // 16, dtype=torch.uint8, device="cuda")
            slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
            if T > 256:  # a prompt fills whole pages, in any order of pages
                order = torch.randperm(pages, generator=g, device="cuda")
                at = torch.arange(T, device="cuda")
                slots = order[at // page] * page + at % page
            if case["pad"]:
                slots[torch.randperm(T, generator=g, device="cuda")[:case["pad"]]] = -1
            st["slots"] = slots
        return st
    page, B = case["page"], case["B"]
    kv_lens, q_lens = _lengths(case, g)
    width = (case["ctx"] + page - 1) // page
    order = torch.randperm(B * width, generator=g, device="cuda")
    tables = order.reshape(B, width).to(torch.int32)
    cache = torch.zeros(B * width, Hk, page * D * 17 // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (width * page * Hk * D))
    for b in range(0, B, step):  # whole pages of a few sequences at a time
        n = min(step, B - b)
        slots = (tables[b:b + n].long()[:, :, None] * page + torch.arange(page, device="cuda")).reshape(-1)
        gain = torch.where(torch.rand(2, Hk, D, generator=g, device="cuda") < 0.02, 6.0, 1.0)
        k = torch.randn(len(slots), Hk, D, generator=g, device="cuda") * gain[0]
        v = torch.randn(len(slots), Hk, D, generator=g, device="cuda") * gain[1]
        _store(cache, slots, page, k, v)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.cumsum(q_lens, 0)
    T = int(cu[-1])
    q = torch.randn(T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    return dict(case=case, q=q, cache=cache, tables=tables, kv_lens=kv_lens, cu=cu, scale=D ** -0.5)


# --------------------------------------------------------------------------------- plain forms

def _stage(x, h):
    x = x.unflatten(-1, (BLOCK // (2 * h), 2, h))
    a, b = x[..., 0, :], x[..., 1, :]
    return torch.stack((a + b, a - b), -2).flatten(-3)


def _transform(x):
    """[..., D] fp32 -> [..., D/32, 32]: times 1/sqrt(32), then the butterfly of distances 1, 2, 4, 8, 16."""
    x = (x * torch.tensor(C0, dtype=torch.float32, device=x.device)).unflatten(-1, (-1, BLOCK))
    return _stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16)


def _untransform(x):
    """[..., D/32, 32] fp32 -> [..., D]."""
    x = _stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16)
    return (x * torch.tensor(C0, dtype=torch.float32, device=x.device)).flatten(-2)


def _codes(v):
    """MXFP4 of [..., nb, 32]: codes (sign << 3 | index) and E8M0 bytes."""
    amax = v.abs().amax(-1)
    e = (((amax.view(torch.int32) >> 23) & 0xFF) - 2).clamp_min(0)
    m = v.abs() * ((254 - e) << 23).view(torch.float32)[..., None]
    index = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (index + 8 * torch.signbit(v)).to(torch.uint8), e.to(torch.uint8)


def _store(cache, slots, page, k, v):
    """Writes fp32 k, v [T, Hk, D] (before the transform) into the slots of the cache."""
    D = k.shape[-1]
    nb = D // BLOCK
    kc, ks = _codes(_transform(k))
    vc, vs = _codes(_transform(v))
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).unflatten(-1, (4, 4)).transpose(-3, -2)   # [T, Hk, c, b, 4]
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).unflatten(-1, (8, 2)).transpose(-3, -2)   # [T, Hk, g, b, 2]
    n = page * D // 2
    p, at = slots // page, slots % page
    cache[:, :, :n].unflatten(-1, (page, 4, nb, 4))[p, :, at] = kb
    cache[:, :, n:2 * n].unflatten(-1, (page // 2, 8, 2, nb, 2))[p, :, at // 2, :, at % 2] = vb
    cache[:, :, 2 * n:2 * n + page * nb].unflatten(-1, (page, nb))[p, :, at] = ks
    cache[:, :, 2 * n + page * nb:].unflatten(-1, (page, nb))[p, :, at] = vs


def _decode(codes, scales):
    """uint8 [..., nb, 16] packed codes and [..., nb] scales -> fp32 [..., nb, 32]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return table[c.long()] * (scales.int() << 23).view(torch.float32)[..., None]


def _read(cache, slots, page, D):
    """The transformed K and V, fp32 [T, Hk, nb, 32], of the given slots."""
    nb = D // BLOCK
    n = page * D // 2
    p, at = slots // page, slots % page
    kb = cache[:, :, :n].unflatten(-1, (page, 4, nb, 4))[p, :, at].transpose(-3, -2).flatten(-2)
    vb = cache[:, :, n:2 * n].unflatten(-1, (page // 2, 8, 2, nb, 2))[p, :, at // 2, :, at % 2].transpose(-3, -2).flatten(-2)
    ks = cache[:, :, 2 * n:2 * n + page * nb].unflatten(-1, (page, nb))[p, :, at]
    vs = cache[:, :, 2 * n + page * nb:].unflatten(-1, (page, nb))[p, :, at]
    return _decode(kb, ks), _decode(vb, vs)


def _sum_squares(x):
    """Over the last axis, neighbours first: distances 1, 2, 4, ... (the order of the entry points)."""
    s = x * x
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    s = s[..., 0::2] + s[..., 1::2]
    return s[..., 0::2] + s[..., 1::2] if s.shape[-1] == 2 else s


def _norm_rope(x, w, table, inter):
    """fp32 [T, H, D] heads -> normed (w not None) and rotated."""
    if w is not None:
        r = 1.0 / torch.sqrt(_sum_squares(x) * (1.0 / x.shape[-1]) + torch.tensor(1e-6, device=x.device))
        x = x * r * w
    half = table.shape[-1] // 2
    c, s = table[:, None, :half], table[:, None, half:]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((rot, rest), -1)


def _attend(st):
    c = st["case"]
    D, Hq, Hk, page, B = c["D"], c["Hq"], c["Hk"], c["page"], c["B"]
    q, cu, kv = st["q"], st["cu"].long(), st["kv_lens"].long()
    width = st["tables"].shape[1]
    L = width * page
    slots = (st["tables"].long()[:, :, None] * page + torch.arange(page, device=q.device)).reshape(-1)
    k, v = _read(st["cache"], slots, page, D)
    k = k.reshape(B, L, Hk, D).permute(0, 2, 3, 1)     # [B, Hk, D, L]
    v = v.reshape(B, L, Hk, D).permute(0, 2, 1, 3)     # [B, Hk, L, D]
    # the queries of each sequence, padded to the longest
    n = cu[1:] - cu[:-1]
    N = c["nq"]
    at = torch.arange(N, device=q.device)
    real = at < n[:, None]
    row = torch.where(real, cu[:-1, None] + at, 0)
    qt = _transform(q.float()).flatten(-2)[row]        # [B, N, Hq, D]
    qt = qt.reshape(B, N, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, Hq // Hk * N, D)
    s = torch.matmul(qt, k) * st["scale"]
    s = s.reshape(B, Hk, Hq // Hk, N, L)
    pos = (kv - n)[:, None] + at                       # [B, N]
    j = torch.arange(L, device=q.device)
    seen = (j <= pos[..., None]) & real[..., None]
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.reshape(B, Hk, -1, L), v).reshape(B, Hk, Hq // Hk, N, D // BLOCK, BLOCK)
    o = _untransform(o).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    return o[real].to(torch.bfloat16)


def run(st):
    c = st["case"]
    D, Hq, Hk = c["D"], c["Hq"], c["Hk"]
    if own:
        import online_hadamard_b200 as mq
        if c["kind"] == "norm_rope":
            return mq.macaq_qk_norm_rope(st["qkv"], Hq, Hk, D, st["rope"], st["positions"], q_weight=st["wq"],
                                         k_weight=st["wk"], interleaved=c["inter"])
        if c["kind"] == "append":
            q = mq.macaq_kv4_append(st["qkv"], Hq, Hk, D, st["cache"], c["page"], st["slots"], st["rope"],
                                    st["positions"], q_weight=st["wq"], k_weight=st["wk"], interleaved=c["inter"])
            return (q, *mq.macaq_kv4_gather(st["cache"], D, c["page"], st["slots"]))
        return mq.macaq_kv4_attention(st["q"], st["cache"], c["page"], st["tables"], st["kv_lens"], st["cu"],
                                      max_q=c["nq"], scale=st["scale"], window=c["window"])
    if c["kind"] == "attend":
        return _attend(st)
    T = c["T"]
    x = st["qkv"].float().reshape(T, Hq + 2 * Hk, D)
    table = st["rope"][st["positions"]]
    q = _norm_rope(x[:, :Hq], st["wq"], table, c["inter"]).to(torch.bfloat16)
    k = _norm_rope(x[:, Hq:Hq + Hk], st["wk"], table, c["inter"])
    if c["kind"] == "norm_rope":
        return q, k.to(torch.bfloat16)
    slots = st["slots"]
    real = slots >= 0
    _store(st["cache"], slots[real], c["page"], k[real], x[real, Hq + Hk:])
    kr, vr = _read(st["cache"], slots.clamp_min(0), c["page"], D)
    gone = ~real[:, None, None]
    return (q, _untransform(kr).masked_fill(gone, 0).to(torch.bfloat16),
            _untransform(vr).masked_fill(gone, 0).to(torch.bfloat16))


# ---------------------------------------------------------------------------------------- work

def work(case):
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    if case["kind"] != "attend":
        T = case["T"]
        table = 4 * case["R"] * min(T, case["pos"]) + 8 * T
        if case["kind"] == "norm_rope":
            return {"bytes": 4.0 * T * (Hq + Hk) * D + table, "flops": 10.0 * T * (Hq + Hk) * D}
        T1 = T - case["pad"]
        cached = 2.0 * T1 * Hk * D * 17 / 32
        # q in and out, K and V in, the cache written and read back, the values read back written
        return {"bytes": 4.0 * T * Hq * D + 4.0 * T1 * Hk * D + 2 * cached + 4.0 * T * Hk * D + table + 8 * T,
                "flops": 10.0 * T * (Hq + Hk) * D + 20.0 * T1 * Hk * D}
    B, nq, ctx, window = case["B"], case["nq"], case["ctx"], case["window"]
    share = 1.0 if case["even"] else (1.0 + 0.5625 * (B - 1)) / B    # lengths between ctx / 8 and ctx
    qshare = 1.0 if case["even"] or nq < 16 else (1.0 + 0.5 * (B - 1)) / B
    kv, n = ctx * share, nq * qshare
    keys = min(kv, window + n) if window else kv                     # keys that any query sees
    pairs = sum(min(window, kv - n + i + 1) if window else kv - n + i + 1 for i in range(max(1, int(n))))
    return {"bytes": B * (2 * keys * Hk * D * 17 / 32 + 4.0 * n * Hq * D + 4 * kv / case["page"] + 8),
            "flops": 4.0 * B * max(pairs, 1.0) * Hq * D}


# --------------------------------------------------------------------------------------- exact

def _exact_table():
    i = torch.arange(32, device="cuda")
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(5)) % 2
    return (1.0 - 2.0 * odd).double() / math.sqrt(32.0)


def _exact_mx(v):
    """fp64 values that the MXFP4 codes of [..., 32] stand for."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=v.device)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    e = torch.where(torch.exp2(e) > amax, e - 1, torch.where(torch.exp2(e + 1) <= amax, e + 1, e))
    x = torch.where(amax > 0, torch.exp2(e - 2), 1.0)
    m = v.abs() / x
    up = torch.bucketize(m, grid).clamp(1, 7)
    lo, hi = grid[up - 1], grid[up]
    near = torch.where((m - lo < hi - m) | ((m - lo == hi - m) & ((up - 1) % 2 == 0)), lo, hi)
    return torch.copysign(near * x, v)


def _exact_cache(cache, page, D, which):
    """fp64 [pages, Hk, P, D] values of K (which 0) or V (1), each by its byte's place."""
    nb = D // 32
    t = torch.arange(page, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")[None, :]
    b, i = d // 32, d % 32
    if which == 0:
        place, low = t * (D // 2) + (i // 8) * 4 * nb + b * 4 + (i % 8) // 2, i % 2 == 0
    else:
        place = page * D // 2 + (t // 2) * D + (i // 4) * 4 * nb + (t % 2) * 2 * nb + b * 2 + (i % 4) // 2
        low = i % 2 == 0
    byte = cache[:, :, place.reshape(-1)].reshape(*cache.shape[:2], page, D)
    code = torch.where(low, byte & 15, byte >> 4).long()
    scale = cache[:, :, (page * D + which * page * nb + t * nb + b).reshape(-1)].reshape(*cache.shape[:2], page, D)
    values = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64, device="cuda")
    out = values[code] * torch.exp2(scale.double() - 127)
    return torch.matmul(out.unflatten(-1, (nb, 32)), _exact_table()).flatten(-2)


def _exact_heads(st, lo, hi, w):
    c = st["case"]
    T, D, R = c["T"], c["D"], c["R"]
    x = st["qkv"].double().reshape(T, -1, D)[:, lo:hi]
    if w is not None:
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * w.double()
    row = st["rope"].double()[st["positions"]]
    y = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + R // 2)
        cs, sn = row[:, None, i], row[:, None, R // 2 + i]
        y[..., a] = x[..., a] * cs - x[..., b] * sn
        y[..., b] = x[..., b] * cs + x[..., a] * sn
    return y


def exact(case, seed):
    if case["kind"] == "attend" and case["Hk"] * case["B"] * case["ctx"] * case["D"] > 1 << 30:
        return None
    st = prepare(case, seed)
    D, Hq, Hk = case["D"], case["Hq"], case["Hk"]
    if case["kind"] != "attend":
        q = _exact_heads(st, 0, Hq, st["wq"])
        k = _exact_heads(st, Hq, Hq + Hk, st["wk"])
        if case["kind"] == "norm_rope":
            return q, k
        v = st["qkv"].double().reshape(case["T"], -1, D)[:, Hq + Hk:]
        H, there = _exact_table(), (st["slots"] >= 0)[:, None, None]

        def held(x):
            x = torch.matmul(_exact_mx(torch.matmul(x.unflatten(-1, (-1, 32)), H)), H).flatten(-2)
            return torch.where(there, x, 0.0)
        return q, held(k), held(v)
    K = _exact_cache(st["cache"], case["page"], D, 0)
    V = _exact_cache(st["cache"], case["page"], D, 1)
    cu, kv = st["cu"].tolist(), st["kv_lens"].tolist()
    out = torch.zeros(cu[-1], Hq, D, dtype=torch.float64, device="cuda")
    G = Hq // Hk
    for b in range(case["B"]):
        pages = st["tables"][b].long()
        n, L = cu[b + 1] - cu[b], kv[b]
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        seen = (j <= pos) & ((j > pos - case["window"]) if case["window"] else (j >= 0))
        for h in range(Hk):
            k = K[pages, h].reshape(-1, D)[:L]
            v = V[pages, h].reshape(-1, D)[:L]
            q = st["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()     # [n, G, D]
            s = torch.einsum("ngd,ld->gnl", q, k) * st["scale"]
            s = torch.where(seen, s, -math.inf)
            p = torch.softmax(s, -1)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", p, v)
    return out
