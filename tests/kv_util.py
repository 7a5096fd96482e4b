"""Plain numpy forms of the attention path: head norm and rotation, the paged MXFP4 cache (written
from the documentation in include/macaq.h) and attention over it.  fp32 where the library promises
codes bit for bit (numpy rounds every fp32 operation once), 64 bits elsewhere."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
C0 = np.float32(1.0 / np.sqrt(32.0))


def bf16(x):
    """fp32 values of x rounded to bf16 (to nearest, ties to even), finite x."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32)


def hadamard(x):
    """Unnormalised FWHT-32 of the last axis in x's own type, stages 1, 2, 4, 8, 16."""
    x = x.copy()
    for h in (1, 2, 4, 8, 16):
        v = x.reshape(*x.shape[:-1], 32 // (2 * h), 2, h)
        a, b = v[..., 0, :].copy(), v[..., 1, :].copy()
        v[..., 0, :], v[..., 1, :] = a + b, a - b
    return x


def norm_rope(x, w, eps, table, R, interleaved):
    """x [T, H, D] (fp32 or fp64), table rows [T, R] or None; every operation in x's type."""
    t = x.dtype.type
    D = x.shape[-1]
    if w is not None:
        s = x * x
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        r = t(1) / np.sqrt(s * t(1.0 / D) + t(np.float32(eps)))
        x = (x * r) * w.astype(t)
    if table is None:
        return x
    y = x.copy()
    c, s = table[:, None, :R // 2].astype(t), table[:, None, R // 2:].astype(t)
    i = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]] = a * c - b * s
    y[..., i[1]] = b * c + a * s
    return y


def quantise(y):
    """MXFP4 of the transform of fp32 y [.., D]: codes [.., D/32, 32] uint8 and scales [.., D/32]."""
    v = hadamard((y.astype(np.float32) * C0).reshape(*y.shape[:-1], -1, 32))
    E = (np.abs(v).max(-1).view(np.uint32) >> 23) & 0xFF
    e = np.maximum(E.astype(np.int64) - 2, 0)
    m = np.abs(v).astype(np.float64) * np.exp2(127.0 - e)[..., None]
    d = np.abs(m[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    tied = d == best
    idx = np.where(tied & (np.arange(8) % 2 == 0), 1, np.where(tied, 0, -1))
    return (idx.argmax(-1) + 8 * np.signbit(v)).astype(np.uint8), e.astype(np.uint8)


def offsets(page, D):
    """Byte offsets inside a (page, head) of element d of token t, [page, D], and of the scale of
    block b, [page, D/32], for K and V; the nibble is d % 2."""
    nb = D // 32
    t, d = np.arange(page)[:, None], np.arange(D)[None, :]
    b, i = d // 32, d % 32
    kc = t * (D // 2) + (i // 8) * 4 * nb + 4 * b + (i % 8) // 2
    vc = page * D // 2 + (t // 2) * D + (i // 4) * 4 * nb + (t % 2) * 2 * nb + 2 * b + (i % 4) // 2
    sb = t * nb + np.arange(nb)[None, :]
    return (kc, page * D + sb), (vc, page * D + page * nb + sb)


def page_bytes(page, D):
    return page * D * 17 // 16


def store(cache, slots, page, k, v):
    """Writes fp32 k, v [T, Hk, D] into cache [pages, Hk, bytes] (numpy, in place)."""
    D = k.shape[-1]
    for (place, sp), x in zip(offsets(page, D), (k, v)):
        c, e = quantise(x)
        c = c.reshape(*c.shape[:2], D)
        for t, s in enumerate(slots):
            if s < 0:
                continue
            row = cache[s // page]
            row[:, place[s % page, 0::2]] = c[t, :, 0::2] | (c[t, :, 1::2] << 4)
            row[:, sp[s % page]] = e[t]


def decode(cache, page, D):
    """fp64 K and V [pages, Hk, page, D] (transformed back) that a cache holds."""
    out = []
    for place, sp in offsets(page, D):
        byte = cache[:, :, place.ravel()].reshape(*cache.shape[:2], page, D)
        code = np.where(np.arange(D) % 2 == 0, byte & 15, byte >> 4)
        x = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
        e = cache[:, :, sp.ravel()].reshape(*cache.shape[:2], page, -1).astype(np.float64)
        x = x.reshape(*x.shape[:-1], -1, 32) * np.exp2(e - 127)[..., None]
        out.append((hadamard(x) / np.sqrt(32.0)).reshape(*x.shape[:-2], D))
    return out


def attend(q, K, V, tables, kv_lens, cu, scale, window, out):
    """Attention in 64 bits of q [T, Hq, D] over decoded pages; out [T, Hq, D] keeps its rows outside
    every sequence.  Returns (out, lse, spread): spread bounds, for each row, what an output element can
    move by when every score moves by one unit (twice the largest |v| seen)."""
    T, Hq, D = q.shape
    Hk, page = K.shape[1], K.shape[2]
    G = Hq // Hk
    out = out.astype(np.float64)
    lse = np.full((T, Hq), np.nan)
    spread = np.zeros((T, Hq))
    for b in range(len(kv_lens)):
        L, n = int(kv_lens[b]), int(cu[b + 1] - cu[b])
        j = np.arange(L)
        pages = tables[b][j // page] if L else np.zeros(0, np.int64)
        k = K[pages, :, j % page] if L else np.zeros((0, Hk, D))
        v = V[pages, :, j % page] if L else np.zeros((0, Hk, D))
        for i in range(n):
            pos, t = L - n + i, int(cu[b]) + i
            seen = (j <= pos) & ((j > pos - window) if window else True)
            for h in range(Hq):
                if not seen.any():
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                s = k[seen, h // G] @ q[t, h] * scale
                p = np.exp(s - s.max())
                out[t, h] = (p / p.sum()) @ v[seen, h // G]
                lse[t, h] = s.max() + np.log(p.sum())
                spread[t, h] = 2 * np.abs(v[seen, h // G]).max()
    return out, lse, spread
