"""Head norms with rotation, the paged MXFP4 cache and reading it back, on the GPU, against numpy."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def mq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import online_hadamard_b200 as m
    m.load_library()
    m.macaq_device_status(clear=True)
    return m


def rows(rng, T, width, gain=12.0):
    x = rng.standard_normal((T, width)) * np.where(rng.random(width) < 0.03, gain, 1.0)
    return kv.bf16(x)


def rope_table(P, R):
    ang = np.arange(P)[:, None] * 1e4 ** (-np.arange(0, R, 2) / R)
    return np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def check_heads(got, x, w, table, R, inter):
    """bf16 outputs against 64 bits: half a bf16 step (2^-8 of the value) for the rounding, and for the
    fp32 arithmetic before it at most 16 roundings of 2^-24 of each of the (two) terms of an element: the norm's
    factor is wrong by at most D/8 + 8 + 4 roundings' worth, 28 at D = 128, of which a sum of squares feels half."""
    ref = kv.norm_rope(x.astype(np.float64), w, EPS, table, R, inter)
    terms = np.abs(ref) if table is None else kv.norm_rope(np.abs(x.astype(np.float64)), w, EPS, np.abs(table), R, inter)
    plus = np.abs(kv.norm_rope(x.astype(np.float64), w, EPS, None, R, inter)).max(-1, keepdims=True)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 40 * 2.0 ** -24 * (np.abs(terms) + 2 * plus)).all(), err.max()


CASES = [  # T, Hq, Hk, D, R (0: none), norm, interleaved, extra columns
    (1, 1, 1, 128, 128, True, False, 0),
    (5, 8, 2, 128, 128, True, False, 256),
    (3, 7, 1, 64, 64, True, True, 64),
    (17, 3, 3, 128, 64, False, False, 8),
    (4, 5, 2, 64, 32, True, False, 0),
    (9, 4, 4, 128, 128, False, True, 0),
    (6, 6, 2, 64, 32, False, True, 0),
    (2, 9, 2, 128, 64, True, True, 0),
    (8, 4, 0, 64, 64, True, False, 0),
    (8, 0, 3, 128, 128, True, False, 0),
    (11, 2, 2, 64, 0, True, False, 0),
    (700, 40, 8, 128, 128, True, False, 1024),
    (1500, 33, 5, 64, 64, True, False, 0),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,norm,inter,extra", CASES)
def test_qk_norm_rope(mq, T, Hq, Hk, D, R, norm, inter, extra):
    rng = np.random.default_rng(T * 131 + D + R)
    x = rows(rng, T, (Hq + Hk) * D + extra)
    wq, wk = (rng.random((2, D)) + 0.5).astype(np.float32)
    P = 977
    table = rope_table(P, R) if R else None
    pos = rng.integers(0, P, T)
    q, k = mq.macaq_qk_norm_rope(cuda(x, torch.bfloat16), Hq, Hk, D, None if table is None else cuda(table), cuda(pos),
                                 q_weight=cuda(wq) if norm else None, k_weight=cuda(wk) if norm else None,
                                 eps=EPS, interleaved=inter)
    heads = x[:, :(Hq + Hk) * D].reshape(T, Hq + Hk, D)
    tr = None if table is None else table[pos]
    if Hq:
        check_heads(q, heads[:, :Hq], wq if norm else None, tr, R, inter)
    if Hk:
        check_heads(k, heads[:, Hq:], wk if norm else None, tr, R, inter)
    assert mq.macaq_device_status() == 0


def test_qk_norm_rope_one_weight_zero_rows_and_no_rows(mq):
    """A norm of the queries only; a head of zeros stays zero (eps keeps the root away from it); T = 0."""
    rng = np.random.default_rng(5)
    x = rows(rng, 4, 3 * 64)
    x[1] = 0
    w = np.full(64, 2.0, np.float32)
    q, k = mq.macaq_qk_norm_rope(cuda(x, torch.bfloat16), 2, 1, 64, q_weight=cuda(w), eps=EPS)
    check_heads(q, x.reshape(4, 3, 64)[:, :2], w, None, 0, False)
    assert torch.equal(k.float().cpu(), torch.from_numpy(x.reshape(4, 3, 64)[:, 2:]))
    assert not q[1].any()
    q, k = mq.macaq_qk_norm_rope(cuda(x[:0], torch.bfloat16), 2, 1, 64)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)


def test_positions_outside_the_table_are_skipped_and_reported(mq):
    rng = np.random.default_rng(6)
    x, table = rows(rng, 4, 5 * 64), rope_table(10, 64)
    pos = np.array([3, 10, -1, 9])
    q = torch.full((4, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((4, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mq.macaq_device_status(clear=True)
    mq.macaq_qk_norm_rope(cuda(x, torch.bfloat16), 3, 1, 64, cuda(table), cuda(pos), q=q, k=k)
    assert mq.macaq_device_status(clear=True) == -9
    assert (q[1:3] == 7).all() and (k[1:3] == 7).all()
    check_heads(q[[0, 3]], x[[0, 3], :192].reshape(2, 3, 64), None, table[pos[[0, 3]]], 64, False)
    cache = torch.zeros(2, 1, mq.kv4_page_bytes(16, 64), dtype=torch.uint8, device="cuda")
    slots = cuda(np.array([0, 1, 2, 32]))  # rows 1 and 2 have bad positions, row 3 a slot outside the cache
    mq.macaq_kv4_append(cuda(x, torch.bfloat16), 3, 1, 64, cache, 16, slots, cuda(table), cuda(pos))
    assert mq.macaq_device_status(clear=True) == -9
    want = np.zeros(cache.shape, np.uint8)
    h = x.reshape(4, 5, 64)
    kv.store(want, [0], 16, kv.norm_rope(h[:1, 3:4], None, EPS, table[pos[:1]], 64, False), h[:1, 4:])
    assert np.array_equal(cache.cpu().numpy(), want)


APPEND = [  # T, Hq, Hk, D, R, norm, interleaved, page, padding rows
    (1, 4, 1, 128, 128, True, False, 16, 0),
    (33, 8, 2, 128, 128, True, False, 32, 4),
    (40, 0, 3, 64, 64, True, True, 16, 7),
    (64, 4, 4, 64, 32, True, False, 64, 0),
    (50, 2, 2, 128, 64, True, False, 128, 5),
    (77, 3, 1, 64, 64, False, False, 128, 1),
    (29, 5, 5, 128, 64, False, True, 64, 29),
    (300, 2, 2, 128, 0, True, False, 16, 13),
    (513, 16, 8, 128, 128, True, False, 128, 0),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,norm,inter,page,pad", APPEND)
def test_append_codes_bit_for_bit(mq, T, Hq, Hk, D, R, norm, inter, page, pad):
    """Every byte of the cache: the stored tokens' codes and scales as numpy's fp32 gives them, all others as
    they were; then the values read back, within the rounding of 64 bits to bf16."""
    rng = np.random.default_rng(T + D + page)
    x = rows(rng, T, (Hq + 2 * Hk) * D + 64, gain=40.0)
    x[0] *= 2.0 ** -60  # far scales are scales like any other
    wq, wk = (rng.random((2, D)) + 0.5).astype(np.float32)
    P = 500
    table = rope_table(P, R) if R else None
    pos = rng.integers(0, P, T)
    pages = (T + page - 1) // page + 2
    slots = rng.permutation(pages * page)[:T]
    slots[rng.permutation(T)[:pad]] = -1 - rng.integers(0, 5)
    before = rng.integers(0, 256, (pages, Hk, kv.page_bytes(page, D))).astype(np.uint8)
    cache = cuda(before)
    xt = cuda(x, torch.bfloat16)
    q = mq.macaq_kv4_append(xt, Hq, Hk, D, cache, page, cuda(slots), None if table is None else cuda(table), cuda(pos),
                            q_weight=cuda(wq) if norm else None, k_weight=cuda(wk) if norm else None, eps=EPS,
                            interleaved=inter)
    heads = x[:, :(Hq + 2 * Hk) * D].reshape(T, Hq + 2 * Hk, D)
    tr = None if table is None else table[pos]
    k = kv.norm_rope(heads[:, Hq:Hq + Hk], wk if norm else None, EPS, tr, R, inter)
    kv.store(before, slots, page, k, heads[:, Hq + Hk:])
    got = cache.cpu().numpy()
    bad = got != before
    assert not bad.any(), f"{bad.sum()} of {bad.size} bytes differ, first at {np.argwhere(bad)[0]}"
    if Hq:
        check_heads(q, heads[:, :Hq], wq if norm else None, tr, R, inter)
    else:
        assert q is None
    K, V = kv.decode(got, page, D)
    gk, gv = mq.macaq_kv4_gather(cache, D, page, cuda(slots))
    for g, full in ((gk, K), (gv, V)):
        ref = np.where((slots >= 0)[:, None, None], full[slots // page, :, slots % page], 0.0)
        # 5 butterfly stages and one factor in fp32: 6 roundings of at most the block's sum of magnitudes
        size = np.abs(ref).reshape(T, Hk, -1, 32).max(-1).repeat(32, -1).reshape(ref.shape) * 32
        assert (np.abs(g.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 6 * 2.0 ** -24 * size).all()
    assert mq.macaq_device_status() == 0


def test_append_ties_zeros_and_negative_zeros(mq):
    """Blocks of zeros (scale 0), of a single spike (every transformed value the same magnitude) and values on
    the rounding boundaries."""
    D, page = 64, 16
    x = np.zeros((6, 2 * D), np.float32)
    x[1, 3], x[1, D + 40] = 4.0, -4.0
    x[2] = np.tile(np.array([1.0, -1.0], np.float32), D)
    x[3, :32] = np.arange(32) - 16
    x[4] = -0.0
    x[5] = np.float32(2.0 ** -126)
    x = kv.bf16(x)
    cache = torch.zeros(1, 1, kv.page_bytes(page, D), dtype=torch.uint8, device="cuda")
    mq.macaq_kv4_append(cuda(x, torch.bfloat16), 0, 1, D, cache, page, cuda(np.arange(6)))
    want = np.zeros(cache.shape, np.uint8)
    h = x.reshape(6, 2, D)
    kv.store(want, range(6), page, h[:, :1], h[:, 1:])
    assert np.array_equal(cache.cpu().numpy(), want)


def test_gather_reports_slots_outside_the_cache(mq):
    cache = torch.full((2, 1, kv.page_bytes(16, 64)), 0x22, dtype=torch.uint8, device="cuda")
    mq.macaq_device_status(clear=True)
    k, v = mq.macaq_kv4_gather(cache, 64, 16, cuda(np.array([31, 32, -5])))
    assert mq.macaq_device_status(clear=True) == -9
    assert k[0].any() and not k[1:].any() and not v[1:].any()
    k, v = mq.macaq_kv4_gather(cache, 64, 16, cuda(np.array([31, -5])))
    assert mq.macaq_device_status() == 0


@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", [(6, 3, 1, 64, 64, False), (9, 16, 2, 128, 64, True), (400, 40, 4, 128, 128, False)])
def test_padding_rows_need_no_position(mq, T, Hq, Hk, D, R, inter):
    """Rows of negative slots whose positions are outside the table, as padding often has them: zero queries, nothing
    stored and nothing reported; with a position of the table they are normed and rotated as before."""
    rng = np.random.default_rng(T)
    x, table = rows(rng, T, (Hq + 2 * Hk) * D), rope_table(50, R)
    w = (rng.random(D) + 0.5).astype(np.float32)
    pos = rng.integers(0, 50, T)
    slots = rng.permutation(T + 32)[:T]
    pad = rng.permutation(T)[:max(3, T // 4)]
    slots[pad] = -1
    pos[pad[:-1]] = rng.choice([-1, 50, 2 ** 40, -2 ** 62], len(pad) - 1)
    page = 32
    cache = torch.zeros((T + 63) // page + 1, Hk, mq.kv4_page_bytes(page, D), dtype=torch.uint8, device="cuda")
    q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    mq.macaq_device_status(clear=True)
    mq.macaq_kv4_append(cuda(x, torch.bfloat16), Hq, Hk, D, cache, page, cuda(slots), cuda(table), cuda(pos), q_weight=cuda(w),
                        eps=EPS, interleaved=inter, q=q)
    assert mq.macaq_device_status(clear=True) == 0
    assert not q[torch.from_numpy(pad[:-1])].any()
    keep = np.setdiff1d(np.arange(T), pad[:-1])
    h = x.reshape(T, Hq + 2 * Hk, D)
    check_heads(q[torch.from_numpy(keep)], h[keep, :Hq], w, table[pos[keep]], R, inter)
    want = np.zeros(cache.shape, np.uint8)
    real = np.flatnonzero(slots >= 0)
    kv.store(want, slots[real], page, kv.norm_rope(h[real, Hq:Hq + Hk], None, EPS, table[pos[real]], R, inter), h[real, Hq + Hk:])
    assert np.array_equal(cache.cpu().numpy(), want)


def test_gather_refuses_slots_that_are_no_row_of_int64(mq):
    cache = torch.zeros(2, 1, mq.kv4_page_bytes(16, 64), dtype=torch.uint8, device="cuda")
    for slots in ([0, 1], torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32, device="cuda"),
                  torch.zeros(1, 2, dtype=torch.int64, device="cuda")):
        with pytest.raises(ValueError, match="slots must"):
            mq.macaq_kv4_gather(cache, 64, 16, slots)
