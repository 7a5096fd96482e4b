"""The cache and attention calls refuse bad arguments before any CUDA call, and the documented cache
layout is a bijection (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import online_hadamard_b200 as mq
from tests import kv_util as kv

FAKE, MIS = 0x10000, 0x10008
P = ctypes.c_void_p


def lib():
    return mq.load_library()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_cache_layout_covers_the_page_once(D, page):
    n = mq.kv4_page_bytes(page, D)
    assert n == kv.page_bytes(page, D)
    (kc, ks), (vc, vs) = kv.offsets(page, D)
    nibbles = np.concatenate([(c * 2 + np.arange(D) % 2).ravel() for c in (kc, vc)])
    assert np.array_equal(np.sort(nibbles), np.arange(2 * page * D))
    assert np.array_equal(np.sort(np.concatenate((ks.ravel(), vs.ravel()))), np.arange(page * D, n))


def test_page_bytes_refuses_other_sizes():
    assert mq.kv4_page_bytes(8, 128) == 0 and mq.kv4_page_bytes(48, 128) == 0 and mq.kv4_page_bytes(256, 64) == 0
    assert mq.kv4_page_bytes(16, 96) == 0 and mq.kv4_page_bytes(16, 256) == 0


def test_norm_rope_validation():
    def call(qkv=FAKE, T=4, ld=640, Hq=4, Hk=1, D=128, wq=FAKE, wk=FAKE, eps=1e-6, rope=FAKE, rows=10, R=128, inter=0,
             pos=FAKE, q=FAKE, k=FAKE):
        return lib().macaq_qk_norm_rope(P(qkv), T, ld, Hq, Hk, D, P(wq), P(wk), eps, P(rope), rows, R, inter, P(pos),
                                        P(q), P(k), None)
    assert call(qkv=0) == -1 and call(q=0) == -1 and call(k=0) == -1 and call(pos=0) == -1
    assert call(inter=2) == -1 and call(eps=-1.0) == -1 and call(eps=float("nan")) == -1 and call(eps=float("inf")) == -1
    assert call(D=96) == -2 and call(T=-1) == -2 and call(ld=632) == -2 and call(ld=644) == -2
    assert call(Hq=-1) == -2 and call(Hq=0, Hk=0) == -2 and call(Hq=2000, ld=1 << 20) == -2
    assert call(R=32) == -2 and call(rows=0) == -2
    assert call(qkv=MIS) == -3 and call(q=MIS) == -3 and call(wq=MIS) == -3 and call(rope=MIS) == -3
    assert call(pos=FAKE + 4) == -3
    assert call(T=0, qkv=0, q=0, k=0) == 0


def test_append_validation():
    def call(qkv=FAKE, T=4, ld=768, Hq=4, Hk=1, D=128, wk=FAKE, rope=FAKE, rows=10, R=128, pos=FAKE, cache=FAKE,
             pages=4, page=16, slots=FAKE, q=FAKE, inter=0):
        return lib().macaq_kv4_append(P(qkv), T, ld, Hq, Hk, D, P(FAKE), P(wk), 1e-6, P(rope), rows, R, inter, P(pos),
                                      P(cache), pages, page, P(slots), P(q), None)
    assert call(qkv=0) == -1 and call(cache=0) == -1 and call(slots=0) == -1 and call(q=0) == -1 and call(pos=0) == -1
    assert call(inter=-1) == -1
    assert call(ld=760) == -2          # no room for the value heads
    assert call(Hk=0) == -2 and call(page=24) == -2 and call(pages=0) == -2 and call(D=80) == -2
    assert call(cache=MIS) == -3 and call(slots=FAKE + 4) == -3
    assert call(T=0, qkv=0, cache=0, slots=0, q=0) == 0


def test_gather_validation():
    def call(cache=FAKE, pages=4, page=16, Hk=1, D=128, slots=FAKE, T=3, k=FAKE, v=FAKE):
        return lib().macaq_kv4_gather(P(cache), pages, page, Hk, D, P(slots), T, P(k), P(v), None)
    assert call(cache=0) == -1 and call(slots=0) == -1 and call(k=0) == -1 and call(v=0) == -1
    assert call(D=32) == -2 and call(page=0) == -2 and call(Hk=0) == -2 and call(T=-2) == -2 and call(pages=0) == -2
    assert call(k=MIS) == -3 and call(cache=MIS) == -3 and call(slots=FAKE + 2) == -3
    assert call(T=0, cache=0) == 0


def test_attention_validation():
    def call(q=FAKE, T=4, ldq=512, Hq=4, Hk=2, D=128, cache=FAKE, pages=4, page=16, tables=FAKE, B=2, width=8,
             lens=FAKE, cu=FAKE, max_q=3, scale=0.1, window=0, out=FAKE, lse=0, ws=FAKE, wsb=1 << 40):
        return lib().macaq_kv4_attention(P(q), T, ldq, Hq, Hk, D, P(cache), pages, page, P(tables), B, width, P(lens),
                                         P(cu), max_q, scale, window, P(out), P(lse), P(ws), wsb, None)
    assert call(q=0) == -1 and call(cache=0) == -1 and call(tables=0) == -1 and call(lens=0) == -1
    assert call(out=0) == -1 and call(ws=0) == -1
    assert call(scale=0.0) == -1 and call(scale=-1.0) == -1 and call(scale=float("nan")) == -1
    assert call(scale=float("inf")) == -1
    assert call(D=96) == -2 and call(Hq=5) == -2 and call(Hk=0) == -2 and call(Hq=2048, ldq=1 << 20) == -2
    assert call(page=20) == -2 and call(pages=0) == -2 and call(width=-1) == -2 and call(width=1 << 30) == -2
    assert call(ldq=504) == -2 and call(ldq=516) == -2 and call(window=-1) == -2 and call(max_q=0) == -2
    assert call(T=-1) == -2 and call(B=-1) == -2
    assert call(cu=0) == -2            # B != T without query ranges
    assert call(q=MIS) == -3 and call(out=MIS) == -3 and call(cache=MIS) == -3 and call(lens=FAKE + 2) == -3
    assert call(cu=FAKE + 1) == -3 and call(lse=FAKE + 2) == -3 and call(tables=FAKE + 2) == -3 and call(ws=MIS) == -3
    assert call(wsb=0) == -6
    assert call(T=0, q=0, out=0) == 0 and call(B=0, T=0, lens=0, cu=FAKE) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 6 * 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mq.macaq_qk_norm_rope(x, 4, 2, 64)
    cache = torch.zeros(2, 1, mq.kv4_page_bytes(16, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mq.macaq_kv4_append(x, 4, 1, 64, cache, 16, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        mq.macaq_kv4_gather(cache, 64, 16, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        mq.macaq_kv4_attention(x.reshape(2, 6, 64), cache, 16, torch.zeros(2, 1, dtype=torch.int32),
                               torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="heads, head_dim"):
        mq.macaq_kv4_attention(x, cache, 16, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_status_string_of_index_events():
    assert mq.status_str(-9).startswith("MACAQ_EINDEX")


def test_attention_counts_stay_in_their_bits():
    """Sizes whose work could not be counted are refused: queries, units, keys of a sequence."""
    def need(T=8, B=8, Hq=64, Hk=8, D=128, max_q=1):
        return lib().macaq_kv4_attention_workspace_bytes(T, B, Hq, Hk, D, max_q)
    assert need() > 0 and need(max_q=1 << 20) > 0
    assert need(max_q=1 << 21) == 0 and need(B=1 << 30) == 0 and need(B=1 << 20, max_q=1 << 20) == 0
    assert need(Hq=65) == 0 and need(D=32) == 0 and need(max_q=0) == 0 and need(T=-1) == 0
    ok = dict(q=FAKE, T=4, ldq=512, Hq=4, Hk=2, D=128, cache=FAKE, pages=4, page=16, tables=FAKE, B=2, width=(1 << 26) + 1)
    assert lib().macaq_kv4_attention(P(ok["q"]), 4, 512, 4, 2, 128, P(FAKE), 4, 16, P(FAKE), 2, ok["width"], P(FAKE),
                                     P(FAKE), 3, 0.1, 0, P(FAKE), None, P(FAKE), 1 << 40, None) == -2
