"""Attention over the paged MXFP4 cache at the edges of its kernels: many sequences, the row counts where another
kernel takes over, ranges cut between CTAs, absent pages, foreign bytes, far pages, non-finite queries."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv
from tests.test_gpu_kv_attention import Problem, cuda, mq  # noqa: F401  (mq is a fixture)

pytestmark = pytest.mark.gpu


def test_many_sequences_one_unit_a_cta(mq):
    """More units than are cut: every (sequence, kv head) is one CTA's; some sequences hold no key."""
    rng = np.random.default_rng(20)
    seqs = [(int(n), 1) for n in rng.integers(0, 70, 230)]
    Problem(seqs, 8, 8, 64, 16, seed=21).check(mq)


def test_many_sequences_of_several_queries(mq):
    rng = np.random.default_rng(22)
    seqs = [(int(n), int(min(4, m))) for n, m in zip(rng.integers(0, 45, 150), rng.integers(0, 6, 150))]
    Problem(seqs, 64, 8, 64, 32, seed=23).check(mq)


@pytest.mark.parametrize("rows", [9, 16, 17, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 513])
@pytest.mark.parametrize("D", [64, 128])
def test_row_counts_around_the_tiles(mq, rows, D):
    """One kv head of `rows` query rows: one query of as many heads, or as many queries of one."""
    heads = rows if rows < 129 else 1
    Problem([(190, rows // heads), (max(33, rows // heads), rows // heads)], heads, 1, D, 64, seed=rows).check(mq)


@pytest.mark.parametrize("window", [1, 63, 64, 65, 130, 300])
@pytest.mark.parametrize("D,page", [(64, 128), (128, 16)])
def test_windows_over_long_prompts(mq, window, D, page):
    """Windows that begin and end inside blocks, and leave whole blocks out."""
    Problem([(700, 300), (150, 150)], 4, 2, D, page, seed=window).check(mq, window)


def test_long_contexts_of_few_and_many_rows(mq):
    """Units cut over many CTAs and joined."""
    Problem([(4001, 1)], 4, 1, 64, 128, seed=30).check(mq)
    Problem([(3000, 70), (2500, 41)], 4, 1, 128, 64, seed=31).check(mq)


def test_max_q_may_be_larger_than_any_sequence_needs(mq):
    p = Problem([(90, 1), (200, 3), (5, 2)], 8, 2, 128, 32, seed=32)
    for max_q in (3, 5, 64, 1000):
        p.check(mq, max_q=max_q)


@pytest.mark.parametrize("nq", [1, 3, 90])
@pytest.mark.parametrize("page", [16, 64])
def test_absent_pages_are_as_if_masked(mq, nq, page):
    """A page number outside the cache: its tokens are not seen, and that is reported."""
    p = Problem([(290, nq), (130, nq)], 8, 2, 128, page, seed=33, extra_rows=0)
    gone = (2, 1)  # page 2 of the first sequence, page 1 of the second
    p.tables[0, gone[0]], p.tables[1, gone[1]] = 10 ** 6, -3
    K, V = kv.decode(p.cache, page, 128)
    mq.macaq_device_status(clear=True)
    out, lse = p.run(mq)
    assert mq.macaq_device_status(clear=True) == -9
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref = np.zeros_like(got)
    for b, L in enumerate(p.kv_lens):
        j = np.arange(L)
        j = j[j // page != gone[b]]
        at = p.tables[b][j // page]
        for i in range(nq):
            t = int(p.cu[b]) + i
            s = j <= L - nq + i
            for h in range(8):
                x = K[at[s], h // 4, j[s] % page] @ p.q[t, h].astype(np.float64) * p.scale
                w = np.exp(x - x.max())
                ref[t, h] = (w / w.sum()) @ V[at[s], h // 4, j[s] % page]
                assert abs(gl[t, h] - x.max() - np.log(w.sum())) < 5e-3  # f16 queries: 2^-11 of sums of |q k| < 10
    # a row whose missing keys were counted would be off by a good part of itself
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("nq", [1, 4, 80])
def test_foreign_bytes_change_nothing(mq, nq):
    """Bytes behind a sequence's end, in other pages, and table entries past the end: the same bits with others."""
    p = Problem([(77, nq), (300, nq), (nq, nq)], 8, 1, 128, 32, seed=34)
    want, wl = p.run(mq, window=50)
    used = np.zeros(p.cache.shape[:1] + (32,), bool)
    for b, L in enumerate(p.kv_lens):
        j = np.arange(L)
        used[p.tables[b][j // 32], j % 32] = True
    (kc, ks), (vc, vs) = kv.offsets(32, 128)
    keep = np.zeros(p.cache.shape, bool)
    for pg in range(len(keep)):
        for place in (kc, ks, vc, vs):
            keep[pg][:, place[used[pg]].ravel()] = True
    other = np.random.default_rng(1).integers(0, 256, p.cache.shape).astype(np.uint8)
    other[:, :, 32 * 128:] = 255  # scales of NaN among them
    p.cache = np.where(keep, p.cache, other)
    p.tables = np.where(p.tables < 0, 2 ** 31 - 1, p.tables)
    out, lse = p.run(mq, window=50)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    assert mq.macaq_device_status() == 0


@pytest.mark.parametrize("nq", [1, 4, 60])
def test_non_finite_queries_stay_in_their_rows(mq, nq):
    p = Problem([(200, nq), (90, nq)], 8, 2, 128, 64, seed=35)
    want, _ = p.run(mq)
    p.q = p.q.copy()
    for t, h, x in ((0, 0, np.inf), (0, 3, np.nan), (nq, 5, -np.inf)):
        p.q[t, h, 17] = x
    out, _ = p.run(mq)
    other = torch.ones(out.shape[:2], dtype=torch.bool)
    other[0, 0] = other[0, 3] = other[nq, 5] = False
    assert torch.equal(out[other], want[other])
    assert not torch.isfinite(out[~other]).any()


def test_queries_of_extreme_size(mq):
    """Rows scaled by powers of two far outside f16, with the scale undoing it: the same softmax."""
    p = Problem([(150, 2), (200, 70)], 4, 2, 64, 16, seed=36)
    want, _ = p.run(mq)
    for e in (-60, 60):
        q = Problem([(150, 2), (200, 70)], 4, 2, 64, 16, seed=36)
        q.q = q.q * np.float32(2.0 ** e)
        out, _ = q.run(mq, scale=p.scale * 2.0 ** -e)
        assert torch.equal(out, want)


def test_pages_behind_four_gigabytes(mq):
    """Byte offsets past 32 bits: the same bits as with the pages at the front (append, gather, attention)."""
    Hq, Hk, D, page = 8, 8, 128, 128
    pages = 2 ** 32 // (Hk * kv.page_bytes(page, D)) + 8
    far = torch.empty(pages, Hk, kv.page_bytes(page, D), dtype=torch.uint8, device="cuda")
    near = torch.empty(8, Hk, kv.page_bytes(page, D), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(37)
    x = torch.randn(600, (Hq + 2 * Hk) * D, generator=g).to(torch.bfloat16).cuda()
    at = torch.arange(600, device="cuda")
    outs = []
    for cache, base in ((near, 0), (far, pages - 8)):
        table = torch.tensor([[3, 7, 0, 5, 2]], dtype=torch.int32, device="cuda") + base
        slots = table[0].long()[at // page] * page + at % page
        q = mq.macaq_kv4_append(x, Hq, Hk, D, cache, page, slots)
        lens = torch.tensor([600], dtype=torch.int32, device="cuda")
        res = [*mq.macaq_kv4_gather(cache, D, page, slots)]
        for n in (1, 4, 600):
            cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            res.append(mq.macaq_kv4_attention(q[600 - n:], cache, page, table, lens, cu, max_q=n))
        outs.append(res)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert mq.macaq_device_status() == 0


def test_two_streams_at_once(mq):
    """Calls on two streams, each with a workspace of its own, and on one stream sharing one."""
    ps = [Problem([(900, 1), (333, 1)], 8, 1, 128, 64, seed=38), Problem([(500, 130)], 8, 1, 128, 64, seed=39)]
    args = [(cuda(p.q, torch.bfloat16), cuda(p.cache), 64, cuda(p.tables), cuda(p.kv_lens), cuda(p.cu)) for p in ps]
    want = [mq.macaq_kv4_attention(*a, max_q=p.max_q) for a, p in zip(args, ps)]
    size = max(mq.kv4_attention_workspace_bytes(p.T, len(p.kv_lens), 8, 1, 128, p.max_q) for p in ps)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(mq.macaq_kv4_attention(*args[i], max_q=ps[i].max_q, workspace=ws[i], stream=streams[i]))
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            got[i].append(mq.macaq_kv4_attention(*args[i], max_q=ps[i].max_q, workspace=ws[0]))
    used = [int(p.cu[-1]) for p in ps]  # rows behind are not written
    for i in range(2):
        assert all(torch.equal(o[:used[i]], want[i][:used[i]]) for o in got[i])


def test_captured_prompt_follows_its_inputs(mq):
    """The kernels of many rows captured and replayed with other lengths, tables and queries."""
    p = Problem([(400, 100), (300, 40)], 8, 2, 64, 32, seed=40)
    q, cache, tab, lens = cuda(p.q, torch.bfloat16), cuda(p.cache), cuda(p.tables), cuda(p.kv_lens)
    cu = cuda(p.cu)
    out = torch.full(p.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mq.kv4_attention_workspace_bytes(p.T, 2, 8, 2, 64, p.max_q), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mq.macaq_kv4_attention(q, cache, 32, tab, lens, cu, max_q=p.max_q, out=out, workspace=ws)
    for lens_now, cu_now in (((400, 300), (0, 100, 140)), ((390, 17), (0, 60, 77)), ((12, 0), (0, 0, 3))):
        lens.copy_(cuda(np.array(lens_now, np.int32)))
        cu.copy_(cuda(np.array(cu_now, np.int32)))
        q.mul_(-1)
        out.fill_(7.0)
        graph.replay()
        want = torch.full_like(out, 7.0)
        mq.macaq_kv4_attention(q, cache, 32, tab, lens, cu, max_q=p.max_q, out=want)
        assert torch.equal(out, want)
        assert (out[cu_now[-1]:] == 7).all()
    assert mq.macaq_device_status() == 0


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_kernels_that_follow_one_another_share_their_buffers(mq, nq):
    """append and attention of several batches in turn, nothing else between them, into the same queries and through
    the same workspace: what one call leaves there (queries, parts, notes of cut units) is not taken for another's."""
    rng = np.random.default_rng(41)
    Hq, Hk, D, page, calls = 8, 1, 128, 32, []
    q = torch.empty(2 * nq, Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mq.kv4_attention_workspace_bytes(2 * nq, 2, Hq, Hk, D, nq), dtype=torch.uint8, device="cuda")
    cu = cuda(np.array([0, nq, 2 * nq], np.int32))
    for lens in ((1500, 70), (90, 1400), (1200, 1200), (64, 100), (40, 1990)):
        p = Problem([(n, nq) for n in lens], Hq, Hk, D, page, seed=42 + lens[0], extra_rows=0)
        x = kv.bf16(rng.standard_normal((2 * nq, (Hq + 2 * Hk) * D)))
        at = np.concatenate([np.arange(n - nq, n) for n in lens])
        slots = p.tables[np.repeat([0, 1], nq), at // page].astype(np.int64) * page + at % page
        calls.append((cuda(x, torch.bfloat16), cuda(p.cache), cuda(slots), cuda(p.tables), cuda(p.kv_lens)))

    def call(x, cache, slots, tables, lens, out=None):
        mq.macaq_kv4_append(x, Hq, Hk, D, cache, page, slots, q=q)
        return mq.macaq_kv4_attention(q, cache, page, tables, lens, cu, max_q=nq, out=out, workspace=ws)

    want = []
    for c in calls:
        want.append(call(*c))
        torch.cuda.synchronize()
    order = rng.integers(0, len(calls), 60)
    outs = [torch.empty_like(want[0]) for _ in order]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, out in zip(order, outs):
            call(*calls[i], out=out)
    for out in outs:
        out.zero_()
    graph.replay()
    assert all(torch.equal(out, want[i]) for i, out in zip(order, outs))
    got = [call(*calls[i]) for i in order]
    assert all(torch.equal(out, want[i]) for i, out in zip(order, got))
    assert mq.macaq_device_status() == 0


def test_more_units_than_a_cta_tells_apart(mq):
    """Hundreds of thousands of short sequences in the kernel of many rows, some with values far apart, one to three
    pages for all of them: every row is one of three results."""
    rng = np.random.default_rng(43)
    D, page, B, L = 64, 16, 330_000, 5
    q = kv.bf16(rng.standard_normal(D))
    cache = np.zeros((3, 1, kv.page_bytes(page, D)), np.uint8)
    for pg in range(3):
        k, v = kv.bf16(rng.standard_normal((2, L, 1, D)))
        if pg == 2:
            v[1] *= np.float32(2.0 ** 40)
            k[1] = -8 * q  # of no weight
        kv.store(cache, pg * page + np.arange(L), page, k, kv.bf16(v))
    which = rng.integers(0, 2, B).astype(np.int32)
    which[[5, 3000, 100_001, B - 1]] = 2
    which[B // 2::977] = 2
    K, V = kv.decode(cache, page, D)
    want = np.stack([kv.attend(q[None, None].astype(np.float64), K, V, np.array([[pg]]), [L], [0, 1], D ** -0.5, 0,
                               np.zeros((1, 1, D)))[0][0, 0] for pg in range(3)])
    out = mq.macaq_kv4_attention(cuda(q, torch.bfloat16).expand(B, 1, D).contiguous(), cuda(cache), page, cuda(which[:, None]),
                                 cuda(np.full(B, L, np.int32)), cuda(np.arange(B + 1, dtype=np.int32)), max_q=40)
    ref = cuda(want)[cuda(which).long()]
    err = (out[:, 0].double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert err.max() <= 5e-3
    assert mq.macaq_device_status() == 0
