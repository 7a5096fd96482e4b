"""Attention over the paged MXFP4 cache on the GPU against numpy in 64 bits."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import online_hadamard_b200 as m
    m.load_library()
    m.macaq_device_status(clear=True)
    return m


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


class Problem:
    """A cache with random pages, sequences of the given (keys, queries), garbage in every other byte."""

    def __init__(self, seqs, Hq, Hk, D, page, seed=0, q_gain=1.0, v_gain=None, extra_rows=3):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hk, self.D, self.page = Hq, Hk, D, page
        self.kv_lens = np.array([s[0] for s in seqs], np.int32)
        n = [s[1] for s in seqs]
        self.cu = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        self.max_q = max(max(n), 1)
        width = max(1, max((s[0] + page - 1) // page for s in seqs))
        total = len(seqs) * width + 1
        order = rng.permutation(total)[:len(seqs) * width].reshape(len(seqs), width)
        self.tables = order.astype(np.int32)
        for b, s in enumerate(seqs):  # entries past a sequence's pages point nowhere and are never read
            self.tables[b, (s[0] + page - 1) // page:] = -7
        cache = rng.integers(0, 256, (total, Hk, kv.page_bytes(page, D))).astype(np.uint8)
        for b, s in enumerate(seqs):
            if s[0] == 0:
                continue
            j = np.arange(s[0])
            slots = order[b][j // page] * page + j % page
            k = rng.standard_normal((s[0], Hk, D)) * np.where(rng.random(D) < 0.03, 6.0, 1.0)
            v = rng.standard_normal((s[0], Hk, D))
            if v_gain is not None:
                v *= v_gain(s[0])[:, None, None]
            kv.store(cache, slots, page, kv.bf16(k), kv.bf16(v))
        self.cache = cache
        self.T = int(self.cu[-1]) + extra_rows
        self.q = kv.bf16(rng.standard_normal((self.T, Hq, D)) * q_gain)
        self.scale = D ** -0.5

    def reference(self, window=0, fill=7.0):
        K, V = kv.decode(self.cache, self.page, self.D)
        return kv.attend(self.q.astype(np.float64), K, V, self.tables, self.kv_lens, self.cu, self.scale, window,
                         np.full(self.q.shape, fill))

    def run(self, mq, window=0, fill=7.0, cu=True, **kw):
        out = torch.full(self.q.shape, fill, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 5.0, dtype=torch.float32, device="cuda")
        kw.setdefault("max_q", self.max_q)
        mq.macaq_kv4_attention(cuda(self.q, torch.bfloat16), cuda(self.cache), self.page, cuda(self.tables),
                               cuda(self.kv_lens), cuda(self.cu) if cu else None, window=window, out=out, lse=lse, **kw)
        return out, lse

    def check(self, mq, window=0, **kw):
        out, lse = self.run(mq, window, **kw)
        ref, rl, spread = self.reference(window)
        used = int(self.cu[-1])
        got = out.double().cpu().numpy()
        assert (got[used:] == 7).all() and (lse.cpu().numpy()[used:] == 5).all(), "rows behind the last sequence"
        # The transformed query is rounded to fp16, 2^-11 of an element in the worst case: a score moves by at most
        # 2^-11 scale sum |q'_i k'_i|, here bounded by 2^-11 * scale * |q| |k| (Cauchy-Schwarz).  A softmax weight is
        # rounded to fp16, 2^-11 of itself.  An output moves by at most `spread` per unit of score, and by 2^-11 of
        # the largest |v| for the weights; then half a bf16 step, and 2^-16 of the largest |v| for the fp32 sums.
        K, _ = kv.decode(self.cache, self.page, self.D)
        kmax = max(self._kmax(K, b, int(L)) for b, L in enumerate(self.kv_lens))
        score = 2.0 ** -11 * self.scale * np.linalg.norm(self.q, axis=-1) * kmax
        tol = spread * (score + 2.0 ** -11 + 2.0 ** -16)
        err = np.abs(got[:used] - ref[:used])
        bad = err > 2.0 ** -8 * np.abs(ref[:used]) + tol[:used, :, None]
        assert not bad.any(), f"{bad.sum()} wrong, worst {err.max()} at {np.argwhere(bad)[0]}"
        # and as a whole, where errors are random: the norms of the two differ by a rounding or two
        den = np.linalg.norm(ref[:used])
        assert den == 0 or np.linalg.norm(got[:used] - ref[:used]) <= 5e-3 * den
        gl = lse.double().cpu().numpy()[:used]
        empty = np.isneginf(rl[:used])
        assert np.array_equal(np.isneginf(gl), empty)
        assert (np.abs(gl - rl[:used])[~empty] <= (score[:used] + 2.0 ** -16 * (1 + np.abs(rl[:used])))[~empty]).all()
        assert not got[:used][empty].any()
        assert mq.macaq_device_status() == 0

    def _kmax(self, K, b, L):
        j = np.arange(L)
        return np.linalg.norm(K[self.tables[b][j // self.page], :, j % self.page], axis=-1).max() if L else 0.0


@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("G,Hk", [(1, 3), (4, 2), (8, 1)])
def test_single_tokens(mq, D, page, G, Hk):
    """One query a sequence; lengths at the edges of tiles and pages, none among them."""
    seqs = [(L, 1) for L in (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 300)]
    Problem(seqs, G * Hk, Hk, D, page, seed=D + page + G).check(mq)


def test_single_tokens_without_query_ranges(mq):
    p = Problem([(L, 1) for L in (5, 130, 77)], 8, 2, 128, 32, seed=3, extra_rows=0)
    p.check(mq, cu=False)


@pytest.mark.parametrize("Hq,Hk,D", [(5, 1, 64), (7, 1, 128), (12, 1, 128), (16, 1, 64), (32, 1, 128), (33, 3, 64),
                                     (71, 1, 128), (9, 9, 64)])
def test_group_sizes(mq, Hq, Hk, D):
    Problem([(200, 1), (3, 1), (129, 1)], Hq, Hk, D, 64, seed=Hq).check(mq)


@pytest.mark.parametrize("window", [0, 1, 7, 64, 100, 1000])
@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 64), (6, 3, 64, 16)])
def test_several_tokens_and_windows(mq, window, Hq, Hk, D, page):
    """A few queries a sequence: more than keys in one (the first see nothing), none in another."""
    seqs = [(300, 4), (2, 5), (5, 5), (65, 3), (0, 2), (128, 0), (257, 5), (1, 1)]
    Problem(seqs, Hq, Hk, D, page, seed=window).check(mq, window)


@pytest.mark.parametrize("Hq,Hk,D,page,window", [(4, 2, 128, 128, 0), (8, 1, 128, 16, 0), (3, 3, 64, 64, 0),
                                                 (8, 2, 64, 16, 40), (16, 2, 128, 32, 200), (7, 1, 128, 64, 0)])
def test_prompts(mq, Hq, Hk, D, page, window):
    """Prompts and chunks of prompts: whole, behind a prefix, odd lengths, beside single tokens."""
    seqs = [(130, 130), (300, 77), (1, 1), (400, 1), (257, 129), (40, 64), (0, 3), (64, 64)]
    Problem(seqs, Hq, Hk, D, page, seed=Hq + page).check(mq, window)


def test_long_prompt_rows(mq):
    """A prompt over several tiles of queries and keys, behind a prefix."""
    Problem([(900, 515)], 4, 2, 128, 64, seed=9).check(mq)


def test_long_single_tokens(mq):
    """Contexts split over many blocks and joined again."""
    Problem([(5000, 1), (77, 1), (3001, 1)], 8, 1, 128, 64, seed=10).check(mq)


def test_large_scores(mq):
    """Scores of some tens: the softmax is nearly one key's, the running maximum moves often."""
    Problem([(500, 1), (500, 3), (200, 200)], 8, 2, 128, 64, seed=11, q_gain=8.0).check(mq)


def test_values_of_very_different_size(mq):
    """Values whose scales lie far apart: ascending, descending, and one huge token among small ones."""
    up = lambda n: 2.0 ** np.linspace(-12, 12, n)
    for gain in (up, lambda n: up(n)[::-1], lambda n: np.where(np.arange(n) == n // 2, 2.0 ** 10, 2.0 ** -6)):
        Problem([(300, 1), (200, 70)], 8, 2, 128, 64, seed=12, v_gain=gain).check(mq)


def test_strided_queries_other_stream_and_same_bits(mq):
    """Rows of q inside a wider tensor, on a stream of its own; two runs give the same bits."""
    p = Problem([(700, 1), (90, 1), (1500, 1)], 8, 2, 128, 32, seed=13, extra_rows=0)
    wide = torch.full((3, 1024 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :1024] = cuda(p.q, torch.bfloat16).reshape(3, 1024)
    args = (cuda(p.cache), 32, cuda(p.tables), cuda(p.kv_lens))
    want = mq.macaq_kv4_attention(cuda(p.q, torch.bfloat16), *args)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mq.macaq_kv4_attention(wide[:, :1024].unflatten(1, (8, 128)), *args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    p.check(mq)


def test_bad_tables_lengths_and_ranges_are_cut_and_reported(mq):
    """Pages outside the cache are as if absent, lengths end with the table, rows past max_q are not written."""
    p = Problem([(100, 1), (100, 3)], 4, 2, 64, 16, seed=14)
    want, _ = p.run(mq)
    mq.macaq_device_status(clear=True)
    q = Problem([(100, 1), (100, 3)], 4, 2, 64, 16, seed=14)
    q.tables[0, 2] = 10 ** 6
    out, _ = q.run(mq)
    assert mq.macaq_device_status(clear=True) == -9
    assert torch.equal(out[1:], want[1:]) and torch.isfinite(out).all()
    q = Problem([(100, 1), (100, 3)], 4, 2, 64, 16, seed=14)
    q.kv_lens[0] = 10 ** 6
    q.tables[0] = np.abs(q.tables[0])
    out, _ = q.run(mq)
    assert mq.macaq_device_status(clear=True) == -9
    assert torch.equal(out[1:], want[1:])
    out, _ = p.run(mq, max_q=2)
    assert mq.macaq_device_status(clear=True) == -9
    assert (out[3] == 7).all() and torch.equal(out[:3], want[:3])
    p.cu[2] = 50  # past the rows of q
    out, _ = p.run(mq)
    assert mq.macaq_device_status(clear=True) == -9


def test_captured_steps_replay(mq):
    """append and attention captured together: replays follow the tensors' new contents, and two graphs
    with one workspace each on one stream do not disturb each other."""
    rng = np.random.default_rng(15)
    Hq, Hk, D, page, B = 8, 2, 128, 32, 3
    lens = np.array([40, 7, 333], np.int32)
    width = 12
    tables = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    cache0 = rng.integers(0, 256, (B * width, Hk, kv.page_bytes(page, D))).astype(np.uint8)
    for b in range(B):
        j = np.arange(lens[b])
        kv.store(cache0, tables[b][j // page] * page + j % page, page, kv.bf16(rng.standard_normal((lens[b], Hk, D))),
                 kv.bf16(rng.standard_normal((lens[b], Hk, D))))
    cache, tab = cuda(cache0), cuda(tables)
    kvl, slots = cuda(lens), cuda(np.zeros(B, np.int64))
    x = cuda(kv.bf16(rng.standard_normal((B, (Hq + 2 * Hk) * D))), torch.bfloat16)
    ws = torch.empty(mq.kv4_attention_workspace_bytes(B, B, Hq, Hk, D, 1), dtype=torch.uint8, device="cuda")
    graphs, outs, queries = [], [], []
    for _ in range(2):
        q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        step = lambda: (mq.macaq_kv4_append(x, Hq, Hk, D, cache, page, slots, q=q),
                        mq.macaq_kv4_attention(q, cache, page, tab, kvl, out=out, workspace=ws))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
        outs.append(out)
        queries.append(q)  # a graph's tensors live as long as the graph
    ref_cache = cache0
    for it in range(3):
        at = lens + it
        new = kv.bf16(rng.standard_normal((B, (Hq + 2 * Hk) * D)))
        sl = tables[np.arange(B), at // page].astype(np.int64) * page + at % page
        x.copy_(cuda(new, torch.bfloat16))
        slots.copy_(cuda(sl))
        kvl.copy_(cuda((at + 1).astype(np.int32)))
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        h = new.reshape(B, Hq + 2 * Hk, D)
        kv.store(ref_cache, sl, page, h[:, Hq:Hq + Hk], h[:, Hq + Hk:])
        torch.cuda.synchronize()
        assert np.array_equal(cache.cpu().numpy(), ref_cache)
        K, V = kv.decode(ref_cache, page, D)
        ref, _, _ = kv.attend(h[:, :Hq].astype(np.float64), K, V, tables, at + 1, np.arange(B + 1), D ** -0.5, 0,
                              np.zeros((B, Hq, D)))
        assert torch.equal(outs[0], outs[1])
        got = outs[0].double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
    assert mq.macaq_device_status() == 0


def test_layer_from_projection_to_projection(mq):
    """The calls as a decoder layer uses them: stacked q/k/v linear, norms + rotation + append, attention, o
    linear; a prompt of 37 tokens, then two steps.  Against 64-bit attention over what the cache holds."""
    rng = np.random.default_rng(16)
    Hq, Hk, D, page, hidden = 4, 2, 128, 16, 512
    Ns = (Hq * D, Hk * D, Hk * D)
    g = torch.Generator().manual_seed(4)
    s = torch.ones(hidden).cuda()
    folds = [mq.macaq_fold_weights((torch.randn(n, hidden, generator=g) * 0.05).cuda(), s) for n in Ns]
    am = torch.stack([f[2] for f in folds])
    Wq, Ws = torch.cat([f[0] for f in folds]), torch.cat([f[1] for f in folds])
    Wo = mq.macaq_fold_weights((torch.randn(hidden, Hq * D, generator=g) * 0.05).cuda(), torch.ones(Hq * D).cuda())
    wq, wk = (torch.rand(2, D, generator=g) + 0.5).cuda()
    ang = np.arange(64)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    rope = cuda(np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32))
    cache = torch.zeros(6, Hk, mq.kv4_page_bytes(page, D), dtype=torch.uint8, device="cuda")
    table = cuda(np.array([[4, 1, 5, 0]], np.int32))
    done = 0
    for n in (37, 1, 1):
        x = torch.randn(n, hidden, generator=g).to(torch.bfloat16).cuda()
        qkv = mq.macaq_w4a4_linear_multi(x, am, Wq, Ws, Ns)
        at = torch.arange(done, done + n, device="cuda")
        slots = table[0].long()[at // page] * page + at % page
        q = mq.macaq_kv4_append(qkv, Hq, Hk, D, cache, page, slots, rope, at, q_weight=wq, k_weight=wk)
        done += n
        lens = torch.tensor([done], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        o = mq.macaq_kv4_attention(q, cache, page, table, lens, cu, max_q=n)
        y = mq.macaq_w4a4_linear(o.flatten(1), Wo[2], Wo[0], Wo[1], hidden)
        q2, k2 = mq.macaq_qk_norm_rope(qkv, Hq, Hk, D, rope, at, q_weight=wq, k_weight=wk)
        assert torch.equal(q2, q)
        K, V = kv.decode(cache.cpu().numpy(), page, D)
        ref, _, _ = kv.attend(q.double().cpu().numpy(), K, V, table.cpu().numpy(), [done], [0, n], D ** -0.5, 0,
                              np.zeros((n, Hq, D)))
        got = o.double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
        gk, _ = mq.macaq_kv4_gather(cache, D, page, slots)  # MXFP4 of the keys: its rounding is some 10 %
        assert (gk.float() - k2.float()).norm() <= 0.2 * k2.float().norm()
        assert torch.isfinite(y).all() and y.shape == (n, hidden)
    assert mq.macaq_device_status() == 0
