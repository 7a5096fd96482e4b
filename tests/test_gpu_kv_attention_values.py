"""Attention where the sizes of values or keys lie far apart: what one key, block or sequence holds must not take
another's place.  Tolerances are relative to each row's own weighted values, for each block of 32 elements."""
import numpy as np
import pytest
import torch

from tests import kv_util as kv
from tests.test_gpu_kv_attention import cuda, mq  # noqa: F401  (mq is a fixture)

pytestmark = pytest.mark.gpu

# (D, query heads a kv head, queries a sequence, kv heads, page, keys the tables have room for): 8, 16 and 32 rows of the
# kernel of few rows, tables that are cut and that are not, and the kernel of many rows
KERNELS = [(128, 2, 3, 2, 32, 0), (64, 4, 4, 1, 16, 0), (128, 8, 2, 1, 64, 2000), (64, 8, 4, 1, 32, 2000),
           (128, 8, 4, 1, 64, 1 << 19), (128, 2, 40, 2, 16, 0), (64, 1, 300, 1, 64, 0)]


class Cached:
    """Sequences given as (k [L, Hk, D], v, q [n, Hq, D]) in a cache of shuffled pages."""

    def __init__(self, seqs, page, room=0, seed=0):
        rng = np.random.default_rng(seed)
        self.Hk, self.D = seqs[0][0].shape[1:]
        self.Hq, self.page = seqs[0][2].shape[1], page
        self.kv_lens = np.array([len(s[0]) for s in seqs], np.int32)
        self.cu = np.concatenate(([0], np.cumsum([len(s[2]) for s in seqs]))).astype(np.int32)
        self.max_q = max(len(s[2]) for s in seqs)
        used = max(-(-int(n) // page) for n in self.kv_lens)
        width = max(used, -(-room // page))
        order = rng.permutation(len(seqs) * used).reshape(len(seqs), used)
        self.tables = np.concatenate((order, np.full((len(seqs), width - used), -7)), 1).astype(np.int32)
        self.cache = np.zeros((len(seqs) * used, self.Hk, kv.page_bytes(page, self.D)), np.uint8)
        with np.errstate(invalid="ignore"):  # infinities
            for b, (k, v, _) in enumerate(seqs):
                j = np.arange(len(k))
                kv.store(self.cache, order[b][j // page] * page + j % page, page, k, v)
        self.q = np.concatenate([s[2] for s in seqs])
        self.scale = self.D ** -0.5

    def run(self, mq):
        """out, fp64 on the host, and the logarithms of the sums."""
        lse = torch.empty(self.q.shape[:2], dtype=torch.float32, device="cuda")
        out = mq.macaq_kv4_attention(cuda(self.q, torch.bfloat16), cuda(self.cache), self.page, cuda(self.tables),
                                     cuda(self.kv_lens), cuda(self.cu), max_q=self.max_q, lse=lse)
        assert mq.macaq_device_status() == 0
        return out, lse

    def check(self, mq, rows=None, block_gain=None):
        """Every element of the rows in `rows` (query index -> bool) against 64 bits.

        A row's weights are off by factors 1 + eps_j: the transformed query is rounded to f16, which moves a score
        by 2^-11 scale sum |q'_i k'_i|; fp32 rounds it by 2^-24 of itself a few times (2^-21 (1 + |s|)); the weight
        is rounded to f16, 2^-11, and scaled in it.  With A_j = sum_i |v'_ji| / sqrt(32), what an element can take
        from a unit of weight j, that moves an element by sum p_j eps_j A_j and, through the denominator, by
        sum p_j eps_j sum p_j A_j.  Weights below f16's normal range are off by half of its smallest step instead, 2^-25,
        where the largest weight is 2^6 or more: 2^-31 of it, in the kernel of few rows times scales that are at most 2^14
        above the smallest in the same part, in the other times values at most 2^20 above it.  Sums are fp32, (n + 64)
        roundings of 2^-24, and the result is rounded to bf16."""
        got, lse = self.run(mq)
        got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
        K, V = kv.decode(self.cache, self.page, self.D)
        G, nb = self.Hq // self.Hk, self.D // 32
        for b, L in enumerate(self.kv_lens):
            j = np.arange(L)
            at = self.tables[b][j // self.page]
            n = int(self.cu[b + 1] - self.cu[b])
            for i in range(n):
                if rows is not None and not rows(i, n):
                    continue
                t, see = int(self.cu[b]) + i, j <= L - n + i
                for h in range(self.Hq):
                    k, v = K[at[see], h // G, j[see] % self.page], V[at[see], h // G, j[see] % self.page]
                    q = self.q[t, h].astype(np.float64)
                    qt, kt, vt = (np.abs(kv.hadamard(x.reshape(-1, nb, 32)) / np.sqrt(32.0)) for x in (q, k, v))
                    s = k @ q * self.scale
                    p = np.exp(s - s.max())
                    top, p = p.max() / p.sum(), p / p.sum()
                    ref = p @ v
                    eps = 2.0 ** -11 * self.scale * (qt * kt).sum((1, 2)) + 2.0 ** -21 * (1 + np.abs(s)) + 2.0 ** -10
                    A = vt.sum(-1) / np.sqrt(32.0)
                    big = vt.max(-1)
                    least = big[big > 0].min() if (big > 0).any() else 0.0
                    weighted = p @ A
                    tol = (p * eps) @ A + (p @ eps) * weighted + (len(p) + 64) * 2.0 ** -24 * weighted
                    tol += 2.0 ** -31 * top * np.minimum(A, 2.0 ** 20 * least).sum(0)
                    tol += len(p) * 2.0 ** -17 * 8.5 * top * least
                    err = np.abs(got[t, h] - ref).reshape(nb, 32)
                    bad = err > 2.0 ** -8 * np.abs(ref).reshape(nb, 32) + tol[:, None]
                    assert not bad.any(), (b, i, h, err.max(-1), tol, np.abs(ref).reshape(nb, 32).max(-1))
                    lref = s.max() + np.log(np.exp(s - s.max()).sum())
                    assert abs(lse[t, h] - lref) <= p @ eps + 2.0 ** -16 * (1 + abs(lref))


def sequence(rng, L, n, Hq, Hk, D, score=None):
    """Random k, v and queries.  score: a key's score by its index, for queries that are all one direction."""
    k, v = rng.standard_normal((2, L, Hk, D))
    q = rng.standard_normal((n, Hq, D))
    if score is not None:
        u = rng.standard_normal(D)
        q = u + 0.05 * q
        for j, s in score.items():
            k[j] = s * D ** 0.5 * u / (u @ u)
    return kv.bf16(k), kv.bf16(v), kv.bf16(q)


def earlier(i, n):
    return i < n - 1


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** 11, 2.0 ** 16, 2.0 ** 30, 2.0 ** 70, np.inf, np.nan])
def test_a_huge_value_that_earlier_queries_do_not_see(mq, D, G, nq, Hk, page, room, gain):
    rng = np.random.default_rng(50)
    seqs = [sequence(rng, L, min(nq, L), G * Hk, Hk, D) for L in (nq + 13, nq + 150)]
    for k, v, q in seqs:
        v[-1, :, 3] *= np.float32(gain)
        v[-1, :, 40] *= np.float32(gain)
    Cached(seqs, page, room).check(mq, None if np.isfinite(gain) else earlier)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** 13, 2.0 ** 30, 2.0 ** 56])
def test_a_huge_value_of_little_weight(mq, D, G, nq, Hk, page, room, gain):
    """A score 40 below the others': nothing of its value at 2^13 and 2^30 times theirs, as much as theirs at 2^56."""
    rng = np.random.default_rng(51)
    L = nq + 140
    k, v, q = sequence(rng, L, nq, G * Hk, Hk, D, {3: -20.0, **{j: 20.0 for j in range(4, 12)}})
    v[3] *= np.float32(gain)
    Cached([(k, v, q)], page, room).check(mq)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("step", [13, 30])
def test_blocks_of_a_head_far_apart(mq, D, G, nq, Hk, page, room, step):
    rng = np.random.default_rng(52)
    k, v, q = sequence(rng, nq + 90, nq, G * Hk, Hk, D)
    v *= np.repeat(np.float32(2.0) ** (-step * np.arange(D // 32)), 32)
    Cached([(k, v, q), sequence(rng, nq, nq, G * Hk, Hk, D)], page, room).check(mq)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
def test_values_that_grow_and_shrink_by_far(mq, D, G, nq, Hk, page, room):
    """From 2^-30 to 2^30 along the keys and back, with the weight on either side, and some values of zero."""
    rng = np.random.default_rng(53)
    L = nq + 200
    for s in (1, -1):
        k, v, q = sequence(rng, L, nq, G * Hk, Hk, D, {j: (-10.0 if j < L // 2 else 10.0) for j in range(0, L, 3)})
        v *= (np.float32(2.0) ** np.linspace(-30 * s, 30 * s, L))[:, None, None]
        v[5] = v[L - 2] = 0
        Cached([(k, kv.bf16(v), q)], page, room).check(mq)


@pytest.mark.parametrize("nq,Hk", [(1, 2), (3, 2), (40, 2), (1, 40)])
@pytest.mark.parametrize("gain", [2.0 ** 30, np.inf, np.nan])
def test_other_sequences_keep_their_bits(mq, nq, Hk, gain):
    """One sequence of a batch with huge or infinite values, others behind it on the same CTAs."""
    rng = np.random.default_rng(54)
    seqs = [sequence(rng, nq + 20, nq, 2 * Hk, Hk, 64) for _ in range(170 if Hk == 2 else 60)]
    want, wl = Cached(seqs, 16).run(mq)
    bad = range(0, len(seqs), 17)
    for b in bad:
        seqs[b][1][7, :, 9] *= np.float32(gain)
        seqs[b][0][4, 0, 5] *= np.float32(gain)
    out, lse = Cached(seqs, 16).run(mq)
    same = torch.ones(len(out), dtype=torch.bool)
    for b in bad:
        same[b * nq:(b + 1) * nq] = False
    assert torch.equal(out[same], want[same]) and torch.equal(lse[same], wl[same])


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** 20, 2.0 ** 40, np.inf, np.nan])
def test_a_huge_key_that_earlier_queries_do_not_see(mq, D, G, nq, Hk, page, room, gain):
    rng = np.random.default_rng(55)
    k, v, q = sequence(rng, nq + 33, nq, G * Hk, Hk, D)
    k *= 2.0
    k[-1, :, 7] *= np.float32(gain)
    Cached([(k, v, q)], page, room).check(mq, earlier)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
def test_a_huge_key_of_no_weight(mq, D, G, nq, Hk, page, room):
    """A key of 2^30 times the others' size against the queries' direction: its neighbours' scores count all the same."""
    rng = np.random.default_rng(56)
    L = nq + 60
    k, v, q = sequence(rng, L, nq, G * Hk, Hk, D, {j: 3.0 * np.sin(j) for j in range(L)})
    k[17] = -np.abs(k[17]).max() * 2.0 ** 30 * np.sign(q[0, 0])
    Cached([(kv.bf16(k), v, q)], page, room).check(mq)


@pytest.mark.parametrize("nq", [1, 50])
def test_keys_that_grow_along_the_sequence(mq, nq):
    """Keys of 2^-40 to 2^4 among neighbours of the same 32 tokens."""
    rng = np.random.default_rng(57)
    k, v, q = sequence(rng, nq + 150, nq, 4, 2, 128)
    k *= np.where(np.arange(len(k)) % 5 == 0, 2.0 ** -40, np.where(np.arange(len(k)) % 7 == 0, 2.0 ** 4, 1.0))[:, None, None]
    Cached([(kv.bf16(k), v, q)], 32).check(mq)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("below", [16, 26])
def test_small_weights_that_are_all_that_counts(mq, D, G, nq, Hk, page, room, below):
    """One key has nearly all the weight and a value of zero; the others, at 2^-16 and 2^-26 of it, make the result.

    A weight is held times 2^10 or more, and in the kernel of few rows times a scale of 2^-3 or more (values that differ
    by little, an exponent above theirs): 2^-19, off by 2^-25 at most, 2^-6 of itself.  The large score, 18 in natural units,
    is off by 2^-11 of the sum of its terms, which are of one sign: 2^-6.8.  All values point one way."""
    rng = np.random.default_rng(58)
    L = nq + 250
    k, v, q = sequence(rng, L, nq, G * Hk, Hk, D, {2: below * np.log(2.0)})
    k[np.arange(L) != 2] *= np.float32(1 / 64)
    v = kv.bf16(rng.standard_normal(D) * (1 + 0.1 * v))
    v[2] = 0
    c = Cached([(kv.bf16(k), v, q)], page, room)
    got, _ = c.run(mq)
    K, V = kv.decode(c.cache, page, D)
    ref, _, _ = kv.attend(c.q.astype(np.float64), K, V, c.tables, c.kv_lens, c.cu, c.scale, 0, np.zeros(c.q.shape))
    err = np.linalg.norm(got.double().cpu().numpy() - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert (err <= 2.0 ** -6 + 2.0 ** -6.8 + 2.0 ** -8).all(), err.max()


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** 22, 2.0 ** 27, 2.0 ** 40, 2.0 ** 70])
def test_scores_beyond_the_steps_of_fp32(mq, D, G, nq, Hk, page, room, gain):
    """The newest key's score is some 2^22 to 2^70, of one sign for even heads and of the other for odd ones: it has all the
    weight, or none.  The newest query's result is that key's value, within its rounding and that of the sums, or what the
    other keys make, as in any other test."""
    rng = np.random.default_rng(59)
    L = nq + 60
    k, v, q = sequence(rng, L, nq, G * Hk, Hk, D)
    u = kv.bf16(rng.standard_normal(D))
    q[-1] = u * np.where(np.arange(G * Hk) % 2, -1, 1)[:, None]
    k[-1] = kv.bf16(u * np.float32(gain))
    c = Cached([(k, v, q)], page, room)
    c.check(mq, earlier)
    got = c.run(mq)[0].double().cpu().numpy()[-1]
    assert np.isfinite(got).all()
    K, V = kv.decode(c.cache, page, D)
    j = np.arange(L)
    vs = V[c.tables[0][j // page], :, j % page]
    for h in range(0, G * Hk, 2):
        ref = vs[-1, h // G]
        size = np.abs(ref).reshape(-1, 32).sum(-1).repeat(32)
        assert (np.abs(got[h] - ref) <= 2.0 ** -8 * np.abs(ref) + (L + 64) * 2.0 ** -24 * size + 2.0 ** -10 * size / 32).all()
    ks = K[c.tables[0][j // page], :, j % page]
    for h in range(1, G * Hk, 2):
        s = ks[:-1, h // G] @ c.q[-1, h].astype(np.float64) * c.scale
        p = np.exp(s - s.max())
        ref = p / p.sum() @ vs[:-1, h // G]
        assert np.linalg.norm(got[h] - ref) <= 0.01 * np.linalg.norm(ref)


@pytest.mark.parametrize("D,G,nq,Hk,page,room", KERNELS)
@pytest.mark.parametrize("gain", [2.0 ** 27, 2.0 ** 50])
def test_ordinary_scores_behind_huge_negative_ones(mq, D, G, nq, Hk, page, room, gain):
    """What a row has summed relative to a reference of -2^27 and below is gone without a trace when its first ordinary
    score comes; rows that see the huge ones alone have those."""
    rng = np.random.default_rng(62)
    L = nq + 200
    k, v, q = sequence(rng, L, nq, G * Hk, Hk, D, {j: 2.0 * np.sin(j) for j in range(150, L)})
    k[:150] = -np.sign(q[0, 0]) * np.abs(k[:150]) * np.float32(gain)
    c = Cached([(kv.bf16(k), v, q)], page, room)
    c.check(mq)
