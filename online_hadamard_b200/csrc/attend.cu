// attend.cu -- attention over the paged MXFP4 cache (layout and masks: include/macaq.h).
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the keys a row's mask leaves (none: o_h = 0)
//
// K and V are held as codes of FWHT32(x c0), c0 = 1/sqrt(32).  The transform is orthogonal, so the
// scores are taken between the transformed query and the codes' values, and the weighted sum of V
// codes is transformed back once per output row: no key or value is ever transformed back.
//
// The query heads of one kv head and the queries of one sequence form the rows r = i G + g (query i,
// head g of the group of G) of one product with that head's keys, so the cache is read and decoded
// once for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "sm100.cuh"

namespace macaq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendParams {
    const uint16_t* q;  // bf16 [T][ldq]
    int64_t T, ldq;
    int Hq, Hk, G;
    const uint8_t* cache;
    int64_t num_pages;
    int page_size, page_shift;
    const int32_t* tables;  // [B][table_width]
    int64_t table_width;
    const int32_t* kv_lens;  // [B]
    const int32_t* cu_q;     // [B + 1], or null: row b is sequence b's only query
    int B;
    int max_q;
    float scale_log2;  // scale * log2(e)
    int window;        // 0: none
    uint16_t* out;     // bf16 [T][Hq][D]
    float* lse;        // fp32 [T][Hq] or null
    // the split of the work (plan_attend): row tiles of tile_rows rows; `ctas` > 0: all blocks of keys of
    // all units in one row, cut into that many equal lengths (Cut); 0: one CTA per unit
    int tile_rows, row_tiles, ctas;
    float* part_o;    // fp32 [ctas][2][tile_rows][D], each row divided by its own sum
    float2* part_ml;  // [ctas][2][tile_rows]: its reference m (base 2) and sum of 2^(s - m)
};

// Sequence b: its first query row, its queries, its keys and its first query's position (negative
// where there are fewer keys than queries), kept inside the buffers (what had to be cut is reported).
struct Sequence {
    int64_t row0;
    int nq, kv, pos0;
};
__device__ __forceinline__ Sequence sequence_of(const AttendParams& p, int b) {
    int64_t lo = p.cu_q ? p.cu_q[b] : b, hi = p.cu_q ? p.cu_q[b + 1] : b + 1;
    bool cut = lo < 0 || hi > p.T || hi < lo;
    lo = lo < 0 ? 0 : lo > p.T ? p.T : lo;
    hi = hi > p.T ? p.T : hi;
    int64_t n = hi > lo ? hi - lo : 0;
    const int64_t all = n;
    if (n > p.max_q) n = p.max_q, cut = true;
    int64_t kv = p.kv_lens[b];
    const int64_t most = p.table_width * p.page_size;
    if (kv < 0 || kv > most) kv = kv < 0 ? 0 : most, cut = true;
    if (cut) report_index();
    return {lo, static_cast<int>(n), static_cast<int>(kv), static_cast<int>(kv - all)};
}

// The keys that the rows [r0, r0 + rows) of a sequence may see: first_lo .. last_hi in all, and
// last_lo .. first_hi by every row.
struct Span {
    int first_lo, last_lo, first_hi, last_hi;
};
__device__ __forceinline__ int first_key(const AttendParams& p, int pos) {
    return p.window && pos >= p.window ? pos - p.window + 1 : 0;
}
__device__ __forceinline__ Span span_of(const AttendParams& p, const Sequence& s, int r0, int rows) {
    const int a = s.pos0 + r0 / p.G, z = s.pos0 + (r0 + rows - 1) / p.G;
    return {first_key(p, a), first_key(p, z), a, z};
}

// A unit is a (sequence, kv head, tile of query rows); its work is its span in blocks of 2^shift keys.
__device__ __forceinline__ int blocks_of(const Span& sp, int shift) {
    return sp.last_hi < 0 ? 0 : (sp.last_hi >> shift) - (sp.first_lo >> shift) + 1;
}
// Blocks of all row tiles of one kv head of a sequence.
__device__ __forceinline__ int64_t sequence_blocks(const AttendParams& p, const Sequence& s, int shift) {
    int64_t n = 0;
    const int rows = s.nq * p.G;
    for (int r0 = 0; r0 < rows; r0 += p.tile_rows) n += blocks_of(span_of(p, s, r0, min(p.tile_rows, rows - r0)), shift);
    return n;
}

// Sequences are of unequal length, known on the device only, and few units leave most of the GPU idle: so
// the blocks of all units stand in one row (sequence, then kv head, then row tile), and CTA i of the
// resident ones takes [i len, (i + 1) len) of it, whatever units those belong to.  A unit that one CTA holds
// whole is written directly, parts of one are joined by attend_join_kernel.  A CTA cuts at most two units:
// its parts go to slot 0 (the unit that its range begins in) and slot 1 (the one it ends in).  No CTA gets
// less than kMinKeys keys (joining would cost more than it saves).
constexpr int kMinKeys = 128;
__device__ __forceinline__ int64_t cut_length(const AttendParams& p, int64_t total, int shift) {
    const int64_t len = (total + p.ctas - 1) / p.ctas;
    return len > (kMinKeys >> shift) ? len : (kMinKeys >> shift);
}

struct Cut {
    int64_t pos, end;  // this CTA's range
    int b;             // the sequence that pos lies in, and where that sequence begins
    int64_t seq_pos;
};
// By all 128 threads of a CTA: thread i adds up its share of the sequences, the one whose share holds the
// CTA's first block walks it.
__device__ __forceinline__ Cut cut_of(const AttendParams& p, int shift, int64_t* scan, int* first_seq, int64_t* first_pos) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = (p.B + 127) / 128, b0 = min(p.B, static_cast<int>(threadIdx.x) * share), b1 = min(p.B, b0 + share);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += sequence_blocks(p, sequence_of(p, b), shift) * p.Hk;
    int64_t upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, x);
        if (lane >= x) upto += y;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) upto += scan[w];
        total += scan[w];
    }
    const int64_t len = cut_length(p, total, shift);
    Cut c;
    c.pos = static_cast<int64_t>(blockIdx.x) * len;
    c.end = c.pos + len < total ? c.pos + len : total;
    if (c.pos < upto && c.pos >= upto - mine) {
        int64_t at = upto - mine;
        for (int b = b0; b < b1; ++b) {
            const int64_t n = sequence_blocks(p, sequence_of(p, b), shift) * p.Hk;
            if (c.pos < at + n) {
                *first_seq = b, *first_pos = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    c.b = *first_seq, c.seq_pos = *first_pos;
    return c;
}

// Query rows are brought to f16 by a power of two of their own: |q| < 2^(E - 126) for the row's largest
// exponent E, so |FWHT32(q) c0| 2^(138 - E) < sqrt(32) 2^12 fits, and elements keep their 11 bits down to
// 2^-26 of the largest.  (bf16 would hold the range without that, but rounds the transformed query at
// 2^-9, as much as the query itself; f16 at 2^-12.)
__device__ __forceinline__ uint32_t query_exponent(uint32_t abs_bits) { return max(abs_bits >> 23, 27u); }
__device__ __forceinline__ float query_multiplier(uint32_t E) { return __uint_as_float((265u - E) << 23); }
// ... and what turns a product with the scaled query into a score in base 2.
__device__ __forceinline__ float score_factor(float scale_log2, uint32_t E) {
    return fmaxf(scale_log2 * __uint_as_float((E - 11u) << 23), 1.17549435e-38f);
}

// FWHT of 32 values held by a warp, lane l element l.
__device__ __forceinline__ float warp_fwht32(float x, int l) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
        x = l & o ? y - x : x + y;
    }
    return x;
}

// Softmax weights are kept in f16 for the second product, relative to a reference within 2^8 of the
// running maximum (it moves only when a score passes it by that much, which is rare, so the sums are
// seldom rescaled) and times 2^6: at most 2^14, with 11 bits down to 2^-20 of the largest.
constexpr float kSlack = 8.0f;
constexpr float kLift = 6.0f;

// --------------------------------------------------------------------------- few query rows
//
// CTAs of 4 warps.  A warp takes blocks of 32 tokens, as two strips of 16: S^T = K Q^T (m = 16 tokens,
// n = 8 rows) and O^T += V^T P^T (m = 16 elements, k = 16 tokens) by warp-level matrix instructions, which
// need 8 rows only where the 128-row tcgen05 tiles would be nearly empty.  Codes go from shared memory
// straight into fragments (the cache's layout is theirs: 16-byte loads, no shuffle) and are widened to f16
// exactly; K's block scales multiply the partial sums of their block, V's the softmax weights, relative to the
// largest scale a warp has met.  Each warp copies its own blocks, kStages deep, with nothing shared
// until the end, where the warps' sums are joined.
constexpr int kFewThreads = 128;
constexpr int kStages = 3;
constexpr int kFewShift = 5;

// A block of 32 tokens in shared memory: K codes, V codes, K scales, V scales.
template <int D>
struct TokenBlock {
    static constexpr int kBlocks = D / 32;
    static constexpr int kV = 16 * D, kKs = 32 * D, kVs = kKs + 32 * kBlocks, kBytes = kVs + 32 * kBlocks;
    static constexpr int kStrip = 8 * D;  // codes of 16 tokens
    // 16-byte pieces of V lie swizzled, so that the fragment loads of 8 lanes meet 8 different banks
    __device__ static __forceinline__ int v_piece(int pair, int piece) {
        return D == 128 ? pair * 8 + (piece ^ ((pair & 3) * 2)) : pair * 4 + (piece ^ (((pair >> 1) & 1) * 2));
    }
};

// CTAs of an SM: what its registers hold (168 a thread, 255 with 32 rows).
constexpr int few_resident(int NT) { return NT == 4 ? 2 : 3; }

template <int D, int NT>
struct FewShared {
    static constexpr int kBlocks = D / 32;
    static constexpr size_t kRing = 4 * kStages * TokenBlock<D>::kBytes, kJoin = 4 * 8 * D * sizeof(float);
    alignas(16) uint8_t ring[kRing > kJoin ? kRing : kJoin];  // in the end the warps' sums of 8 rows
    alignas(16) __half q[8 * NT][D + 8];
    alignas(16) float kscale[4][2][16][kBlocks];    // a warp's strips: 2^(e - 127) of K's blocks
    alignas(16) uint32_t vscale[4][2][8][kBlocks];  // f16 2^(e - vref) of V's, two tokens
    float factor[8 * NT];
    int lo[8 * NT], hi[8 * NT];
    float2 ml[4][8];
    float vref[4];
    int64_t scan[4];
    int first_seq;
    int64_t first_pos;
};

// One unit, blocks [begin, end) of its span (absolute block numbers); slot < 0: the result itself.
template <int D, int NT>
__device__ __forceinline__ void few_unit(const AttendParams& p, FewShared<D, NT>& sm, const Sequence& s, int b, int kvh,
                                         int r0, int nrows, const Span& sp, int begin, int end, int64_t slot) {
    using S = TokenBlock<D>;
    constexpr int kBlocks = D / 32, kRows = 8 * NT;
    constexpr int kSub = NT == 4 ? 1 : 2;  // strips worked on together, as registers allow
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const int g = lane >> 2, c = lane & 3;
    const int count = max(0, (end - begin - warp + 3) >> 2);  // blocks of this warp
    const int32_t* table = p.tables + b * p.table_width;
    uint8_t* ring = sm.ring + warp * kStages * S::kBytes;
    unsigned gone_bits = 0;  // bits 2 stage + u: strips (16 tokens) that were not copied
    // what a lane copies: 16 bytes of every 512 of the codes, and a piece of the scales
    const PageLayout<D> lay{p.page_size};
    const uint8_t* head = p.cache + kvh * lay.bytes();
    const uint32_t page_stride = static_cast<uint32_t>(p.Hk * lay.bytes());
    const uint32_t ring_at = smem_u32(ring) + 16 * lane;
    const uint32_t v_at = smem_u32(ring) + S::kV + 16 * S::v_piece(lane / (D / 16), lane % (D / 16));
    const bool small_pages = p.page_size < 32;
    const int scale_at = lane < 2 * kBlocks ? lay.k_scales() + 16 * lane : lay.v_scales() + 16 * (lane - 2 * kBlocks);
    int ahead = (begin + warp) * 32;  // first token of the block to fetch next
    const int fetch_end = end * 32;
    auto page_of = [&](int t) { return t < fetch_end ? table[t >> p.page_shift] : -1; };
    auto fetch = [&](unsigned stage, int pg) {
        if (ahead < fetch_end) {
            const uint32_t to = stage * S::kBytes;
            gone_bits &= ~(3u << (2 * stage));
            if (small_pages) {  // the block's strips lie in pages of their own
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int t = ahead + 16 * u;
                    const bool seen = t <= sp.last_hi && t + 15 >= sp.first_lo;
                    const int pu = seen ? table[t >> 4] : -1;
                    if (static_cast<unsigned>(pu) < static_cast<uint64_t>(p.num_pages)) {
                        const uint8_t* page = head + static_cast<uint64_t>(static_cast<uint32_t>(pu)) * page_stride;
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            const uint32_t at = to + u * S::kStrip + 512 * x;
                            cp_async16(ring_at + at, page + 16 * lane + 512 * x);
                            cp_async16(v_at + at, page + lay.v_codes() + 16 * lane + 512 * x);
                        }
                        if (lane < 2 * kBlocks)  // of K, then of V: the block's K scales lie between
                            cp_async16(ring_at + to + S::kKs + 16 * kBlocks * u + (lane < kBlocks ? 0 : 16 * kBlocks),
                                       page + lay.k_scales() + 16 * lane);
                    } else {
                        gone_bits |= 1u << (2 * stage + u);
                        if (seen && lane == 0) report_index();
                    }
                }
            } else if (static_cast<unsigned>(pg) < static_cast<uint64_t>(p.num_pages)) {
                const int at = ahead & (p.page_size - 1);
                const uint8_t* page = head + static_cast<uint64_t>(static_cast<uint32_t>(pg)) * page_stride;
                const uint8_t* kc = page + (at * lay.kRow + 16 * lane);  // V's pair rows lie as far apart as two K rows
                const uint8_t* vc = kc + lay.v_codes();
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    cp_async16(ring_at + to + 512 * x, kc + 512 * x);
                    cp_async16(v_at + to + 512 * x, vc + 512 * x);
                }
                if (lane < 4 * kBlocks) cp_async16(ring_at + to + S::kKs, page + (scale_at + at * kBlocks));
            } else {
                gone_bits |= 3u << (2 * stage);
                if (lane == 0) report_index();
            }
        }
        cp_async_commit();
        ahead += 128;
    };
    int next_page = page_of(ahead);
#pragma unroll
    for (unsigned i = 0; i < kStages - 1; ++i) {
        const int pg = next_page;
        next_page = page_of(ahead + 128);
        fetch(i, pg);
    }

    for (int r = warp; r < kRows; r += 4) {
        const bool real = r < nrows;
        const int qi = (r0 + r) / p.G;
        const uint16_t* src = p.q + (s.row0 + qi) * p.ldq + static_cast<int64_t>(kvh * p.G + (r0 + r) - qi * p.G) * D;
        float x[kBlocks];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const uint32_t w = real ? static_cast<uint32_t>(src[32 * i + lane]) << 16 : 0u;
            x[i] = __uint_as_float(w);
            top = max(top, w & 0x7FFFFFFFu);
        }
        const uint32_t E = query_exponent(__reduce_max_sync(0xFFFFFFFFu, top));
        const float mul = query_multiplier(E);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
            sm.q[r][32 * i + lane] = __float2half_rn(warp_fwht32(x[i] * mul, lane) * kHadamardNorm);
        if (lane == 0) {
            sm.factor[r] = score_factor(p.scale_log2, E);
            sm.lo[r] = first_key(p, s.pos0 + qi);
            sm.hi[r] = real ? s.pos0 + qi : -1;
        }
    }
    __syncthreads();

    // thread (g, c): tokens g, g + 8 of a strip and rows 2c, 2c + 1 of each n-tile; of Q rows g
    uint4 qf[kBlocks];
    if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) qf[i] = *reinterpret_cast<const uint4*>(&sm.q[g][32 * i + 8 * c]);
    }
    float f[NT][2], ref[NT][2], bound[NT][2], sum[NT][2], o[NT][2 * kBlocks][4];
    const int vp = D == 128 ? lane >> 2 : (lane >> 1) & 7, vb = lane & (kBlocks - 1);
    int vref = 0;  // above the largest V scale met, which the sums are relative to
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f[n][e] = sm.factor[8 * n + 2 * c + e];
            ref[n][e] = 0.0f, bound[n][e] = -INFINITY, sum[n][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 2 * kBlocks; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
    }

    unsigned stage = 0;
    int base = (begin + warp) * 32;
    for (int i = 0; i < count; ++i, base += 128) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const unsigned gone2 = gone_bits >> (2 * stage);
        {
            const int pg = next_page;
            next_page = page_of(ahead + 128);
            fetch(stage == 0 ? kStages - 1 : stage - 1, pg);
        }
        const uint8_t* st0 = ring + stage * S::kBytes;
        stage = stage == kStages - 1 ? 0 : stage + 1;

        // The scales are widened once for the warp, here two (D = 64: one) K values a lane and strip.  (e = 0,
        // below the smallest normal, counts as 0.)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t* st = st0 + S::kKs + 16 * kBlocks * u;
            float* ks = &sm.kscale[warp][u][0][0];
            if constexpr (D == 128) {
                const uint32_t w = *reinterpret_cast<const uint16_t*>(st + 2 * lane);
                *reinterpret_cast<float2*>(ks + 2 * lane) =
                    make_float2(__uint_as_float((w & 0xFFu) << 23), __uint_as_float((w << 15) & 0x7F800000u));
            } else {
                ks[lane] = __uint_as_float(static_cast<uint32_t>(st[lane]) << 23);
            }
        }
        __syncwarp();

#pragma unroll 1
        for (int half = 0; half < 2; half += kSub) {
            float sc[kSub][NT][4];
            int ve[kSub][2];  // scales of block vb of V's tokens 2 vp, 2 vp + 1
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const uint8_t* st = st0 + (half + u) * S::kStrip;
                const uint8_t* vs = st0 + S::kVs + 16 * kBlocks * (half + u) + 2 * kBlocks * vp + vb;
                ve[u][0] = vs[0], ve[u][1] = vs[kBlocks];
                const float* ks = &sm.kscale[warp][half + u][0][0];
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[u][n][0] = sc[u][n][1] = sc[u][n][2] = sc[u][n][3] = 0.0f;
                uint32_t k0[kBlocks], k1[kBlocks];
                float x0[kBlocks], x1[kBlocks];
                if constexpr (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4*>(st + g * 64 + c * 16);
                    const uint4 z = *reinterpret_cast<const uint4*>(st + (g + 8) * 64 + c * 16);
                    k0[0] = a.x, k0[1] = a.y, k0[2] = a.z, k0[3] = a.w;
                    k1[0] = z.x, k1[1] = z.y, k1[2] = z.z, k1[3] = z.w;
                    const float4 y = *reinterpret_cast<const float4*>(ks + 4 * g);
                    const float4 v = *reinterpret_cast<const float4*>(ks + 4 * (g + 8));
                    x0[0] = y.x, x0[1] = y.y, x0[2] = y.z, x0[3] = y.w;
                    x1[0] = v.x, x1[1] = v.y, x1[2] = v.z, x1[3] = v.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(st + g * 32 + c * 8);
                    const uint2 z = *reinterpret_cast<const uint2*>(st + (g + 8) * 32 + c * 8);
                    k0[0] = a.x, k0[1] = a.y, k1[0] = z.x, k1[1] = z.y;
                    const float2 y = *reinterpret_cast<const float2*>(ks + 2 * g);
                    const float2 v = *reinterpret_cast<const float2*>(ks + 2 * (g + 8));
                    x0[0] = y.x, x0[1] = y.y, x1[0] = v.x, x1[1] = v.y;
                }
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    uint32_t a[4], z[4];
                    e2m1x8_to_f16(k0[j], a);
                    e2m1x8_to_f16(k1[j], z);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint4 q;
                        if constexpr (NT == 1)
                            q = qf[j];
                        else
                            q = *reinterpret_cast<const uint4*>(&sm.q[8 * n + g][32 * j + 8 * c]);
                        float acc[4];
                        mma_f16_16x8x16_first(acc, a[0], z[0], a[1], z[1], q.x, q.y);
                        mma_f16_16x8x16(acc, a[2], z[2], a[3], z[3], q.z, q.w);
                        sc[u][n][0] += acc[0] * x0[j], sc[u][n][1] += acc[1] * x0[j];
                        sc[u][n][2] += acc[2] * x1[j], sc[u][n][3] += acc[3] * x1[j];
                    }
                }
            }

            const int from = base + 16 * half;
            if (((gone2 >> half) & ((1u << kSub) - 1)) || from < sp.last_lo || from + 16 * kSub - 1 > sp.first_hi) {
                // strips that some row's mask cuts
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const bool gone = (gone2 >> (half + u)) & 1u;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int lo = sm.lo[8 * n + 2 * c + e], hi = gone ? -1 : sm.hi[8 * n + 2 * c + e];
                            const int t = from + 16 * u + g;
                            if (t < lo || t > hi) sc[u][n][e] = -INFINITY;
                            if (t + 8 < lo || t + 8 > hi) sc[u][n][2 + e] = -INFINITY;
                        }
                    }
                    // what lies there may be anything: no scale of a token that no row sees is used
                    const int t = from + 16 * u + 2 * vp;
                    if (gone || t < sp.first_lo || t > sp.last_hi) ve[u][0] = 0;
                    if (gone || t + 1 < sp.first_lo || t + 1 > sp.last_hi) ve[u][1] = 0;
                }
            }
            int vmax = max(ve[0][0], ve[0][1]);
            if constexpr (kSub == 2) vmax = max(vmax, max(ve[1][0], ve[1][1]));

            float top[NT][2];
            bool grow = vmax > vref;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[n][e] = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
                    if constexpr (kSub == 2) top[n][e] = fmaxf(top[n][e], fmaxf(sc[1][n][e], sc[1][n][2 + e]));
                    top[n][e] *= f[n][e];
                    grow |= top[n][e] > bound[n][e];
                }
            }
            if (__any_sync(0xFFFFFFFFu, grow)) {
                float vf = 1.0f;
                const int nv = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(vmax)));
                if (nv > vref) {  // with room for three doublings before the next time
                    const int to = min(nv + 3, 254);
                    vf = to - vref < 127 ? __uint_as_float(static_cast<uint32_t>(127 - (to - vref)) << 23) : 0.0f;
                    vref = to;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = top[n][e];
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                        float scale = vf;
                        if (m > bound[n][e] - kSlack) {  // false while a row has seen nothing
                            const float old = ref[n][e];
                            ref[n][e] = m - kLift;
                            const float shift = bound[n][e] == -INFINITY ? 0.0f : exp2_approx(old - ref[n][e]);
                            bound[n][e] = m + kSlack;
                            sum[n][e] *= shift;
                            scale *= shift;
                        }
#pragma unroll
                        for (int x = 0; x < 2 * kBlocks; ++x) o[n][x][e] *= scale, o[n][x][2 + e] *= scale;
                    }
                }
            }

            // exponent field e - vref + 15 of two tokens, 0 below it
            const uint32_t k2 = static_cast<uint32_t>((15 - vref) & 0xFFFF) * 0x00010001u;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                sm.vscale[warp][half + u][vp][vb] =
                    __viaddmin_s16x2_relu(static_cast<uint32_t>(ve[u][0] | ve[u][1] << 16), k2, 0x000F000Fu) << 10;
            __syncwarp();

#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const uint8_t* st = st0 + (half + u) * S::kStrip;
                // softmax weights, transposed into fragments: tokens 2c, 2c + 1 (2c + 8, 2c + 9) of row g
                uint32_t pt0[NT], pt1[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float e0 = exp2_approx(fmaf(sc[u][n][0], f[n][0], -ref[n][0]));
                    const float e1 = exp2_approx(fmaf(sc[u][n][1], f[n][1], -ref[n][1]));
                    const float e2 = exp2_approx(fmaf(sc[u][n][2], f[n][0], -ref[n][0]));
                    const float e3 = exp2_approx(fmaf(sc[u][n][3], f[n][1], -ref[n][1]));
                    sum[n][0] += e0 + e2, sum[n][1] += e1 + e3;
                    const __half2 a = __floats2half2_rn(e0, e1), z = __floats2half2_rn(e2, e3);
                    pt0[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&a));
                    pt1[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&z));
                }
                uint32_t va[4], vz[4];  // pairs c and c + 4: (first token: blocks 01, 23), (second token: 01, 23)
                uint32_t vx0[kBlocks], vx1[kBlocks];
                const uint32_t* vs = &sm.vscale[warp][half + u][0][0];
                if constexpr (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4*>(st + S::kV + 16 * S::v_piece(c, g));
                    const uint4 z = *reinterpret_cast<const uint4*>(st + S::kV + 16 * S::v_piece(c + 4, g));
                    va[0] = a.x, va[1] = a.y, va[2] = a.z, va[3] = a.w;
                    vz[0] = z.x, vz[1] = z.y, vz[2] = z.z, vz[3] = z.w;
                    const uint4 y = *reinterpret_cast<const uint4*>(vs + 4 * c);
                    const uint4 w = *reinterpret_cast<const uint4*>(vs + 4 * (c + 4));
                    vx0[0] = y.x, vx0[1] = y.y, vx0[2] = y.z, vx0[3] = y.w;
                    vx1[0] = w.x, vx1[1] = w.y, vx1[2] = w.z, vx1[3] = w.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(st + S::kV + 16 * S::v_piece(c, g >> 1) + 8 * (g & 1));
                    const uint2 z = *reinterpret_cast<const uint2*>(st + S::kV + 16 * S::v_piece(c + 4, g >> 1) + 8 * (g & 1));
                    va[0] = a.x, va[1] = a.y, vz[0] = z.x, vz[1] = z.y;
                    const uint2 y = *reinterpret_cast<const uint2*>(vs + 2 * c);
                    const uint2 w = *reinterpret_cast<const uint2*>(vs + 2 * (c + 4));
                    vx0[0] = y.x, vx0[1] = y.y, vx1[0] = w.x, vx1[1] = w.y;
                }
#pragma unroll
                for (int h = 0; h < kBlocks / 2; ++h) {
                    // bytes whose nibbles are one element of the two tokens: elements 0, 2 and 1, 3 of two blocks
                    const uint32_t a0 = va[h], a1 = va[kBlocks / 2 + h], z0 = vz[h], z1 = vz[kBlocks / 2 + h];
                    const uint32_t ae = (a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u);
                    const uint32_t ao = ((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u);
                    const uint32_t ze = (z0 & 0x0F0F0F0Fu) | ((z1 << 4) & 0xF0F0F0F0u);
                    const uint32_t zo = ((z0 >> 4) & 0x0F0F0F0Fu) | (z1 & 0xF0F0F0F0u);
                    uint32_t ea[4], oa[4], ez[4], oz[4];
                    e2m1x8_to_f16(ae, ea), e2m1x8_to_f16(ao, oa);
                    e2m1x8_to_f16(ze, ez), e2m1x8_to_f16(zo, oz);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = 2 * h + y;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const __half2 b0 = __hmul2(*reinterpret_cast<const __half2*>(&pt0[n]), *reinterpret_cast<const __half2*>(&vx0[j]));
                            const __half2 b1 = __hmul2(*reinterpret_cast<const __half2*>(&pt1[n]), *reinterpret_cast<const __half2*>(&vx1[j]));
                            const uint32_t u0 = *reinterpret_cast<const uint32_t*>(&b0), u1 = *reinterpret_cast<const uint32_t*>(&b1);
                            mma_f16_16x8x16(o[n][2 * j], ea[2 * y], oa[2 * y], ez[2 * y], oz[2 * y], u0, u1);
                            mma_f16_16x8x16(o[n][2 * j + 1], ea[2 * y + 1], oa[2 * y + 1], ez[2 * y + 1], oz[2 * y + 1], u0, u1);
                        }
                    }
                }
            }
        }
    }
    cp_async_wait<0>();

    // join the warps, one n-tile (8 rows) at a time: warp w's sums of row r at joined[w][r][..]
    float* joined = reinterpret_cast<float*>(sm.ring);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (8 * n >= nrows) break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = sum[n][e];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
            if (g == 0) sm.ml[warp][2 * c + e] = make_float2(bound[n][e] == -INFINITY ? -INFINITY : ref[n][e], t);
#pragma unroll
            for (int j = 0; j < 2 * kBlocks; ++j) {
                float* row = joined + (warp * 8 + 2 * c + e) * D + 16 * j + 4 * g - (j & 1) * 14;
                *reinterpret_cast<float2*>(row) = make_float2(o[n][j][e], o[n][j][2 + e]);
            }
        }
        if (lane == 0) sm.vref[warp] = __uint_as_float(static_cast<uint32_t>(vref) << 23);
        __syncthreads();
        constexpr int kAtOnce = kFewThreads / D;
        const int d = threadIdx.x % D;
#pragma unroll
        for (int r1 = 0; r1 < 8; r1 += kAtOnce) {
            const int r = r1 + threadIdx.x / D;  // uniform over a warp
            if (8 * n + r >= nrows) continue;
            float m = -INFINITY, total = 0.0f, x = 0.0f, w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, sm.ml[k][r].x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = sm.ml[k][r].x == -INFINITY ? 0.0f : exp2_approx(sm.ml[k][r].x - m);
                total += w[k] * sm.ml[k][r].y;
            }
            const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // divided first: the sums times a large scale might not fit
                if (w[k] != 0.0f) x += joined[(k * 8 + r) * D + d] * (w[k] * inv) * sm.vref[k];
            if (slot >= 0) {
                const int64_t at = slot * p.tile_rows + 8 * n + r;
                p.part_o[at * D + d] = x;
                if (d == 0) p.part_ml[at] = make_float2(m, total);
            } else {
                const int rr = r0 + 8 * n + r, qi = rr / p.G;
                const int64_t row = (s.row0 + qi) * p.Hq + kvh * p.G + rr - qi * p.G;
                x = warp_fwht32(x * kHadamardNorm, lane);
                p.out[row * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
                if (p.lse && d == 0) p.lse[row] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
            }
        }
    }
    __syncthreads();
}

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, few_resident(NT)) attend_few_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ uint4 dynamic_smem[];
    FewShared<D, NT>& sm = *reinterpret_cast<FewShared<D, NT>*>(dynamic_smem);
    constexpr int kRows = 8 * NT;
    griddep_launch_dependents();
    griddep_wait();
    Cut cut;
    if (p.ctas) {
        cut = cut_of(p, kFewShift, sm.scan, &sm.first_seq, &sm.first_pos);
    } else {  // one unit
        cut.b = static_cast<int>(blockIdx.x / p.row_tiles / p.Hk);
        cut.pos = cut.seq_pos = 0, cut.end = 1;
    }
    while (cut.pos < cut.end) {
        const Sequence s = sequence_of(p, cut.b);
        const int rows = s.nq * p.G;
        int kvh, r0, from, to;
        int64_t slot = -1;
        Span sp;
        if (p.ctas) {
            const int64_t per_head = sequence_blocks(p, s, kFewShift);
            int64_t off = cut.pos - cut.seq_pos;
            if (per_head == 0 || off >= per_head * p.Hk) {
                cut.seq_pos += per_head * p.Hk;
                ++cut.b;
                continue;
            }
            kvh = static_cast<int>(off / per_head);
            off -= kvh * per_head;
            int n;
            for (r0 = 0;; r0 += kRows) {
                sp = span_of(p, s, r0, min(kRows, rows - r0));
                n = blocks_of(sp, kFewShift);
                if (off < n) break;
                off -= n;
            }
            from = static_cast<int>(off), to = static_cast<int>(min(static_cast<int64_t>(n), off + cut.end - cut.pos));
            cut.pos += to - from;
            if (from != 0 || to != n) slot = 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
        } else {
            kvh = static_cast<int>(blockIdx.x / p.row_tiles % p.Hk), r0 = static_cast<int>(blockIdx.x % p.row_tiles) * kRows;
            if (r0 >= rows) return;
            sp = span_of(p, s, r0, min(kRows, rows - r0));
            from = 0, to = blocks_of(sp, kFewShift);
            cut.pos = cut.end;
        }
        const int begin = sp.first_lo >> kFewShift;
        few_unit<D, NT>(p, sm, s, cut.b, kvh, r0, min(kRows, rows - r0), sp, begin + from, begin + to, slot);
    }
}

// Joins the parts of a row: one warp per (sequence, query, head).  Rows that one CTA wrote are left alone,
// rows that see nothing get their zeros here.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendParams p, int shift) {
    constexpr int kElems = D / 32;  // of a lane, neighbours
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int64_t query = item / p.Hq;
    const int h = static_cast<int>(item - query * p.Hq);
    const int b = static_cast<int>(query / p.max_q), qi = static_cast<int>(query % p.max_q);
    if (b >= p.B) return;
    int64_t before = 0, total_blocks = 0;
    for (int x = lane; x < p.B; x += 32) {
        const int64_t n = sequence_blocks(p, sequence_of(p, x), shift) * p.Hk;
        total_blocks += n;
        if (x < b) before += n;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        total_blocks += __shfl_xor_sync(0xFFFFFFFFu, total_blocks, x);
        before += __shfl_xor_sync(0xFFFFFFFFu, before, x);
    }
    const Sequence s = sequence_of(p, b);
    if (qi >= s.nq) return;
    const int kvh = h / p.G, r = qi * p.G + h - kvh * p.G, rows = s.nq * p.G;
    int64_t u0 = before + kvh * sequence_blocks(p, s, shift);
    int r0 = 0, n = blocks_of(span_of(p, s, 0, min(p.tile_rows, rows)), shift);
    while (r0 + p.tile_rows <= r) {
        u0 += n;
        r0 += p.tile_rows;
        n = blocks_of(span_of(p, s, r0, min(p.tile_rows, rows - r0)), shift);
    }
    const int64_t len = cut_length(p, total_blocks, shift);
    const int64_t c0 = u0 / len, c1 = n ? (u0 + n - 1) / len : c0 - 1;  // the CTAs that hold parts
    if (c0 == c1) return;
    // the first part is what its CTA's range ends in (slot 1), the others are what theirs begin with (slot 0)
    const int64_t stride = 2 * p.tile_rows;
    const int64_t at = c0 * stride + r - r0;
    auto place = [&](int64_t k) { return at + k * stride + (k == 0 ? p.tile_rows : 0); };
    const int parts = static_cast<int>(c1 - c0 + 1);
    float m = -INFINITY;
    for (int k = lane; k < parts; k += 32) m = fmaxf(m, p.part_ml[place(k)].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    float total = 0.0f, o[kElems] = {};
    for (int k0 = 0; k0 < parts; k0 += 32) {
        float w = 0.0f;  // of part k0 + lane
        if (k0 + lane < parts) {
            const float2 ml = p.part_ml[place(k0 + lane)];
            if (ml.x != -INFINITY) w = exp2_approx(ml.x - m) * ml.y;
        }
        const int n = min(32, parts - k0);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const float* src = p.part_o + place(k0 + k) * D + kElems * lane;
            total += wk;
#pragma unroll
            for (int j = 0; j < kElems; ++j) o[j] += wk == 0.0f ? 0.0f : wk * src[j];
        }
    }
    const float inv = total > 0.0f ? kHadamardNorm / total : total == 0.0f ? 0.0f : total;
#pragma unroll
    for (int j = 0; j < kElems; ++j) o[j] *= inv;
#pragma unroll
    for (int x = 1; x < kElems; x <<= 1)  // distances inside the lane
#pragma unroll
        for (int j = 0; j < kElems; ++j)
            if ((j & x) == 0) {
                const float a = o[j], z = o[j + x];
                o[j] = a + z, o[j + x] = a - z;
            }
#pragma unroll
    for (int x = 1; x * kElems < 32; x <<= 1) {
#pragma unroll
        for (int j = 0; j < kElems; ++j) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, o[j], x);
            o[j] = lane & x ? y - o[j] : o[j] + y;
        }
    }
    const int64_t row = (s.row0 + qi) * p.Hq + h;
    uint16_t* dst = p.out + row * D + kElems * lane;
#pragma unroll
    for (int j = 0; j < kElems; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = pack_bf16(o[j], o[j + 1]);
    if (p.lse && lane == 0) p.lse[row] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
}

// ------------------------------------------------------------------------------------ host side

constexpr int64_t kMaxKeys = int64_t{1} << 30;  // of a sequence: positions and block ends stay in 32 bits

// How a call is split, from what the host knows (not the sequences' lengths).
struct AttendPlan {
    int tile_rows, row_tiles, ctas;
    int64_t units;
    size_t bytes;
};
static AttendPlan plan_attend(int64_t B, int Hq, int Hk, int D, int64_t max_q) {
    AttendPlan a;
    const int64_t rows = max_q * (Hq / Hk);
    a.tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    a.row_tiles = static_cast<int>((rows + a.tile_rows - 1) / a.tile_rows);
    a.units = B * Hk * a.row_tiles;
    // cut while there are few units: many balance themselves, and need no joining
    const int resident = sm_count() * few_resident(a.tile_rows / 8);
    a.ctas = a.units >= 4 * resident ? 0 : resident;
    a.bytes = static_cast<size_t>(a.ctas) * 2 * a.tile_rows * (static_cast<size_t>(D) * 4 + 8);
    a.bytes = (a.bytes + 255) / 256 * 256 + 256;
    return a;
}

template <int D, int NT>
static int launch_few(const AttendParams& p, unsigned blocks, cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(FewShared<D, NT>);
    static_assert(few_resident(NT) * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    if (cudaFuncSetAttribute(attend_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return MACAQ_ECUDA;
    return launch_dependent_smem(attend_few_kernel<D, NT>, dim3(blocks), kFewThreads, kSmem, stream, p);
}

template <int D>
static int launch_attend(const AttendParams& p, int64_t units, cudaStream_t stream) {
    const int64_t blocks = p.ctas ? p.ctas : units;
    const int64_t join = (static_cast<int64_t>(p.B) * p.max_q * p.Hq + 3) / 4;
    if (blocks > kMaxDim || join > kMaxDim) return MACAQ_ESHAPE;
    const auto n = static_cast<unsigned>(blocks);
    const int st = p.tile_rows == 8    ? launch_few<D, 1>(p, n, stream)
                   : p.tile_rows == 16 ? launch_few<D, 2>(p, n, stream)
                                       : launch_few<D, 4>(p, n, stream);
    if (st != MACAQ_OK || !p.ctas) return st;
    return launch_dependent(attend_join_kernel<D>, dim3(static_cast<unsigned>(join)), 128, stream, p, kFewShift);
}

}  // namespace macaq

extern "C" size_t macaq_kv4_attention_workspace_bytes(int64_t T, int64_t B, int Hq, int Hk, int head_dim, int64_t max_q) {
    if (!head_dim_ok(head_dim) || T < 0 || T > kMaxDim || B < 0 || B > kMaxDim || Hk < 1 || Hq < Hk || Hq > kMaxHeads ||
        Hq % Hk != 0 || max_q < 1 || max_q > kMaxDim / kMaxHeads)
        return 0;
    if (T == 0 || B == 0) return 256;
    return plan_attend(B, Hq, Hk, head_dim, max_q).bytes;
}

extern "C" int macaq_kv4_attention(const uint16_t* q, int64_t T, int64_t ldq, int Hq, int Hk, int head_dim,
                                   const uint8_t* cache, int64_t num_pages, int page_size, const int32_t* tables,
                                   int64_t B, int64_t table_width, const int32_t* kv_lens, const int32_t* cu_q,
                                   int64_t max_q, float scale, int64_t window, uint16_t* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    const size_t need = macaq_kv4_attention_workspace_bytes(T, B, Hq, Hk, head_dim, max_q);
    if (need == 0 || !page_size_ok(page_size) || num_pages < 1 || num_pages > kMaxDim || table_width < 0 ||
        table_width > kMaxKeys / page_size || ldq < static_cast<int64_t>(Hq) * head_dim || ldq > kMaxDim || ldq % 8 != 0 ||
        window < 0)
        return MACAQ_ESHAPE;
    if (!cu_q && (B != T || max_q != 1)) return MACAQ_ESHAPE;
    if (!(scale > 0.0f) || std::isinf(scale)) return MACAQ_EINVAL;
    if (T == 0 || B == 0) return MACAQ_OK;
    if (!q || !cache || !kv_lens || !out || !workspace || (table_width && !tables)) return MACAQ_EINVAL;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(tables) & 3u) || (reinterpret_cast<uintptr_t>(kv_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_q) & 3u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
        return MACAQ_EALIGN;
    if (workspace_bytes < need) return MACAQ_EWORKSPACE;
    const AttendPlan plan = plan_attend(B, Hq, Hk, head_dim, max_q);
    AttendParams p = {};
    p.q = q, p.T = T, p.ldq = ldq, p.Hq = Hq, p.Hk = Hk, p.G = Hq / Hk, p.cache = cache, p.num_pages = num_pages;
    p.page_size = page_size, p.page_shift = __builtin_ctz(page_size), p.tables = tables, p.table_width = table_width;
    p.kv_lens = kv_lens, p.cu_q = cu_q, p.B = static_cast<int>(B), p.max_q = static_cast<int>(max_q);
    p.scale_log2 = scale * kLog2e, p.window = static_cast<int>(window < kMaxDim ? window : 0), p.out = out, p.lse = lse;
    p.tile_rows = plan.tile_rows, p.row_tiles = plan.row_tiles, p.ctas = plan.ctas;
    p.part_ml = static_cast<float2*>(workspace);
    p.part_o = reinterpret_cast<float*>(p.part_ml + static_cast<int64_t>(p.ctas) * 2 * p.tile_rows);
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_attend<64>(p, plan.units, s) : launch_attend<128>(p, plan.units, s);
}
