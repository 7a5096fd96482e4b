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
    // the split of the work (plan_attend): row tiles of tile_rows rows, each cut along its keys into
    // at most `splits` parts whose results are joined by attend_join_kernel (splits = 1: written directly)
    int tile_rows, row_tiles, splits;
    float* part_o;    // fp32 [splits][units][tile_rows][D], each row divided by its own sum
    float2* part_ml;  // [splits][units][tile_rows]: its reference m (base 2) and sum of 2^(s - m)
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

// Part `split` of a span in blocks of 2^shift keys: blocks [begin, end) of it, of `parts` parts in use.
// No part is shorter than kMinKeys keys (a shorter one costs more to join than it saves).
constexpr int kMinKeys = 128;
struct Part {
    int begin, end, parts;
};
__device__ __forceinline__ Part part_of(const AttendParams& p, const Span& sp, int shift, int split) {
    if (sp.last_hi < 0) return {0, 0, 0};
    const int b0 = sp.first_lo >> shift, n = (sp.last_hi >> shift) - b0 + 1;
    const int len = max((n + p.splits - 1) / p.splits, kMinKeys >> shift);
    const int begin = min(n, split * len);
    return {b0 + begin, b0 + min(n, begin + len), (n + len - 1) / len};
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
// One CTA of 4 warps per (sequence, kv head, tile of 8 NT rows, part of the keys).  A warp takes strips
// of 16 tokens: S^T = K Q^T (m = 16 tokens, n = 8 rows) and O^T += V^T P^T (m = 16 elements, k = 16
// tokens) by warp-level matrix instructions, which need 8 rows only where the 128-row tcgen05 tiles would
// be nearly empty.  Codes go from shared memory straight into fragments (the cache's layout is theirs:
// 16-byte loads, no shuffle) and are widened to f16 exactly; K's block scales multiply the partial sums of
// their block, V's the softmax weights, relative to the largest scale a warp has met.  Each warp copies its
// own strips, kStages deep, with nothing shared until the end, where the warps' sums are joined.
// Bound by the cache's bytes at long contexts; the work of widening (a conversion per two codes) comes next.
constexpr int kFewThreads = 128;
constexpr int kStages = 4;

template <int D>
struct Strip {
    static constexpr int kBlocks = D / 32;
    static constexpr int kV = 8 * D;         // K codes of 16 tokens come first
    static constexpr int kKs = 16 * D;       // then V codes, then the scales
    static constexpr int kVs = kKs + 16 * kBlocks;
    static constexpr int kBytes = kVs + 16 * kBlocks;
    // 16-byte pieces of V lie swizzled, so that the fragment loads of 8 lanes meet 8 different banks
    __device__ static __forceinline__ int v_piece(int pair, int piece) {
        return D == 128 ? pair * 8 + (piece ^ ((pair & 3) * 2)) : pair * 4 + (piece ^ (((pair >> 1) & 1) * 2));
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads) attend_few_kernel(const __grid_constant__ AttendParams p) {
    using S = Strip<D>;
    constexpr int kBlocks = D / 32, kRows = 8 * NT, kQStride = D + 8;
    extern __shared__ uint4 dynamic_smem[];
    __shared__ __align__(16) __half q_s[kRows][kQStride];
    __shared__ float factor_s[kRows];
    __shared__ int lo_s[kRows], hi_s[kRows];
    __shared__ float2 ml_s[4][8];
    __shared__ float vref_s[4];

    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int64_t block = blockIdx.x;
    const int rt = static_cast<int>(block % p.row_tiles);
    const int split = static_cast<int>(block / p.row_tiles % p.splits);
    const int64_t bh = block / p.row_tiles / p.splits;
    const int kvh = static_cast<int>(bh % p.Hk), b = static_cast<int>(bh / p.Hk);
    const Sequence s = sequence_of(p, b);
    const int r0 = rt * kRows;
    const int nrows = min(kRows, s.nq * p.G - r0);
    if (nrows <= 0) return;
    const Span sp = span_of(p, s, r0, nrows);
    const Part part = part_of(p, sp, 4, split);
    if (p.splits > 1 && part.begin >= part.end) return;

    const int count = max(0, (part.end - part.begin - warp + 3) >> 2);  // strips of this warp
    const PageLayout<D> lay{p.page_size};
    const int32_t* table = p.tables + b * p.table_width;
    uint8_t* ring = reinterpret_cast<uint8_t*>(dynamic_smem) + warp * kStages * S::kBytes;
    unsigned bad = 0;  // stages whose page lies outside the cache
    auto page_of = [&](int i) { return i < count ? table[((part.begin + warp + 4 * i) * 16) >> p.page_shift] : 0; };
    auto fetch = [&](int i, int32_t pg) {
        if (i < count) {
            const int stage = i % kStages;
            const bool ok = pg >= 0 && pg < p.num_pages;
            bad = (bad & ~(1u << stage)) | (ok ? 0u : 1u << stage);
            if (ok) {
                const int at = ((part.begin + warp + 4 * i) * 16) & (p.page_size - 1);
                const uint8_t* page = p.cache + (static_cast<int64_t>(pg) * p.Hk + kvh) * lay.bytes();
                const uint8_t* kc = page + at * lay.kRow;
                const uint8_t* vc = page + lay.v_codes() + (at >> 1) * D;
                uint8_t* dst = ring + stage * S::kBytes;
#pragma unroll
                for (int u = 0; u < D / 64; ++u) {
                    const int x = lane + 32 * u;
                    cp_async16(dst + 16 * x, kc + 16 * x);
                    cp_async16(dst + S::kV + 16 * S::v_piece(x / (D / 16), x % (D / 16)), vc + 16 * x);
                }
                if (lane < kBlocks)
                    cp_async16(dst + S::kKs + 16 * lane, page + lay.k_scales() + at * kBlocks + 16 * lane);
                else if (lane < 2 * kBlocks)
                    cp_async16(dst + S::kVs + 16 * (lane - kBlocks),
                               page + lay.v_scales() + at * kBlocks + 16 * (lane - kBlocks));
            } else if (lane == 0) {
                report_index();
            }
        }
        cp_async_commit();
    };
    {
        int32_t pg[kStages - 1];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) pg[i] = page_of(i);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i, pg[i]);
    }
    int32_t next_page = page_of(kStages - 1);

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
            q_s[r][32 * i + lane] = __float2half_rn(warp_fwht32(x[i] * mul, lane) * kHadamardNorm);
        if (lane == 0) {
            factor_s[r] = score_factor(p.scale_log2, E);
            lo_s[r] = first_key(p, s.pos0 + qi);
            hi_s[r] = real ? s.pos0 + qi : -1;
        }
    }
    __syncthreads();

    // thread (g, c): tokens g, g + 8 of a strip and rows 2c, 2c + 1 of each n-tile; of Q rows g
    uint4 qf[kBlocks];
    if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) qf[i] = *reinterpret_cast<const uint4*>(&q_s[g][32 * i + 8 * c]);
    }
    float f[NT][2], ref[NT][2], bound[NT][2], sum[NT][2], o[NT][2 * kBlocks][4];
    int vref = 0;  // the largest V scale met, to which the sums are relative
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            f[n][e] = factor_s[8 * n + 2 * c + e];
            ref[n][e] = 0.0f, bound[n][e] = -INFINITY, sum[n][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 2 * kBlocks; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
    }

    for (int i = 0; i < count; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        fetch(i + kStages - 1, next_page);
        next_page = page_of(i + kStages);
        const int stage = i % kStages;
        const uint8_t* st = ring + stage * S::kBytes;
        const int base = (part.begin + warp + 4 * i) * 16;
        const bool gone = (bad >> stage) & 1u;

        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
        uint32_t k0[kBlocks], k1[kBlocks], ks0, ks1;
        if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(st + g * 64 + c * 16);
            const uint4 z = *reinterpret_cast<const uint4*>(st + (g + 8) * 64 + c * 16);
            k0[0] = a.x, k0[1] = a.y, k0[2] = a.z, k0[3] = a.w;
            k1[0] = z.x, k1[1] = z.y, k1[2] = z.z, k1[3] = z.w;
            ks0 = *reinterpret_cast<const uint32_t*>(st + S::kKs + 4 * g);
            ks1 = *reinterpret_cast<const uint32_t*>(st + S::kKs + 4 * (g + 8));
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(st + g * 32 + c * 8);
            const uint2 z = *reinterpret_cast<const uint2*>(st + (g + 8) * 32 + c * 8);
            k0[0] = a.x, k0[1] = a.y, k1[0] = z.x, k1[1] = z.y;
            ks0 = *reinterpret_cast<const uint16_t*>(st + S::kKs + 2 * g);
            ks1 = *reinterpret_cast<const uint16_t*>(st + S::kKs + 2 * (g + 8));
        }
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const uint32_t a[4] = {e2m1x2_to_f16x2<0>(k0[j]), e2m1x2_to_f16x2<1>(k0[j]), e2m1x2_to_f16x2<2>(k0[j]),
                                   e2m1x2_to_f16x2<3>(k0[j])};
            const uint32_t z[4] = {e2m1x2_to_f16x2<0>(k1[j]), e2m1x2_to_f16x2<1>(k1[j]), e2m1x2_to_f16x2<2>(k1[j]),
                                   e2m1x2_to_f16x2<3>(k1[j])};
            // 2^(e - 127) of the two tokens' blocks (e = 0, below the smallest normal, counts as 0)
            const float x0 = __uint_as_float(((ks0 >> (8 * j)) & 0xFFu) << 23);
            const float x1 = __uint_as_float(((ks1 >> (8 * j)) & 0xFFu) << 23);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 q;
                if constexpr (NT == 1)
                    q = qf[j];
                else
                    q = *reinterpret_cast<const uint4*>(&q_s[8 * n + g][32 * j + 8 * c]);
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16_16x8x16(acc, a[0], z[0], a[1], z[1], q.x, q.y);
                mma_f16_16x8x16(acc, a[2], z[2], a[3], z[3], q.z, q.w);
                sc[n][0] += acc[0] * x0, sc[n][1] += acc[1] * x0;
                sc[n][2] += acc[2] * x1, sc[n][3] += acc[3] * x1;
            }
        }

        // V scales of tokens 2c, 2c + 1 and 2c + 8, 2c + 9, two tokens' bytes of block j in 16-bit lanes
        uint32_t vs0[kBlocks], vs1[kBlocks];
        {
            uint32_t w[4];
            if constexpr (D == 128) {
                const uint2 lo = *reinterpret_cast<const uint2*>(st + S::kVs + 8 * c);
                const uint2 hi = *reinterpret_cast<const uint2*>(st + S::kVs + 8 * c + 32);
                w[0] = lo.x, w[1] = lo.y, w[2] = hi.x, w[3] = hi.y;
            } else {
                const uint32_t lo = *reinterpret_cast<const uint32_t*>(st + S::kVs + 4 * c);
                const uint32_t hi = *reinterpret_cast<const uint32_t*>(st + S::kVs + 4 * c + 16);
                w[0] = lo & 0xFFFFu, w[1] = lo >> 16, w[2] = hi & 0xFFFFu, w[3] = hi >> 16;
            }
            if (gone || base < sp.last_lo || base + 15 > sp.first_hi) {  // a strip that some row's mask cuts
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int lo = lo_s[8 * n + 2 * c + e], hi = gone ? -1 : hi_s[8 * n + 2 * c + e];
                        const int t = base + g;
                        if (t < lo || t > hi) sc[n][e] = -INFINITY;
                        if (t + 8 < lo || t + 8 > hi) sc[n][2 + e] = -INFINITY;
                    }
                }
                // what lies there may be anything: no scale of a token that no row sees is used
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t = base + 2 * c + (u & 1) + 4 * (u & 2);
                    if (gone || t < sp.first_lo || t > sp.last_hi) w[u] = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                const uint32_t sel = j | j << 4 | (4 + j) << 8 | (4 + j) << 12;
                vs0[j] = __byte_perm(w[0], w[1], sel) & 0x00FF00FFu;
                vs1[j] = __byte_perm(w[2], w[3], sel) & 0x00FF00FFu;
            }
        }
        uint32_t vtop = __vmaxs2(vs0[0], vs1[0]);
#pragma unroll
        for (int j = 1; j < kBlocks; ++j) vtop = __vimax3_s16x2(vtop, vs0[j], vs1[j]);
        const int vmax = max(static_cast<int>(vtop & 0xFFFFu), static_cast<int>(vtop >> 16));

        bool grow = vmax > vref;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) grow |= fmaxf(sc[n][e], sc[n][2 + e]) * f[n][e] > bound[n][e];
        if (__any_sync(0xFFFFFFFFu, grow)) {
            const int nv = max(vref, static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(vmax))));
            const float vf = nv - vref < 127 ? __uint_as_float(static_cast<uint32_t>(127 - (nv - vref)) << 23) : 0.0f;
            vref = nv;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(sc[n][e], sc[n][2 + e]) * f[n][e];
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

        // softmax weights, transposed into fragments: tokens 2c, 2c + 1 (2c + 8, 2c + 9) of row g
        uint32_t pt0[NT], pt1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e0 = exp2_approx(fmaf(sc[n][0], f[n][0], -ref[n][0])), e1 = exp2_approx(fmaf(sc[n][1], f[n][1], -ref[n][1]));
            float e2 = exp2_approx(fmaf(sc[n][2], f[n][0], -ref[n][0])), e3 = exp2_approx(fmaf(sc[n][3], f[n][1], -ref[n][1]));
            sum[n][0] += e0 + e2, sum[n][1] += e1 + e3;
            const __half2 a = __floats2half2_rn(e0, e1), z = __floats2half2_rn(e2, e3);
            pt0[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&a));
            pt1[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&z));
        }

        uint32_t va[4], vz[4];  // pairs c and c + 4: (first token: blocks 01, 23), (second token: 01, 23)
        if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(st + S::kV + 16 * S::v_piece(c, g));
            const uint4 z = *reinterpret_cast<const uint4*>(st + S::kV + 16 * S::v_piece(c + 4, g));
            va[0] = a.x, va[1] = a.y, va[2] = a.z, va[3] = a.w;
            vz[0] = z.x, vz[1] = z.y, vz[2] = z.z, vz[3] = z.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(st + S::kV + 16 * S::v_piece(c, g >> 1) + 8 * (g & 1));
            const uint2 z = *reinterpret_cast<const uint2*>(st + S::kV + 16 * S::v_piece(c + 4, g >> 1) + 8 * (g & 1));
            va[0] = a.x, va[1] = a.y, vz[0] = z.x, vz[1] = z.y;
        }
        const uint32_t k2 = static_cast<uint32_t>((15 - vref) & 0xFFFF) * 0x00010001u;
#pragma unroll
        for (int h = 0; h < kBlocks / 2; ++h) {
            // bytes whose nibbles are one element of the two tokens: elements 0, 2 and 1, 3 of two blocks
            const uint32_t a0 = va[h], a1 = va[kBlocks / 2 + h], z0 = vz[h], z1 = vz[kBlocks / 2 + h];
            const uint32_t ae = (a0 & 0x0F0F0F0Fu) | ((a1 << 4) & 0xF0F0F0F0u), ao = ((a0 >> 4) & 0x0F0F0F0Fu) | (a1 & 0xF0F0F0F0u);
            const uint32_t ze = (z0 & 0x0F0F0F0Fu) | ((z1 << 4) & 0xF0F0F0F0u), zo = ((z0 >> 4) & 0x0F0F0F0Fu) | (z1 & 0xF0F0F0F0u);
            const uint32_t ea[4] = {e2m1x2_to_f16x2<0>(ae), e2m1x2_to_f16x2<1>(ae), e2m1x2_to_f16x2<2>(ae), e2m1x2_to_f16x2<3>(ae)};
            const uint32_t oa[4] = {e2m1x2_to_f16x2<0>(ao), e2m1x2_to_f16x2<1>(ao), e2m1x2_to_f16x2<2>(ao), e2m1x2_to_f16x2<3>(ao)};
            const uint32_t ez[4] = {e2m1x2_to_f16x2<0>(ze), e2m1x2_to_f16x2<1>(ze), e2m1x2_to_f16x2<2>(ze), e2m1x2_to_f16x2<3>(ze)};
            const uint32_t oz[4] = {e2m1x2_to_f16x2<0>(zo), e2m1x2_to_f16x2<1>(zo), e2m1x2_to_f16x2<2>(zo), e2m1x2_to_f16x2<3>(zo)};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = 2 * h + y;
                // f16 2^(e - vref) of two tokens: exponent field e - vref + 15, 0 below it
                const uint32_t x0 = __viaddmin_s16x2_relu(vs0[j], k2, 0x000F000Fu) << 10;
                const uint32_t x1 = __viaddmin_s16x2_relu(vs1[j], k2, 0x000F000Fu) << 10;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const __half2 b0 = __hmul2(*reinterpret_cast<const __half2*>(&pt0[n]), *reinterpret_cast<const __half2*>(&x0));
                    const __half2 b1 = __hmul2(*reinterpret_cast<const __half2*>(&pt1[n]), *reinterpret_cast<const __half2*>(&x1));
                    const uint32_t u0 = *reinterpret_cast<const uint32_t*>(&b0), u1 = *reinterpret_cast<const uint32_t*>(&b1);
                    mma_f16_16x8x16(o[n][2 * j], ea[2 * y], oa[2 * y], ez[2 * y], oz[2 * y], u0, u1);
                    mma_f16_16x8x16(o[n][2 * j + 1], ea[2 * y + 1], oa[2 * y + 1], ez[2 * y + 1], oz[2 * y + 1], u0, u1);
                }
            }
        }
    }
    cp_async_wait<0>();

    // join the warps, one n-tile (8 rows) at a time: warp w's sums of row r at joined[w][r][..]
    float* joined = reinterpret_cast<float*>(dynamic_smem);
    const int64_t units = static_cast<int64_t>(p.B) * p.Hk * p.row_tiles;
    const int64_t unit = bh * p.row_tiles + rt;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (8 * n >= nrows) break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = sum[n][e];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
            if (g == 0) ml_s[warp][2 * c + e] = make_float2(bound[n][e] == -INFINITY ? -INFINITY : ref[n][e], t);
#pragma unroll
            for (int j = 0; j < 2 * kBlocks; ++j) {
                float* row = joined + (warp * 8 + 2 * c + e) * D + 16 * j + 4 * g - (j & 1) * 14;
                row[0] = o[n][j][e], row[1] = o[n][j][2 + e];
            }
        }
        if (lane == 0) vref_s[warp] = vref ? __uint_as_float(static_cast<uint32_t>(vref) << 23) : 0.0f;
        __syncthreads();
        constexpr int kAtOnce = kFewThreads / D;
        const int d = threadIdx.x % D;
#pragma unroll
        for (int r1 = 0; r1 < 8; r1 += kAtOnce) {
            const int r = r1 + threadIdx.x / D;  // uniform over a warp
            if (8 * n + r >= nrows) continue;
            float m = -INFINITY, total = 0.0f, x = 0.0f, w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, ml_s[k][r].x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = ml_s[k][r].x == -INFINITY ? 0.0f : exp2_approx(ml_s[k][r].x - m);
                total += w[k] * ml_s[k][r].y;
            }
            const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // divided first: the sums times a large scale might not fit
                if (w[k] != 0.0f) x += joined[(k * 8 + r) * D + d] * (w[k] * inv) * vref_s[k];
            if (p.splits > 1) {
                const int64_t at = (split * units + unit) * p.tile_rows + 8 * n + r;
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
}

// Joins the parts of a row: one warp per (sequence, query, head).
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
    const Sequence s = sequence_of(p, b);
    if (qi >= s.nq) return;
    const int kvh = h / p.G, r = qi * p.G + h - kvh * p.G;
    const int rt = r / p.tile_rows, r0 = rt * p.tile_rows;
    const Part part = part_of(p, span_of(p, s, r0, min(p.tile_rows, s.nq * p.G - r0)), shift, 0);
    const int64_t stride = static_cast<int64_t>(p.B) * p.Hk * p.row_tiles * p.tile_rows;
    const int64_t at = ((static_cast<int64_t>(b) * p.Hk + kvh) * p.row_tiles + rt) * p.tile_rows + (r - r0);
    float m = -INFINITY;
    for (int k = lane; k < part.parts; k += 32) m = fmaxf(m, p.part_ml[k * stride + at].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    float total = 0.0f, o[kElems] = {};
    for (int k = 0; k < part.parts; ++k) {
        const float2 ml = p.part_ml[k * stride + at];
        const float w = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - m) * ml.y;
        if (w == 0.0f) continue;
        total += w;
        const float* src = p.part_o + (k * stride + at) * D + kElems * lane;
#pragma unroll
        for (int j = 0; j < kElems; ++j) o[j] += w * src[j];
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

// How a call is split, from what the host knows (not the sequences' lengths).
struct AttendPlan {
    int tile_rows, row_tiles, splits;
    int64_t units;
    size_t bytes;
};
static AttendPlan plan_attend(int64_t B, int Hq, int Hk, int D, int64_t max_q) {
    AttendPlan a;
    const int64_t rows = max_q * (Hq / Hk);
    a.tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
    a.row_tiles = static_cast<int>((rows + a.tile_rows - 1) / a.tile_rows);
    a.units = B * Hk * a.row_tiles;
    const int64_t wanted = static_cast<int64_t>(sm_count()) * 8;
    a.splits = static_cast<int>(a.units >= wanted ? 1 : (wanted + a.units - 1) / a.units);
    if (a.splits > 64) a.splits = 64;
    const size_t rows_all = static_cast<size_t>(a.splits) * a.units * a.tile_rows;
    a.bytes = a.splits > 1 ? rows_all * (static_cast<size_t>(D) * 4 + 8) : 0;
    a.bytes = (a.bytes + 255) / 256 * 256 + 256;
    return a;
}

template <int D, int NT>
static int launch_few(const AttendParams& p, unsigned blocks, cudaStream_t stream) {
    constexpr size_t kRing = 4 * kStages * Strip<D>::kBytes, kJoin = 4 * 8 * D * sizeof(float);
    constexpr size_t kSmem = kRing > kJoin ? kRing : kJoin;
    static_assert(kSmem + sizeof(__half) * 8 * NT * (D + 8) + 1024 <= 48 * 1024, "within the default limit");
    return launch_dependent_smem(attend_few_kernel<D, NT>, dim3(blocks), kFewThreads, kSmem, stream, p);
}

template <int D>
static int launch_attend(const AttendParams& p, int64_t units, cudaStream_t stream) {
    const int64_t blocks = units * p.splits;
    const int64_t join = (static_cast<int64_t>(p.B) * p.max_q * p.Hq + 3) / 4;
    if (blocks > kMaxDim || join > kMaxDim) return MACAQ_ESHAPE;
    const auto n = static_cast<unsigned>(blocks);
    const int st = p.tile_rows == 8    ? launch_few<D, 1>(p, n, stream)
                   : p.tile_rows == 16 ? launch_few<D, 2>(p, n, stream)
                                       : launch_few<D, 4>(p, n, stream);
    if (st != MACAQ_OK || p.splits == 1) return st;
    return launch_dependent(attend_join_kernel<D>, dim3(static_cast<unsigned>(join)), 128, stream, p, 4);
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
        table_width > kMaxDim / page_size || ldq < static_cast<int64_t>(Hq) * head_dim || ldq > kMaxDim || ldq % 8 != 0 ||
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
    p.tile_rows = plan.tile_rows, p.row_tiles = plan.row_tiles, p.splits = plan.splits;
    // no more parts than a full table gives
    const int64_t most = (table_width * page_size + kMinKeys - 1) / kMinKeys;
    if (p.splits > most) p.splits = static_cast<int>(most > 1 ? most : 1);
    p.part_ml = static_cast<float2*>(workspace);
    p.part_o = reinterpret_cast<float*>(p.part_ml + static_cast<int64_t>(p.splits) * plan.units * p.tile_rows);
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_attend<64>(p, plan.units, s) : launch_attend<128>(p, plan.units, s);
}
