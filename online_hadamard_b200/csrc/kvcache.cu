// kvcache.cu -- norms and rotation of query and key heads, and the paged MXFP4 key/value cache:
// appending to it and reading tokens back (the layout is documented in include/macaq.h).
//
//   head norm   y_d = fl(fl(x_d r) w_d), r = 1 / sqrt(mean_d x_d^2 + eps)
//   rotation    (y_i, y_j) -> (y_i c - y_j s, y_j c + y_i s) for the pairs of the first R elements
//   cache       MXFP4 (the E8M0 and E2M1 rules of quant.cu) of the unnormalised 32-point
//               Walsh-Hadamard transform of fl(y_d c0), c0 = fl32(1 / sqrt(32))
//
// Everything is fp32.  What reaches the cache runs in one canonical order, one rounding per operation (the sum of
// squares adds neighbours first: distances 1, 2, 4, ..), so its codes are reproducible bit for bit.  The bf16 outputs
// are rounded once, from fp32 that sums in the order of its threads and fuses multiplications with additions: the keys
// of macaq_qk_norm_rope and those that macaq_kv4_append quantises may differ in the last bits of fp32.
//
// Work split.  Query heads (and the key heads of macaq_qk_norm_rope): D / 8 lanes own one head, lane
// l its elements 4l .. 4l+3 of each half, so the pairs (i, i + D/2) meet in one thread and a head's
// halves are loaded in contiguous 8-byte pieces; a unit walks several heads of one token with the
// token's angles and the weights in registers.  Key and value heads bound for the cache: one thread
// owns one 32-element block, so the whole transform and quantisation runs in its registers as in
// quant.cu; the D / 32 threads of a head exchange their sums of squares and code words by shuffles.
// Both are bound by the bytes of the rows (2 B an element in and out, 17/32 B into the cache).  4096 rows of
// 64 + 8 heads of 128, device time of a call in a captured graph: norm and rotation 29.5 us (5.2 TB/s; the public call
// takes as long), with 8 value heads and the cache 37.7 us (4.2 TB/s: the threads of the cache's blocks read and
// transform 64 bytes each, 1000 instructions), reading back 7.0 us (13.5 with the host's call).
// 64 registers a thread: at 78 the append takes 40 us (30 % of the warps resident), at 48 43 us (spills).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "sm100.cuh"

namespace macaq {

constexpr int kHeadThreads = 128;
constexpr float kHadamardNorm = 0.17677669529663687f;  // fl32(1 / sqrt(32))

// Records a device-side index (position, slot, page) that was out of range and skipped.
__device__ __forceinline__ void report_index() { atomicExch(&g_device_status, MACAQ_EINDEX); }

enum class RopeMode { kNone = 0, kHalf = 1, kHalfPart = 2, kPair = 3 };

// The rows of a stacked projection and what is applied to their heads.
struct HeadParams {
    const uint16_t* qkv;  // bf16 [T][ld]: Hq query heads, Hk key heads (and, for the cache, Hk value heads)
    int64_t T, ld;
    int Hq, Hk;
    const float* wq;  // fp32 [D] or null
    const float* wk;
    float eps;
    const float* rope;  // fp32 [rope_rows][R]: R/2 cosines, then R/2 sines
    int64_t rope_rows;
    int R;
    const int64_t* positions;
    uint16_t* q;  // bf16 [T][Hq][D]
    uint16_t* k;  // bf16 [T][Hk][D] (macaq_qk_norm_rope)
    int heads_per_unit, q_chunks, k_chunks;  // units of a token: q_chunks, then k_chunks
    uint8_t* cache;
    int64_t num_pages;
    int page_size;
    const int64_t* slots;
    int64_t head_blocks;   // CTAs of the head units
    int64_t cache_blocks;  // CTAs of the cache's blocks, which come first: theirs is the longer work
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// One unit (D / 8 lanes): heads [0, n) at src (contiguous), to dst.
template <int D, RopeMode MODE>
__device__ __forceinline__ void head_unit(const uint16_t* src, uint16_t* dst, int n, const float* w, float eps,
                                          const float* trow, int R, int l) {
    constexpr int kLanes = D / 8;
    float wl[4], wh[4], c[4], s[4];
    const bool norm = w != nullptr;
    if (norm) {
        const float4 a = *reinterpret_cast<const float4*>(w + 4 * l);
        const float4 b = *reinterpret_cast<const float4*>(w + D / 2 + 4 * l);
        wl[0] = a.x, wl[1] = a.y, wl[2] = a.z, wl[3] = a.w;
        wh[0] = b.x, wh[1] = b.y, wh[2] = b.z, wh[3] = b.w;
    }
    if constexpr (MODE == RopeMode::kHalf || MODE == RopeMode::kHalfPart) {
        const int i = MODE == RopeMode::kHalf ? 4 * l : 4 * (l % (kLanes / 2));
        const float4 a = *reinterpret_cast<const float4*>(trow + i);
        const float4 b = *reinterpret_cast<const float4*>(trow + R / 2 + i);
        c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
        s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    }
    if constexpr (MODE == RopeMode::kPair) {  // two angles of the low half, two of the high half
        const float2 a = *reinterpret_cast<const float2*>(trow + 2 * l);
        const float2 b = *reinterpret_cast<const float2*>(trow + R / 2 + 2 * l);
        c[0] = a.x, c[1] = a.y, s[0] = b.x, s[1] = b.y;
        c[2] = c[3] = 1.0f, s[2] = s[3] = 0.0f;
        if (R == D) {
            const float2 d = *reinterpret_cast<const float2*>(trow + D / 4 + 2 * l);
            const float2 e = *reinterpret_cast<const float2*>(trow + R / 2 + D / 4 + 2 * l);
            c[2] = d.x, c[3] = d.y, s[2] = e.x, s[3] = e.y;
        }
    }
    constexpr int kAhead = 4;
    for (int h0 = 0; h0 < n; h0 += kAhead) {
        uint2 lo[kAhead], hi[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h0 + u < n) {
                const uint16_t* p = src + (h0 + u) * D + 4 * l;
                lo[u] = *reinterpret_cast<const uint2*>(p);
                hi[u] = *reinterpret_cast<const uint2*>(p + D / 2);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h0 + u >= n) break;  // uniform over the unit's lanes
            float a[4] = {bf_lo(lo[u].x), bf_hi(lo[u].x), bf_lo(lo[u].y), bf_hi(lo[u].y)};
            float b[4] = {bf_lo(hi[u].x), bf_hi(hi[u].x), bf_lo(hi[u].y), bf_hi(hi[u].y)};
            const unsigned unit = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << kLanes) - 1u))
                                  << ((threadIdx.x & 31) / kLanes * kLanes);
            if (norm) {
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) t += a[i] * a[i] + b[i] * b[i];
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(unit, t, o);
                const float r = __fdiv_rn(1.0f, __fsqrt_rn(t * (1.0f / D) + eps));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = a[i] * r * wl[i];
                    b[i] = b[i] * r * wh[i];
                }
            }
            if constexpr (MODE == RopeMode::kHalf) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = a[i], y = b[i];
                    a[i] = x * c[i] - y * s[i];
                    b[i] = y * c[i] + x * s[i];
                }
            }
            if constexpr (MODE == RopeMode::kHalfPart) {  // pairs (i, i + D/4) of the low half
                const float sign = l < kLanes / 2 ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float o = __shfl_xor_sync(unit, a[i], kLanes / 2);
                    a[i] = a[i] * c[i] + sign * o * s[i];
                }
            }
            if constexpr (MODE == RopeMode::kPair) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = a[2 * i], y = a[2 * i + 1];
                    a[2 * i] = x * c[i] - y * s[i];
                    a[2 * i + 1] = y * c[i] + x * s[i];
                    const float z = b[2 * i], v = b[2 * i + 1];
                    b[2 * i] = z * c[2 + i] - v * s[2 + i];
                    b[2 * i + 1] = v * c[2 + i] + z * s[2 + i];
                }
            }
            uint16_t* o = dst + (h0 + u) * D + 4 * l;
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
            *reinterpret_cast<uint2*>(o + D / 2) = make_uint2(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]));
        }
    }
}

// The angles of token t, or null where its position is outside the table (reported by the caller).
__device__ __forceinline__ const float* angles_of(const HeadParams& p, int64_t t, bool& ok) {
    if (!p.rope) return nullptr;
    const int64_t pos = p.positions[t];
    ok = pos >= 0 && pos < p.rope_rows;
    return p.rope + (ok ? pos : 0) * p.R;
}

template <int D, RopeMode MODE>
__device__ __forceinline__ void run_head_units(const HeadParams& p, int64_t block) {
    constexpr int kLanes = D / 8;
    const int l = threadIdx.x % kLanes;
    const int64_t unit = (block * kHeadThreads + threadIdx.x) / kLanes;
    const int per_token = p.q_chunks + p.k_chunks;
    const int64_t t = unit / per_token;
    if (t >= p.T) return;
    bool ok = true;
    const float* trow = angles_of(p, t, ok);
    const bool padding = !ok && p.slots && p.slots[t] < 0;  // any position will do there: zeros
    if (!ok && !padding) {
        report_index();
        return;
    }
    int chunk = static_cast<int>(unit - t * per_token);
    const bool is_k = chunk >= p.q_chunks;
    if (is_k) chunk -= p.q_chunks;
    const int heads = is_k ? p.Hk : p.Hq;
    const int h0 = chunk * p.heads_per_unit;
    const int n = min(p.heads_per_unit, heads - h0);
    const uint16_t* src = p.qkv + t * p.ld + static_cast<int64_t>((is_k ? p.Hq : 0) + h0) * D;
    uint16_t* dst = (is_k ? p.k : p.q) + (t * heads + h0) * D;
    if (padding) {
        for (int i = l; i < n * (D / 8); i += kLanes) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    head_unit<D, MODE>(src, dst, n, is_k ? p.wk : p.wq, p.eps, trow, p.R, l);
}

// ------------------------------------------------------------------------------ cache blocks

// Byte offsets inside one (page, kv head) of the cache (include/macaq.h).
template <int D>
struct PageLayout {
    static constexpr int kBlocks = D / 32;
    static constexpr int kRow = D / 2;  // code bytes of a token
    int page;
    __device__ __forceinline__ int64_t bytes() const { return static_cast<int64_t>(page) * D * 17 / 16; }
    __device__ __forceinline__ int v_codes() const { return page * kRow; }
    __device__ __forceinline__ int k_scales() const { return 2 * page * kRow; }
    __device__ __forceinline__ int v_scales() const { return 2 * page * kRow + page * kBlocks; }
};

__device__ __forceinline__ void load32(const uint16_t* p, uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * j);
        w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    }
}

// Element i of 32 bf16 in 16 words (i a compile-time constant after unrolling).
__device__ __forceinline__ float elem(const uint32_t (&w)[16], int i) {
    return i & 1 ? bf_hi(w[i >> 1]) : bf_lo(w[i >> 1]);
}

// The sum of 32 values, neighbours first.
__device__ __forceinline__ float sum_squares32(const uint32_t (&w)[16]) {
    float s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = bf_lo(w[i]), b = bf_hi(w[i]);
        s[i] = __fadd_rn(__fmul_rn(a, a), __fmul_rn(b, b));
    }
#pragma unroll
    for (int n = 8; n > 0; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] = __fadd_rn(s[2 * i], s[2 * i + 1]);
    return s[0];
}

// Block b (32 elements) of one key head, normed and rotated, in the canonical order.
template <int D>
__device__ __forceinline__ void key_block(const HeadParams& p, const uint16_t* head, int b, const float* trow,
                                          unsigned row_mask, bool interleaved, float2 (&u)[16]) {
    constexpr int kBlocks = D / 32;
    uint32_t w[16];
    load32(head + 32 * b, w);
    float* y = reinterpret_cast<float*>(u);
    float r = 1.0f;
    const bool norm = p.wk != nullptr;
    if (norm) {
        float t = sum_squares32(w);
#pragma unroll
        for (int o = 1; o < kBlocks; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(row_mask, t, o));
        r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(t, 1.0f / D), p.eps)));
    }
    const float* wt = p.wk + 32 * b;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float x = elem(w, i);
        y[i] = norm ? __fmul_rn(__fmul_rn(x, r), wt[i]) : x;
    }
    if (!trow || 32 * b >= p.R) return;
    const float* cs = trow;
    const float* sn = trow + p.R / 2;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float c = cs[16 * b + i], s = sn[16 * b + i], x = y[2 * i], z = y[2 * i + 1];
            y[2 * i] = __fsub_rn(__fmul_rn(x, c), __fmul_rn(z, s));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(z, c), __fmul_rn(x, s));
        }
    } else if (p.R == 32) {  // both halves of the pairs in this block
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float c = cs[i], s = sn[i], x = y[i], z = y[i + 16];
            y[i] = __fsub_rn(__fmul_rn(x, c), __fmul_rn(z, s));
            y[i + 16] = __fadd_rn(__fmul_rn(z, c), __fmul_rn(x, s));
        }
    } else {  // the other halves are block b +- R/64
        const int step = p.R / 64;
        const bool low = b < step;
        const int ob = low ? b + step : b - step;
        load32(head + 32 * ob, w);
        const float* ow = p.wk + 32 * ob;
        const int a0 = 32 * (low ? b : ob);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = elem(w, i);
            const float o = norm ? __fmul_rn(__fmul_rn(x, r), ow[i]) : x;
            const float os = __fmul_rn(o, sn[a0 + i]), yc = __fmul_rn(y[i], cs[a0 + i]);
            y[i] = low ? __fsub_rn(yc, os) : __fadd_rn(yc, os);
        }
    }
}

// Exchanges code words between the kBlocks threads of one head so that each ends with whole
// stretches of the row.  In: word c of block b in thread b (c = 0..3).  Out, kBlocks = 4: thread i
// holds (c = i; b = 0..3).  kBlocks = 2: thread i holds (c = 2i; b = 0, 1), (c = 2i + 1; b = 0, 1).
template <int NB>
__device__ __forceinline__ uint4 transpose_words(uint4 w, int b, unsigned mask) {
    // words c and c + 2 between threads whose index differs in the top bit, then c and c + 1
    const int top = NB / 2;
    const bool up = (b & top) != 0;
    uint32_t g0 = up ? w.x : w.z, g1 = up ? w.y : w.w;  // given away
    g0 = __shfl_xor_sync(mask, g0, top);
    g1 = __shfl_xor_sync(mask, g1, top);
    // kept words c0, c0 + 1 (c0 = 0 or 2) of this thread's block and of the partner's
    const uint32_t k0 = up ? w.z : w.x, k1 = up ? w.w : w.y;
    const uint32_t lo0 = up ? g0 : k0, lo1 = up ? g1 : k1;  // of the lower of the two blocks
    const uint32_t hi0 = up ? k0 : g0, hi1 = up ? k1 : g1;
    if constexpr (NB == 2) return make_uint4(lo0, hi0, lo1, hi1);
    const bool odd = (b & 1) != 0;
    uint32_t a0 = odd ? lo0 : lo1, a1 = odd ? hi0 : hi1;
    a0 = __shfl_xor_sync(mask, a0, 1);
    a1 = __shfl_xor_sync(mask, a1, 1);
    const uint32_t m0 = odd ? lo1 : lo0, m1 = odd ? hi1 : hi0;
    // even thread: blocks (0|2 mine, 1|3 partner's); m0/a0 belong to blocks 0, 1 and m1/a1 to 2, 3
    return odd ? make_uint4(a0, m0, a1, m1) : make_uint4(m0, a0, m1, a1);
}

// The inverse of transpose_words (it is its own inverse up to the order of the words).
template <int NB>
__device__ __forceinline__ uint4 untranspose_words(uint4 w, int b, unsigned mask) {
    if constexpr (NB == 4) return transpose_words<4>(w, b, mask);
    const bool up = b != 0;  // thread i holds (c = 2i; b = 0, 1), (c = 2i + 1; b = 0, 1)
    uint32_t g0 = up ? w.x : w.y, g1 = up ? w.z : w.w;
    g0 = __shfl_xor_sync(mask, g0, 1);
    g1 = __shfl_xor_sync(mask, g1, 1);
    return up ? make_uint4(g0, g1, w.y, w.w) : make_uint4(w.x, w.z, g0, g1);
}

// One thread per (token, K or V, kv head, 32-element block), blocks fastest.
template <int D>
__device__ __forceinline__ void run_cache_blocks(const HeadParams& p, int64_t block, bool interleaved) {
    constexpr int kBlocks = D / 32;
    const int64_t item = block * kHeadThreads + threadIdx.x;
    const int b = static_cast<int>(item % kBlocks);
    int64_t rest = item / kBlocks;
    const int h = static_cast<int>(rest % p.Hk);
    rest /= p.Hk;
    const bool is_v = rest & 1;
    const int64_t t = rest >> 1;
    if (t >= p.T) return;  // whole heads leave together
    const unsigned mask = ((1u << kBlocks) - 1u) << ((threadIdx.x & 31) / kBlocks * kBlocks);
    const int64_t slot = p.slots[t];
    if (slot < 0) return;  // padding row
    bool ok = true;
    const float* trow = angles_of(p, t, ok);
    const int64_t pg = slot / p.page_size;
    if (!ok || pg >= p.num_pages) {
        report_index();
        return;
    }
    const int at = static_cast<int>(slot - pg * p.page_size);
    const PageLayout<D> lay{p.page_size};
    uint8_t* page = p.cache + (pg * p.Hk + h) * lay.bytes();
    const uint16_t* head = p.qkv + t * p.ld + static_cast<int64_t>(p.Hq + (is_v ? p.Hk : 0) + h) * D;
    float2 u[16];
    if (!is_v) {
        key_block<D>(p, head, b, trow, mask, interleaved, u);
    } else {
        uint32_t w[16];
        load32(head + 32 * b, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = make_float2(bf_lo(w[i]), bf_hi(w[i]));
    }
    float2 m[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i] = make_float2(kHadamardNorm, kHadamardNorm);
    scale_fwht32(u, m);
    uint4 c;
    const uint32_t e = quantize32(u, c);
    c = transpose_words<kBlocks>(c, b, mask);
    if (!is_v) {
        *reinterpret_cast<uint4*>(page + at * lay.kRow + 16 * b) = c;
        page[lay.k_scales() + at * kBlocks + b] = static_cast<uint8_t>(e);
    } else {
        // a word's low half is g = 2c, its high half g = 2c + 1
        uint8_t* pair = page + lay.v_codes() + (at >> 1) * D + (at & 1) * 2 * kBlocks;
        if constexpr (kBlocks == 4) {
            *reinterpret_cast<uint2*>(pair + (2 * b) * 16) =
                make_uint2(__byte_perm(c.x, c.y, 0x5410), __byte_perm(c.z, c.w, 0x5410));
            *reinterpret_cast<uint2*>(pair + (2 * b + 1) * 16) =
                make_uint2(__byte_perm(c.x, c.y, 0x7632), __byte_perm(c.z, c.w, 0x7632));
        } else {
            *reinterpret_cast<uint32_t*>(pair + (4 * b) * 8) = __byte_perm(c.x, c.y, 0x5410);
            *reinterpret_cast<uint32_t*>(pair + (4 * b + 1) * 8) = __byte_perm(c.x, c.y, 0x7632);
            *reinterpret_cast<uint32_t*>(pair + (4 * b + 2) * 8) = __byte_perm(c.z, c.w, 0x5410);
            *reinterpret_cast<uint32_t*>(pair + (4 * b + 3) * 8) = __byte_perm(c.z, c.w, 0x7632);
        }
        page[lay.v_scales() + at * kBlocks + b] = static_cast<uint8_t>(e);
    }
}

template <int D, RopeMode MODE, bool CACHE>
__global__ void __launch_bounds__(kHeadThreads, 8) heads_kernel(const __grid_constant__ HeadParams p) {
    griddep_wait();  // the rows may be written, and the outputs read, by the preceding kernel
    griddep_launch_dependents();  // (behind the wait: attend.cu says why)
    if constexpr (CACHE) {
        if (blockIdx.x < p.cache_blocks) {
            run_cache_blocks<D>(p, blockIdx.x, MODE == RopeMode::kPair);
            return;
        }
    }
    run_head_units<D, MODE>(p, blockIdx.x - p.cache_blocks);
}

// Eight E2M1 codes of a word (element j in nibble j) as floats.
__device__ __forceinline__ void decode_e2m1x8(uint32_t w, float* f) {
    uint32_t h[4];
    e2m1x8_to_f16(w, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        f[2 * j] = v.x, f[2 * j + 1] = v.y;
    }
}

// Reads tokens back: one thread per (token, K or V, kv head, block); bf16(FWHT32(codes) c0).
template <int D>
__global__ void __launch_bounds__(kHeadThreads) kv4_gather_kernel(const uint8_t* cache, int64_t num_pages,
                                                                  int page_size, int Hk, const int64_t* slots,
                                                                  int64_t T, uint16_t* k, uint16_t* v) {
    constexpr int kBlocks = D / 32;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kHeadThreads + threadIdx.x;
    const int b = static_cast<int>(item % kBlocks);
    int64_t rest = item / kBlocks;
    const int h = static_cast<int>(rest % Hk);
    rest /= Hk;
    const bool is_v = rest & 1;
    const int64_t t = rest >> 1;
    if (t >= T) return;
    const unsigned mask = ((1u << kBlocks) - 1u) << ((threadIdx.x & 31) / kBlocks * kBlocks);
    uint16_t* out = (is_v ? v : k) + (t * Hk + h) * D + 32 * b;
    const int64_t slot = slots[t];
    const int64_t pg = slot < 0 ? 0 : slot / page_size;
    if (slot < 0 || pg >= num_pages) {
        if (slot >= 0) report_index();
#pragma unroll
        for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(out)[j] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int at = static_cast<int>(slot - pg * page_size);
    const PageLayout<D> lay{page_size};
    const uint8_t* page = cache + (pg * Hk + h) * lay.bytes();
    uint4 c;
    uint32_t e;
    if (!is_v) {
        c = *reinterpret_cast<const uint4*>(page + at * lay.kRow + 16 * b);
        e = page[lay.k_scales() + at * kBlocks + b];
    } else {
        const uint8_t* pair = page + lay.v_codes() + (at >> 1) * D + (at & 1) * 2 * kBlocks;
        if constexpr (kBlocks == 4) {
            const uint2 lo = *reinterpret_cast<const uint2*>(pair + (2 * b) * 16);
            const uint2 hi = *reinterpret_cast<const uint2*>(pair + (2 * b + 1) * 16);
            c = make_uint4(__byte_perm(lo.x, hi.x, 0x5410), __byte_perm(lo.x, hi.x, 0x7632),
                           __byte_perm(lo.y, hi.y, 0x5410), __byte_perm(lo.y, hi.y, 0x7632));
        } else {
            const uint32_t g0 = *reinterpret_cast<const uint32_t*>(pair + (4 * b) * 8);
            const uint32_t g1 = *reinterpret_cast<const uint32_t*>(pair + (4 * b + 1) * 8);
            const uint32_t g2 = *reinterpret_cast<const uint32_t*>(pair + (4 * b + 2) * 8);
            const uint32_t g3 = *reinterpret_cast<const uint32_t*>(pair + (4 * b + 3) * 8);
            c = make_uint4(__byte_perm(g0, g1, 0x5410), __byte_perm(g0, g1, 0x7632), __byte_perm(g2, g3, 0x5410),
                           __byte_perm(g2, g3, 0x7632));
        }
        e = page[lay.v_scales() + at * kBlocks + b];
    }
    c = untranspose_words<kBlocks>(c, b, mask);
    float2 u[16];
    float* f = reinterpret_cast<float*>(u);
    decode_e2m1x8(c.x, f), decode_e2m1x8(c.y, f + 8), decode_e2m1x8(c.z, f + 16), decode_e2m1x8(c.w, f + 24);
    // 2^(e - 127), exact; e = 0 stands for the subnormal 2^-127
    const float x = e ? __uint_as_float(e << 23) : __uint_as_float(1u << 22);
    float2 m[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i] = make_float2(x, x);
    scale_fwht32(u, m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float* y = f + 8 * j;
        reinterpret_cast<uint4*>(out)[j] = make_uint4(
            pack_bf16(__fmul_rn(y[0], kHadamardNorm), __fmul_rn(y[1], kHadamardNorm)),
            pack_bf16(__fmul_rn(y[2], kHadamardNorm), __fmul_rn(y[3], kHadamardNorm)),
            pack_bf16(__fmul_rn(y[4], kHadamardNorm), __fmul_rn(y[5], kHadamardNorm)),
            pack_bf16(__fmul_rn(y[6], kHadamardNorm), __fmul_rn(y[7], kHadamardNorm)));
    }
}

// ------------------------------------------------------------------------------- host side

inline bool head_dim_ok(int D) { return D == 64 || D == 128; }
inline bool page_size_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
constexpr int kMaxHeads = 1024;

// The checks that both head calls share.  `value_heads`: the rows also hold Hk value heads.
static int check_heads(const HeadParams& p, int D, int64_t rope_dim, bool value_heads) {
    if (!head_dim_ok(D) || p.T < 0 || p.T > kMaxDim || p.Hq < 0 || p.Hk < 0 || p.Hq > kMaxHeads || p.Hk > kMaxHeads)
        return MACAQ_ESHAPE;
    const int64_t width = static_cast<int64_t>(p.Hq + p.Hk * (value_heads ? 2 : 1)) * D;
    if (p.ld < width || p.ld > kMaxDim || p.ld % 8 != 0) return MACAQ_ESHAPE;
    if (!(p.eps >= 0.0f) || std::isinf(p.eps)) return MACAQ_EINVAL;
    if (p.rope) {
        if (rope_dim != D && rope_dim != D / 2) return MACAQ_ESHAPE;
        if (p.rope_rows < 1 || p.rope_rows > kMaxDim) return MACAQ_ESHAPE;
        if (!p.positions) return MACAQ_EINVAL;
    }
    if (!aligned16(p.qkv) || !aligned16(p.wq) || !aligned16(p.wk) || !aligned16(p.rope) || !aligned16(p.q) ||
        !aligned16(p.k) || !aligned16(p.cache) || (reinterpret_cast<uintptr_t>(p.positions) & 7u) ||
        (reinterpret_cast<uintptr_t>(p.slots) & 7u))
        return MACAQ_EALIGN;
    return MACAQ_OK;
}

// Heads per unit: one while the units do not fill the GPU (a step is bound by latency), else enough
// that a token's angles and the weights are loaded once for several heads.
static void split_heads(HeadParams& p, int D, bool with_k) {
    const int64_t rows = p.T * (p.Hq + (with_k ? p.Hk : 0));
    const int64_t resident = static_cast<int64_t>(sm_count()) * 2048 / (D / 8);
    p.heads_per_unit = rows <= resident ? 1 : rows <= 4 * resident ? 4 : 8;
    p.q_chunks = (p.Hq + p.heads_per_unit - 1) / p.heads_per_unit;
    p.k_chunks = with_k ? (p.Hk + p.heads_per_unit - 1) / p.heads_per_unit : 0;
    const int64_t threads = p.T * (p.q_chunks + p.k_chunks) * (D / 8);
    p.head_blocks = (threads + kHeadThreads - 1) / kHeadThreads;
}

template <int D, bool CACHE>
static int launch_heads(const HeadParams& p, int interleaved, int64_t blocks, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(blocks));
    if (!p.rope) return launch_dependent(heads_kernel<D, RopeMode::kNone, CACHE>, grid, kHeadThreads, stream, p);
    if (interleaved) return launch_dependent(heads_kernel<D, RopeMode::kPair, CACHE>, grid, kHeadThreads, stream, p);
    if (p.R == D) return launch_dependent(heads_kernel<D, RopeMode::kHalf, CACHE>, grid, kHeadThreads, stream, p);
    return launch_dependent(heads_kernel<D, RopeMode::kHalfPart, CACHE>, grid, kHeadThreads, stream, p);
}

}  // namespace macaq

using namespace macaq;

extern "C" size_t macaq_kv4_page_bytes(int page_size, int head_dim) {
    if (!page_size_ok(page_size) || !head_dim_ok(head_dim)) return 0;
    return static_cast<size_t>(page_size) * head_dim * 17 / 16;
}

extern "C" int macaq_qk_norm_rope(const uint16_t* qkv, int64_t T, int64_t ld, int Hq, int Hk, int head_dim,
                                  const float* q_weight, const float* k_weight, float eps, const float* rope,
                                  int64_t rope_rows, int rope_dim, int interleaved, const int64_t* positions,
                                  uint16_t* q, uint16_t* k, void* stream) {
    HeadParams p = {};
    p.qkv = qkv, p.T = T, p.ld = ld, p.Hq = Hq, p.Hk = Hk, p.wq = q_weight, p.wk = k_weight, p.eps = eps;
    p.rope = rope, p.rope_rows = rope_rows, p.R = rope_dim, p.positions = positions, p.q = q, p.k = k;
    if (int st = check_heads(p, head_dim, rope_dim, false)) return st;
    if (Hq + Hk < 1) return MACAQ_ESHAPE;
    if (T == 0) return MACAQ_OK;
    if (!qkv || (Hq && !q) || (Hk && !k) || (interleaved & ~1)) return MACAQ_EINVAL;
    split_heads(p, head_dim, true);
    if (p.head_blocks > kMaxDim) return MACAQ_ESHAPE;
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_heads<64, false>(p, interleaved, p.head_blocks, s)
                          : launch_heads<128, false>(p, interleaved, p.head_blocks, s);
}

extern "C" int macaq_kv4_append(const uint16_t* qkv, int64_t T, int64_t ld, int Hq, int Hk, int head_dim,
                                const float* q_weight, const float* k_weight, float eps, const float* rope,
                                int64_t rope_rows, int rope_dim, int interleaved, const int64_t* positions,
                                uint8_t* cache, int64_t num_pages, int page_size, const int64_t* slots, uint16_t* q,
                                void* stream) {
    HeadParams p = {};
    p.qkv = qkv, p.T = T, p.ld = ld, p.Hq = Hq, p.Hk = Hk, p.wq = q_weight, p.wk = k_weight, p.eps = eps;
    p.rope = rope, p.rope_rows = rope_rows, p.R = rope_dim, p.positions = positions, p.q = q;
    p.cache = cache, p.num_pages = num_pages, p.page_size = page_size, p.slots = slots;
    if (int st = check_heads(p, head_dim, rope_dim, true)) return st;
    if (Hk < 1 || !page_size_ok(page_size) || num_pages < 1 || num_pages > kMaxDim) return MACAQ_ESHAPE;
    if (T == 0) return MACAQ_OK;
    if (!qkv || (Hq && !q) || !cache || !slots || (interleaved & ~1)) return MACAQ_EINVAL;
    split_heads(p, head_dim, false);
    const int64_t items = 2 * T * Hk * (head_dim / 32);
    p.cache_blocks = (items + kHeadThreads - 1) / kHeadThreads;
    const int64_t blocks = p.cache_blocks + p.head_blocks;
    if (blocks > kMaxDim) return MACAQ_ESHAPE;
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_heads<64, true>(p, interleaved, blocks, s)
                          : launch_heads<128, true>(p, interleaved, blocks, s);
}

extern "C" int macaq_kv4_gather(const uint8_t* cache, int64_t num_pages, int page_size, int Hk, int head_dim,
                                const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v, void* stream) {
    if (!head_dim_ok(head_dim) || !page_size_ok(page_size) || num_pages < 1 || num_pages > kMaxDim || Hk < 1 ||
        Hk > kMaxHeads || T < 0 || T > kMaxDim)
        return MACAQ_ESHAPE;
    if (T == 0) return MACAQ_OK;
    if (!cache || !slots || !k || !v) return MACAQ_EINVAL;
    if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u))
        return MACAQ_EALIGN;
    const int64_t items = 2 * T * Hk * (head_dim / 32);
    const int64_t blocks = (items + kHeadThreads - 1) / kHeadThreads;
    if (blocks > kMaxDim) return MACAQ_ESHAPE;
    const dim3 grid(static_cast<unsigned>(blocks));
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64
               ? launch_dependent(kv4_gather_kernel<64>, grid, kHeadThreads, s, cache, num_pages, page_size, Hk, slots, T, k, v)
               : launch_dependent(kv4_gather_kernel<128>, grid, kHeadThreads, s, cache, num_pages, page_size, Hk, slots, T, k, v);
}
