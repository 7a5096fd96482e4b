// attend.cu -- attention over the paged MXFP4 cache (layout and masks: include/macaq.h).
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the keys a row's mask leaves (none: o_h = 0)
//
// K and V are held as codes of FWHT32(x c0), c0 = 1/sqrt(32).  The transform is orthogonal, so the
// scores are taken between the transformed query and the codes' values, and the weighted sum of V
// codes is transformed back once per output row: no key or value is ever transformed back.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "sm100.cuh"

namespace macaq {

constexpr float kLog2e = 1.4426950408889634f;

struct AttendParams {
    const uint16_t* q;  // bf16 [T][ldq]
    int64_t T, ldq;
    int Hq, Hk;
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
    int64_t window;    // 0: none
    uint16_t* out;     // bf16 [T][Hq][D]
    float* lse;        // fp32 [T][Hq] or null
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

// One warp per (query row, query head); lane l holds element l of every 32-element block.
template <int D>
__global__ void __launch_bounds__(128) attend_rows_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kBlocks = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    const int l = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int64_t t = item / p.Hq;
    const int h = static_cast<int>(item - t * p.Hq);
    if (t >= p.T) return;
    int b = static_cast<int>(t);
    if (p.cu_q) {  // the last sequence that begins at or before row t
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu_q[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
    }
    const Sequence s = sequence_of(p, b);
    if (t < s.row0 || t >= s.row0 + s.nq) return;
    const int kvh = h / (p.Hq / p.Hk);
    float q[kBlocks], o[kBlocks];
    const uint16_t* qp = p.q + t * p.ldq + static_cast<int64_t>(h) * D;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        float x = __uint_as_float(static_cast<uint32_t>(qp[32 * i + l]) << 16) * kHadamardNorm;
#pragma unroll
        for (int o2 = 1; o2 < 32; o2 <<= 1) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, x, o2);
            x = l & o2 ? y - x : x + y;
        }
        q[i] = x;
        o[i] = 0.0f;
    }
    const int64_t pos = s.pos0 + (t - s.row0);
    const int64_t first = p.window && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    const PageLayout<D> lay{p.page_size};
    float m = -INFINITY, sum = 0.0f;
    for (int64_t j = first; j <= pos; ++j) {
        const int64_t pg = p.tables[b * p.table_width + (j >> p.page_shift)];
        if (pg < 0 || pg >= p.num_pages) {
            report_index();
            continue;
        }
        const uint8_t* page = p.cache + (pg * p.Hk + kvh) * lay.bytes();
        const int at = static_cast<int>(j & (p.page_size - 1));
        float dot = 0.0f, v[kBlocks];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const uint32_t kb = page[at * lay.kRow + (l / 8) * 4 * kBlocks + 4 * i + (l % 8) / 2];
            const uint32_t vb = page[lay.v_codes() + (at >> 1) * D + (l / 4) * 4 * kBlocks + (at & 1) * 2 * kBlocks +
                                     2 * i + (l % 4) / 2];
            const uint32_t ke = page[lay.k_scales() + at * kBlocks + i], ve = page[lay.v_scales() + at * kBlocks + i];
            float kf[8], vf[8];
            decode_e2m1x8((l & 1 ? kb >> 4 : kb) & 15, kf);
            decode_e2m1x8((l & 1 ? vb >> 4 : vb) & 15, vf);
            dot += q[i] * kf[0] * __uint_as_float(ke << 23);
            v[i] = vf[0] * __uint_as_float(ve << 23);
        }
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o2);
        dot *= p.scale_log2;
        const float mn = fmaxf(m, dot);
        const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), e = exp2f(dot - mn);
        m = mn;
        sum = sum * f + e;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) o[i] = o[i] * f + e * v[i];
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    uint16_t* op = p.out + (t * p.Hq + h) * D;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        float x = o[i] * (inv * kHadamardNorm);
#pragma unroll
        for (int o2 = 1; o2 < 32; o2 <<= 1) {
            const float y = __shfl_xor_sync(0xFFFFFFFFu, x, o2);
            x = l & o2 ? y - x : x + y;
        }
        op[32 * i + l] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    if (p.lse && l == 0) p.lse[t * p.Hq + h] = sum > 0.0f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace macaq

extern "C" size_t macaq_kv4_attention_workspace_bytes(int64_t T, int64_t B, int Hq, int Hk, int head_dim, int64_t max_q) {
    if (!head_dim_ok(head_dim) || T < 0 || T > kMaxDim || B < 0 || B > kMaxDim || Hk < 1 || Hq < Hk || Hq > kMaxHeads ||
        Hq % Hk != 0 || max_q < 1 || max_q > kMaxDim)
        return 0;
    return 256;
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
    AttendParams p = {};
    p.q = q, p.T = T, p.ldq = ldq, p.Hq = Hq, p.Hk = Hk, p.cache = cache, p.num_pages = num_pages;
    p.page_size = page_size, p.page_shift = __builtin_ctz(page_size), p.tables = tables, p.table_width = table_width;
    p.kv_lens = kv_lens, p.cu_q = cu_q, p.B = static_cast<int>(B), p.max_q = static_cast<int>(max_q);
    p.scale_log2 = scale * kLog2e, p.window = window, p.out = out, p.lse = lse;
    const auto s = static_cast<cudaStream_t>(stream);
    const int64_t blocks = (T * Hq + 3) / 4;
    if (blocks > kMaxDim) return MACAQ_ESHAPE;
    const dim3 grid(static_cast<unsigned>(blocks));
    return head_dim == 64 ? launch_dependent(attend_rows_kernel<64>, grid, 128, s, p)
                          : launch_dependent(attend_rows_kernel<128>, grid, 128, s, p);
}
