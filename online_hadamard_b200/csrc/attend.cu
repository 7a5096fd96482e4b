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
//
// These kernels start before the one ahead of them has ended (launch_dependent), and each lets its own dependents start only
// behind its wait.  So while a kernel is resident and waits, the one ahead is the only other one that runs: all before it
// have ended and their writes are visible, and no line that a kernel further ahead could have read too early comes to an
// SM's L1 after the launch.  What the one ahead writes (queries, codes, parts, notes of cut units) it does not read
// through L1 itself.  Lengths, tables, queries, notes and parts are therefore read by ordinary loads or through L2 alike.
// (Dependents started before the wait would save 0.3 to 0.7 us a call: one sequence of 2047 keys 12.9 against 13.4 us on the
// device.  A fence behind the wait costs as much as this order.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"

namespace macaq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The unit that a CTA's range ends in, if the range holds its beginning but not its end: `parts` CTAs, this one
// and the next, hold it (0: there is none).
struct __align__(16) CutUnit {
    int64_t row0;  // its sequence's first query row
    int r0, nrows, kvh, parts, unused[2];
};

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
    int tile_rows, row_tiles, ctas, unit_cost;
    float* part_o;    // fp32 [ctas][2][tile_rows][D], each row divided by its own sum
    float2* part_ml;  // [ctas][2][tile_rows]: its reference m (base 2) and sum of 2^(s - m)
    CutUnit* cuts;    // [ctas]
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

// A unit is a (sequence, tile of query rows, kv head); its work is its span in blocks of 2^shift keys (one
// block where nothing is seen).
__device__ __forceinline__ int blocks_of(const Span& sp, int shift) {
    return sp.last_hi < 0 ? 1 : (sp.last_hi >> shift) - (sp.first_lo >> shift) + 1;
}
struct Tile {  // of a sequence; nrows <= 0: none
    Sequence s;
    Span sp;
    int b, r0, nrows, blocks;
};
__device__ __forceinline__ Tile tile_of(const AttendParams& p, int64_t item, int shift) {
    Tile t;
    t.b = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(p.row_tiles));  // fewer than 2^31 tiles
    t.r0 = static_cast<int>(item - static_cast<int64_t>(t.b) * p.row_tiles) * p.tile_rows;
    t.s = sequence_of(p, t.b);
    t.nrows = min(p.tile_rows, t.s.nq * p.G - t.r0);
    t.sp = span_of(p, t.s, t.r0, max(t.nrows, 1));
    t.blocks = t.nrows > 0 ? blocks_of(t.sp, shift) : 0;
    return t;
}

// Sequences are of unequal length, known on the device only, and few units leave most of the GPU idle: so
// the blocks of all units stand in one row (tiles, then their kv heads), each unit behind `unit_cost` empty
// places for what starting and ending it costs, and CTA i of the resident ones takes the places [i len,
// (i + 1) len), whatever units they belong to.  A unit that one CTA holds whole is written directly, parts of one
// are joined by attend_join_kernel.  A CTA cuts at most two units: its parts go to slot 0 (the unit that its
// range begins in) and slot 1 (the one it ends in).  No range is shorter than kMinKeys keys (joining would
// cost more than it saves: one sequence of 30000 keys, 7 heads on one, takes 22.5, 17.6 and 16.3 us with 128, 256
// and 512 keys; of 300 keys, 64 heads on 8, 11.7, 12.7 and 15.0 us).
constexpr int kMinKeys = 256;
__device__ __forceinline__ int64_t tile_places(const AttendParams& p, const Tile& t) {
    return t.nrows > 0 ? static_cast<int64_t>(t.blocks + p.unit_cost) * p.Hk : 0;
}
struct Place {  // the tile that a place lies in, and where that tile begins
    int64_t pos, len, total;
    int64_t item, item_pos;
};
struct PlaceShared {
    int64_t scan[32], item, item_pos;
};
// Place i len, by all THREADS threads of a CTA: a thread adds up its share of the tiles, the one whose share
// holds the place walks it.
template <int THREADS>
__device__ __forceinline__ Place find_place(const AttendParams& p, int shift, int64_t i, PlaceShared& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = static_cast<int64_t>(p.B) * p.row_tiles, share = (items + THREADS - 1) / THREADS;
    const int64_t a = min(items, threadIdx.x * share), z = min(items, a + share);
    int64_t mine = 0;
#pragma unroll 1
    for (int64_t x = a; x < z; ++x) mine += tile_places(p, tile_of(p, x, shift));
    int64_t upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, x);
        if (lane >= x) upto += y;
    }
    if (lane == 31) sm.scan[warp] = upto;
    __syncthreads();
    Place c;
    c.total = 0;
#pragma unroll 4
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) upto += sm.scan[w];
        c.total += sm.scan[w];
    }
    const int64_t len = (c.total + p.ctas - 1) / p.ctas;
    c.len = len > (kMinKeys >> shift) ? len : (kMinKeys >> shift);
    c.pos = i * c.len;
    if (c.pos < upto && c.pos >= upto - mine) {
        int64_t at = upto - mine;
#pragma unroll 1
        for (int64_t x = a; x < z; ++x) {
            const int64_t n = tile_places(p, tile_of(p, x, shift));
            if (c.pos < at + n) {
                sm.item = x, sm.item_pos = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    c.item = sm.item, c.item_pos = sm.item_pos;
    return c;
}

// The units of a CTA in order, as parts [begin, end) in block numbers; slot < 0: whole.
struct Unit {
    Tile t;
    int kvh, begin, end;
    int64_t slot;
};
struct Walk {
    int64_t pos, end, item, item_pos, len;
    CutUnit cut = {};
    __device__ __forceinline__ Walk(const AttendParams& p, const Place& c)
        : pos(c.pos), end(c.pos + c.len < c.total ? c.pos + c.len : c.total), item(c.item), item_pos(c.item_pos), len(c.len) {}
    __device__ __forceinline__ Walk(uint32_t unit, uint32_t Hk) : pos(unit % Hk), end(-1), item(unit / Hk), item_pos(0), len(1) {}
    __device__ __forceinline__ bool next(const AttendParams& p, int shift, Unit& u) {
        if (!p.ctas) {  // one unit
            if (end == 0) return false;
            end = 0;
            u.t = tile_of(p, item, shift);
            u.kvh = static_cast<int>(pos);
            u.begin = u.t.sp.first_lo >> shift, u.end = u.begin + u.t.blocks, u.slot = -1;
            return u.t.nrows > 0;
        }
        while (pos < end) {
            u.t = tile_of(p, item, shift);
            const int64_t places = tile_places(p, u.t), off = pos - item_pos;
            if (off >= places) {
                item_pos += places;
                ++item;
                continue;
            }
            const int per = u.t.blocks + p.unit_cost;
            u.kvh = static_cast<int>(off / per);
            const int x0 = static_cast<int>(off - static_cast<int64_t>(u.kvh) * per);
            const int x1 = static_cast<int>(min(static_cast<int64_t>(per), x0 + end - pos));
            pos += x1 - x0;
            const int from = max(0, x0 - p.unit_cost), to = max(0, x1 - p.unit_cost);
            if (to <= from) continue;
            u.begin = (u.t.sp.first_lo >> shift) + from, u.end = u.begin + to - from;
            u.slot = from == 0 && to == u.t.blocks ? -1 : 2 * static_cast<int64_t>(blockIdx.x) + (from == 0 ? 1 : 0);
            if (from == 0 && to < u.t.blocks)  // (a range is much shorter than 2^31 blocks where it cuts anything)
                cut = {u.t.s.row0, u.t.r0, u.t.nrows, u.kvh, 1 + static_cast<int>((u.t.blocks - to + len - 1) / len), {0, 0}};
            return true;
        }
        return false;
    }
};

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

// Softmax weights are kept in f16 for the second product, relative to a reference within 2^5 of the
// running maximum (it moves only when a score passes it by that much, which is rare, so the sums are
// seldom rescaled) and times 2^10: at most 2^15, with 11 bits down to 2^-24 of the largest.  (Within 2^8 and
// times 2^6 is no faster, and 2^-26 of the largest, all that counts where that one's value is zero, is off by 3 to 8 %.)
constexpr float kSlack = 5.0f;
constexpr float kLift = 10.0f;

// A weight's exponent is fma(product, factor, -reference), with the reference made of the largest score rounded to fp32:
// for scores of 2^24 and more that rounding could be the whole exponent.  Where a row's last reference is this large, the
// unit is done again (WIDE), with scores that are rounded before the reference is taken from them.  (Infinite: a row
// that is NaN.)  Sums relative to earlier references as large are wiped when the reference moves on.
__device__ __forceinline__ bool too_large(float ref) { return fabsf(ref) >= 8388608.0f && fabsf(ref) < INFINITY; }
__device__ __forceinline__ float rescaled(float x, float by) { return by == 0.0f ? 0.0f : x * by; }  // x may be infinite

// Where V's scales lie too far apart for f16, weights times scales are bf16, whose exponents are fp32's, relative to
// a reference 2^70 below the largest scale of the same 32 elements: 2^70, times 6, a weight of 2^15 and 2^30 keys, stays
// below 2^118, and scales down to 2^-196 of the largest are not lost beside it (an infinity is stored as 2^126, so values
// of 2^-70 count even there).
__device__ __forceinline__ int wide_reference(int top) { return max(top - 70, 1); }

// --------------------------------------------------------------------------- few query rows
//
// CTAs of 4 warps.  A warp takes blocks of 32 tokens, as two strips of 16: S^T = K Q^T (m = 16 tokens,
// n = 8 rows) and O^T += V^T P^T (m = 16 elements, k = 16 tokens) by warp-level matrix instructions, which
// need 8 rows only where the 128-row tcgen05 tiles would be nearly empty.  Codes go from shared memory
// straight into fragments (the cache's layout is theirs: 16-byte loads, no shuffle) and are widened to f16
// exactly; K's block scales multiply the partial sums of their block, V's the softmax weights, relative to the
// largest scale a warp has met.  Each warp copies its own blocks, kStages deep, with nothing shared
// until the end, where the warps' sums are joined.
//
// Measured (heads of 128, 64 on 8; the kernel and the joining one, in a captured graph): 16 sequences of 32768 keys, 570 MB
// of cache, 124 us, 4.6 TB/s; 32 on 8, 32 sequences of up to 8000 keys (157 MB), 48 us, 3.3 TB/s.  The public call takes
// 121 to 135 and 45 to 49 us.  A strip of 16 tokens takes about 284 warp
// instructions (a conversion per two codes, 64, and 32 matrix instructions and their scales among them); they fill 56 %
// of the issue slots of three CTAs an SM.  Four CTAs (128 registers, spilling) issue no more; one strip at a time
// is 9 % slower, as two in flight hide each other's latencies; a CTA's start and end cost some 15 us in all.
//
// V's scale goes into the weight, as an f16 relative to a reference up to 2^1 above the largest scale met: with the
// largest weights 2^10 and more, what a row weighs by 2^-12 of them keeps 11 bits at scales down to 2^-12 of the reference.
// A warp notes the smallest it met, too; where that lies lower (V blocks 2^12 and more apart, and it does not matter which
// row sees them) the CTA does the unit again, WIDE: weights and scales as bf16, the weights as a sum of two (2^-17 of
// themselves), relative to a reference of each block of elements.  That is twice the matrix instructions for V and some
// more for its codes.
constexpr int kFewThreads = 128;
constexpr int kFewSpan = 12;
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
    struct Scales {
        alignas(16) float k[4][2][16][kBlocks];    // a warp's strips: 2^(e - 127) of K's blocks
        alignas(16) uint32_t v[4][2][8][kBlocks];  // f16 (WIDE: bf16) 2^(e - reference) of V's, two tokens
    };
    struct Both {
        Scales scale;
        alignas(16) __half q[8 * NT][D + 8];
    };
    union Either {  // 8 rows of Q go to registers before the first block
        Scales scale;
        alignas(16) __half q[8 * NT][D + 8];
    };
    typename std::conditional<NT == 1, Either, Both>::type u;
    float factor[8 * NT];
    int lo[8 * NT], hi[8 * NT];
    float2 ml[4][8];
    float vref[4][kBlocks];  // what a warp's sums of a block are relative to
    int vtop[4][kBlocks];    // the largest scale that a warp met there
    PlaceShared place;
};

// One unit, or a CTA's part of it.  False where it is to be done again, WIDE: V's scales lie too far apart for f16, or
// scores are too large (results of some of its rows may have been written then).
template <int D, int NT, bool WIDE>
__device__ __forceinline__ bool few_unit(const AttendParams& p, FewShared<D, NT>& sm, const Unit& unit) {
    const Sequence& s = unit.t.s;
    const Span& sp = unit.t.sp;
    const int kvh = unit.kvh, r0 = unit.t.r0, nrows = unit.t.nrows, begin = unit.begin, end = unit.end;
    const int64_t slot = unit.slot;
    using S = TokenBlock<D>;
    constexpr int kBlocks = D / 32, kRows = 8 * NT;
    constexpr int kSub = NT == 4 || WIDE ? 1 : 2;  // strips worked on together, as registers allow
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const int g = lane >> 2, c = lane & 3;
    const int count = max(0, (end - begin - warp + 3) >> 2);  // blocks of this warp
    const int32_t* table = p.tables + unit.t.b * p.table_width;
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
    auto page_of = [&](int t) { return t < fetch_end && t <= sp.last_hi ? table[t >> p.page_shift] : -1; };
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
                if (ahead <= sp.last_hi && lane == 0) report_index();
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

    uint16_t raw[kRows / 4][kBlocks];  // of all rows first: one wait for them
#pragma unroll
    for (int y = 0; y < kRows / 4; ++y) {
        const int r = warp + 4 * y, qi = (r0 + r) / p.G;
        const uint16_t* src = p.q + (s.row0 + qi) * p.ldq + static_cast<int64_t>(kvh * p.G + (r0 + r) - qi * p.G) * D;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) raw[y][i] = r < nrows ? __ldcg(src + 32 * i + lane) : 0;
    }
#pragma unroll
    for (int y = 0; y < kRows / 4; ++y) {
        const int r = warp + 4 * y, qi = (r0 + r) / p.G;
        float x[kBlocks];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const uint32_t w = static_cast<uint32_t>(raw[y][i]) << 16;
            x[i] = __uint_as_float(w);
            top = max(top, w & 0x7FFFFFFFu);
        }
        const uint32_t E = query_exponent(__reduce_max_sync(0xFFFFFFFFu, top));
        const float mul = query_multiplier(E);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
            sm.u.q[r][32 * i + lane] = __float2half_rn(warp_fwht32(x[i] * mul, lane) * kHadamardNorm);
        if (lane == 0) {
            sm.factor[r] = score_factor(p.scale_log2, E);
            sm.lo[r] = first_key(p, s.pos0 + qi);
            sm.hi[r] = r < nrows ? s.pos0 + qi : -1;
        }
    }
    __syncthreads();

    // thread (g, c): tokens g, g + 8 of a strip and rows 2c, 2c + 1 of each n-tile; of Q rows g
    uint4 qf[kBlocks];
    if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) qf[i] = *reinterpret_cast<const uint4*>(&sm.u.q[g][32 * i + 8 * c]);
        __syncthreads();
    }
    float f[NT][2], ref[NT][2], bound[NT][2], sum[NT][2], o[NT][2 * kBlocks][4];
    const int vp = D == 128 ? lane >> 2 : (lane >> 1) & 7, vb = lane & (kBlocks - 1);
    // V's scales: above the largest met, which the sums are relative to (WIDE: of the lane's block); the largest this lane
    // met; the smallest but 0, less 1, in either half
    int vref = WIDE ? wide_reference(sm.vtop[warp][vb]) : 0, vtop = 0;
    uint32_t vlow = 0xFFFFFFFFu;
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
            float* ks = &sm.u.scale.k[warp][u][0][0];
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
                const float* ks = &sm.u.scale.k[warp][half + u][0][0];
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
                            q = *reinterpret_cast<const uint4*>(&sm.u.q[8 * n + g][32 * j + 8 * c]);
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
            uint32_t v2[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                v2[u] = static_cast<uint32_t>(ve[u][0] | ve[u][1] << 16);
                if constexpr (!WIDE) {
                    vtop = max(max(ve[u][0], ve[u][1]), vtop);
                    vlow = __viaddmin_u16x2(v2[u], 0xFFFFFFFFu, vlow);
                }
            }

            float top[NT][2];
            bool grow = !WIDE && vtop > vref;
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
                const int nv = WIDE ? 0 : static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(vtop)));
                if (!WIDE && nv > vref) {  // with room for a doubling before the next time
                    const int to = min(nv + 1, 254);
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
                            sum[n][e] = rescaled(sum[n][e], shift);
                            scale *= shift;
                        }
#pragma unroll
                        for (int x = 0; x < 2 * kBlocks; ++x) o[n][x][e] = rescaled(o[n][x][e], scale), o[n][x][2 + e] = rescaled(o[n][x][2 + e], scale);
                    }
                }
            }

            // exponent field e - vref + 15 (bf16: 127) of two tokens, 0 below it
            const uint32_t k2 = static_cast<uint32_t>(((WIDE ? 127 : 15) - vref) & 0xFFFF) * 0x00010001u;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                sm.u.scale.v[warp][half + u][vp][vb] =
                    WIDE ? __viaddmin_s16x2_relu(v2[u], k2, 0x00FE00FEu) << 7 : __viaddmin_s16x2_relu(v2[u], k2, 0x000F000Fu) << 10;
            __syncwarp();

#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const uint8_t* st = st0 + (half + u) * S::kStrip;
                // softmax weights, transposed into fragments: tokens 2c, 2c + 1 (2c + 8, 2c + 9) of row g
                uint32_t pt0[NT], pt1[NT], pl0[NT], pl1[NT];  // (pl: what bf16 leaves of the weights)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float e0, e1, e2, e3;
                    if constexpr (WIDE) {
                        e0 = exp2_approx(__fsub_rn(__fmul_rn(sc[u][n][0], f[n][0]), ref[n][0]));
                        e1 = exp2_approx(__fsub_rn(__fmul_rn(sc[u][n][1], f[n][1]), ref[n][1]));
                        e2 = exp2_approx(__fsub_rn(__fmul_rn(sc[u][n][2], f[n][0]), ref[n][0]));
                        e3 = exp2_approx(__fsub_rn(__fmul_rn(sc[u][n][3], f[n][1]), ref[n][1]));
                    } else {
                        e0 = exp2_approx(fmaf(sc[u][n][0], f[n][0], -ref[n][0]));
                        e1 = exp2_approx(fmaf(sc[u][n][1], f[n][1], -ref[n][1]));
                        e2 = exp2_approx(fmaf(sc[u][n][2], f[n][0], -ref[n][0]));
                        e3 = exp2_approx(fmaf(sc[u][n][3], f[n][1], -ref[n][1]));
                    }
                    sum[n][0] += e0 + e2, sum[n][1] += e1 + e3;
                    if constexpr (WIDE) {
                        const uint32_t a = pack_bf16(e0, e1), z = pack_bf16(e2, e3);
                        pt0[n] = movmatrix_trans(a), pl0[n] = movmatrix_trans(pack_bf16(e0 - bf_lo(a), e1 - bf_hi(a)));
                        pt1[n] = movmatrix_trans(z), pl1[n] = movmatrix_trans(pack_bf16(e2 - bf_lo(z), e3 - bf_hi(z)));
                    } else {
                        const __half2 a = __floats2half2_rn(e0, e1), z = __floats2half2_rn(e2, e3);
                        pt0[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&a));
                        pt1[n] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&z));
                    }
                }
                uint32_t va[4], vz[4];  // pairs c and c + 4: (first token: blocks 01, 23), (second token: 01, 23)
                uint32_t vx0[kBlocks], vx1[kBlocks];
                const uint32_t* vs = &sm.u.scale.v[warp][half + u][0][0];
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
                    if constexpr (WIDE) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            ea[y] = e2m1_f16_to_bf16(ea[y]), oa[y] = e2m1_f16_to_bf16(oa[y]);
                            ez[y] = e2m1_f16_to_bf16(ez[y]), oz[y] = e2m1_f16_to_bf16(oz[y]);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = 2 * h + y;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (WIDE) {
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const uint32_t u0 = mul_bf16x2(x ? pl0[n] : pt0[n], vx0[j]), u1 = mul_bf16x2(x ? pl1[n] : pt1[n], vx1[j]);
                                    mma_bf16_16x8x16(o[n][2 * j], ea[2 * y], oa[2 * y], ez[2 * y], oz[2 * y], u0, u1);
                                    mma_bf16_16x8x16(o[n][2 * j + 1], ea[2 * y + 1], oa[2 * y + 1], ez[2 * y + 1], oz[2 * y + 1], u0, u1);
                                }
                            } else {
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
    }
    cp_async_wait<0>();
    if constexpr (!WIDE) {
        const int low = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, min(vlow & 0xFFFFu, vlow >> 16))) + 1;
        if (__syncthreads_or(low < vref - kFewSpan)) {
#pragma unroll
            for (int x = kBlocks; x < 32; x <<= 1) vtop = max(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, x));
            if (lane < kBlocks) sm.vtop[warp][lane] = vtop;
            __syncwarp();
            return false;
        }
    } else {
        __syncthreads();
    }

    // join the warps, one n-tile (8 rows) at a time: warp w's sums of row r at joined[w][r][..]
    float* joined = reinterpret_cast<float*>(sm.ring);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (8 * n >= nrows) break;
        if (n > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = sum[n][e];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
            // (nothing seen: no reference and no sum; the sum of a row that is not finite is NaN)
            if (g == 0) sm.ml[warp][2 * c + e] = make_float2(bound[n][e] == -INFINITY && t == 0.0f ? -INFINITY : ref[n][e], t);
#pragma unroll
            for (int j = 0; j < 2 * kBlocks; ++j) {
                float* row = joined + (warp * 8 + 2 * c + e) * D + 16 * j + 4 * g - (j & 1) * 14;
                *reinterpret_cast<float2*>(row) = make_float2(o[n][j][e], o[n][j][2 + e]);
            }
        }
        if (lane < kBlocks) sm.vref[warp][lane] = __uint_as_float(static_cast<uint32_t>(vref) << 23);
        if constexpr (WIDE) {
            __syncthreads();
        } else if (__syncthreads_or(too_large(ref[n][0]) || too_large(ref[n][1]))) {
            if (lane < kBlocks) sm.vtop[warp][lane] = vref;  // above the largest of all blocks
            __syncwarp();
            return false;
        }
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
                if (w[k] != 0.0f) x += joined[(k * 8 + r) * D + d] * (w[k] * inv) * sm.vref[k][d / 32];
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
    return true;
}

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads, few_resident(NT)) attend_few_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ uint4 dynamic_smem[];
    FewShared<D, NT>& sm = *reinterpret_cast<FewShared<D, NT>*>(dynamic_smem);
    griddep_wait();
    griddep_launch_dependents();
    const Place place = p.ctas ? find_place<kFewThreads>(p, kFewShift, blockIdx.x, sm.place) : Place{};
    Walk walk = p.ctas ? Walk(p, place) : Walk(blockIdx.x, p.Hk);
    Unit unit;
    while (walk.next(p, kFewShift, unit))
        if (!few_unit<D, NT, false>(p, sm, unit)) few_unit<D, NT, true>(p, sm, unit);
    if (p.ctas && threadIdx.x == 0) p.cuts[blockIdx.x] = walk.cut;
}

// ------------------------------------------------------------------------------ many query rows
//
// Persistent CTAs of five warpgroups, one per SM, on units of 256 rows (two tensor-core tiles of 128) and
// blocks of 128 keys:
//   warpgroups 0, 1  softmax of one tile each, a thread a row: scores out of tensor memory, weights (f16) back
//                    in their place, the tile's sums rescaled there when the reference moves; before that
//                    the rows' queries (transform, f16, shared memory), after it the results
//   warpgroup 2      K: codes to f16 in shared memory, K-major
//   warpgroup 3      V: likewise, elements along the rows (MN-major, as V's codes lie)
//   warp 17          finds the CTA's units
//   warp 19          looks for scales that lie too far apart
//   warps 16, 18     issue S_t = Q_t K^T and O_t += P_t V of one tile each (tcgen05, f16 operands, fp32 sums)
// so matrix products, exponentials and the widening of the next blocks' codes run side by side.  A block is worked on
// in halves of 64 keys: in tensor memory stand S_0, S_1 (two halves of 64 columns each, the first 32 of a half
// then P) and O_0, O_1 (128 each), so that a half's scores are there before the softmax of the one ahead ends.
// E2M1 times a power of two is exact in f16: K is held relative to the largest scale of a warp's 32 tokens (which
// goes into those columns' score factor), V relative to a reference above the largest scale met in the unit (rescaled like
// the softmax reference when it moves), with 2^12 on top, so scales down to 2^-26 of the largest are exact.
//
// That is not enough where V's scales lie further apart than 2^kManySpan: blocks vanish, and the weights are f16, too, off by
// 2^-35 of the largest where they are small, which a value 2^16 larger than the largest weight's makes 2^-19 of that
// one's share.  Where K's scales lie as far apart, a token can be lost beside another of the 32 that a row may not see
// or gives no weight.  Warp 19 looks at the units' scales on its own, and when the CTA is through its units it does those again,
// WIDE, with operands in bf16, whose exponents are fp32's: weights as the sum of two (2^-17 of themselves; the second over
// the other half of the scores' columns), V relative to wide_reference of each block of elements, and K's tokens relative to
// their own largest scales, which then go into each column's score.  A unit takes 1.8 times
// as long that way, 2.8 times in all (prompt of 8192 tokens, a value 2^40 times larger in each head: 0.64 / 1.8 ms).  A
// branch in the roles' loops instead, or the look at the scales in the role that widens V, cost every call 15 % and more.
//
// Measured: a prompt of 8192 tokens, 32 heads of 128 on 8, 629 us with the joining kernel in a captured graph, 875 TFLOP/s
// of the pairs the mask leaves (tensor pipe less than half busy); the public call takes 640 to 680 us.  When this kernel
// alone took 605 us, neither the exponentials (replaced by a product: 583 us) nor the widening (left out: 577 us) bound it,
// but the chain scores - maximum - weights - products of a tile with only two softmax warps a scheduler to hide it.
// On the way there: products issued by a thread that the compiler did not know to be one 1713 us, by a converged
// warp 1310; code cut so that the roles' loops fit the instruction cache 718; scores of half blocks ahead, two issuing
// warps 640.  Letting the two tiles' exponentials take turns cost 3 %.
constexpr int kManyShift = 7;
constexpr int kManyRows = 256;
constexpr int kManyThreads = 640;
// Registers of a thread: 96 at launch (640 threads), then split 112 / 96 / 64 (softmax / codes / products).
constexpr int kManyLaunchRegs = 96, kSoftmaxRegs = 112, kCodeRegs = 96, kIssueRegs = 64;
static_assert(2 * kSoftmaxRegs + 2 * kCodeRegs + kIssueRegs <= 5 * kManyLaunchRegs, "registers of a CTA");
constexpr int kOperandLift = 12;
constexpr int kManyUnits = 4, kUnitReaders = 18;
constexpr int kManySpan = 16;
constexpr int kRedoUnits = 2048;  // units of a CTA that are told apart (of those behind, all are done again or none)
static_assert(kRedoUnits / 4 + 1 <= kManyThreads, "one word a thread");
// WIDE, a column's factor is 2^(its token's largest scale - kKeyReference): 2^60 for an infinity's, where products reach 2^38
constexpr int kKeyReference = 193;

template <int D>
struct ManyShared {
    static constexpr int kTile = 128 * D * 2;  // bytes of 128 rows of f16, in panels of 64 elements (16 KB)
    static constexpr int kRaw = 16 * D + 32 * (D / 32);  // codes and scales of a warp's 32 tokens of K or V
    alignas(1024) uint8_t q[2][kTile];
    alignas(1024) uint8_t k[2][kTile];
    alignas(1024) uint8_t v[2][kTile];
    alignas(16) uint8_t raw[8][kRaw];
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], q_full[2], s_full[2][2], p_full[2][2], o_done[2], o_full[2];
    uint64_t r_full[4], drained[2];
    // of block j at [j % 4]: each K warp's largest scale and its strips (16 tokens) whose page is not there,
    // and V's reference; a slot is rewritten after the products of block j + 2, whose softmax follows that of j.  r_full: V's is there
    int k_ref[4][4], gone[4][4], v_ref[4];
    int v_top[4];
    // of units done again: what each key's scores are multiplied by, V's references of each block of elements (bytes)
    alignas(16) float k_factor[4][128];
    uint32_t v_refs[4];
    uint2 v_tops[4];
    int abort;
    uint32_t tmem;
    PlaceShared place;
    Place start;  // the CTA's range
    alignas(4) uint8_t redo[kRedoUnits + 4];  // units (by their number in the range) to be done again
    int redo_any;
    // the CTA's units in order, written by one warp (so that no other spends registers on finding them) and read
    // by the 18 that work on them; past the last one stands an empty one
    Unit unit[kManyUnits];
    uint64_t unit_full[kManyUnits], unit_free[kManyUnits];
};

// Waits for the phase with the given parity, with one answer for the whole warp: false (and the abort flag and
// the device status are set) after some 4 s, which means a logic error.  A few instructions, since every
// role has several of these in its loop, and the roles' loops share one instruction cache.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort) {
    constexpr uint32_t kPause = 2000;  // ns
    for (int n = 0; !__all_sync(0xFFFFFFFFu, mbar_try_wait_for(bar, parity, kPause)); ++n) {
        if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(abort) != 0) || n > 2000000) {
            atomicExch(&g_device_status, MACAQ_ETIMEOUT);
            *reinterpret_cast<volatile int*>(abort) = 1;
            return false;
        }
    }
    return true;
}

// One arrival for what all lanes have done (32 of them would queue up at the barrier).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// A warp's next unit: waits for number n, and gives number n - 1 back first.  False: there is none.
template <int D>
__device__ __forceinline__ bool next_unit(ManyShared<D>& sm, int n, int lane) {
    __syncwarp();
    if (n > 0 && lane == 0) mbar_arrive(&sm.unit_free[(n - 1) % kManyUnits]);
    if (!warp_wait(&sm.unit_full[n % kManyUnits], (n / kManyUnits) & 1, &sm.abort)) return false;
    return sm.unit[n % kManyUnits].end > 0;
}

template <int D>
__device__ __forceinline__ void mark_redo(ManyShared<D>& sm, int n) {
    sm.redo[min(n, kRedoUnits)] = 1;
    sm.redo_any = 1;
}
template <int D>
__device__ __forceinline__ bool must_redo(const ManyShared<D>& sm, int n) {
    return sm.redo[min(n, kRedoUnits)] != 0;
}

// One warp: writes the units (WIDE: those that are done again).
template <int D, bool WIDE>
__device__ __forceinline__ void many_units(const AttendParams& p, ManyShared<D>& sm, int lane) {
    Walk walk(p, sm.start);
    bool more = true;
    int number = 0;
    for (int n = 0; more; ++n) {
        const int at = n % kManyUnits;
        if (n >= kManyUnits && !warp_wait(&sm.unit_free[at], ((n / kManyUnits) & 1) ^ 1, &sm.abort)) {
            walk.cut.parts = 0;  // nothing to join of a launch that gave up
            break;
        }
        Unit u;
        do
            more = walk.next(p, kManyShift, u);
        while (WIDE && more && !must_redo<D>(sm, number++));
        if (!more) u.end = 0;
        if (lane == 0) {
            sm.unit[at] = u;
            mbar_arrive(&sm.unit_full[at]);
        }
    }
    if (lane == 0 && (!WIDE || walk.cut.parts == 0)) p.cuts[blockIdx.x] = walk.cut;
}

// One warp: looks at the scales of the units' K and V, and notes the units whose scales lie too far apart.  (It reads them
// for itself: the roles that widen codes have no time for it.)  A first look, of 2 instructions a word: four scales plus
// 136 - c, c one of the unit's own, are 128 .. 143, or off by a carry, if all of them lie within 2^8 of c (c far enough
// from 0 and 255 that nothing wraps into that).  Where one does not, a second look takes the largest and the smallest but 0.
template <int D>
__device__ __forceinline__ void many_ranges(const AttendParams& p, ManyShared<D>& sm, int lane) {
    constexpr int kBlocks = D / 32, kTokens = 16 / kBlocks;  // of a lane's 16 bytes of scales
    const PageLayout<D> lay{p.page_size};
    const uint32_t page_stride = static_cast<uint32_t>(p.Hk * lay.bytes());
    for (int n = 0; next_unit<D>(sm, n, lane); ++n) {
        const Unit& u = sm.unit[n % kManyUnits];
        const int32_t* table = p.tables + u.t.b * p.table_width;
        const int first = max(u.t.sp.first_lo, u.begin << kManyShift), last = min(u.t.sp.last_hi, (u.end << kManyShift) - 1);
        const uint8_t* head = p.cache + u.kvh * lay.bytes() + lay.k_scales();
        const int v_at = p.page_size * kBlocks;
        // the scales of K at token t (those of V are v_at further), or null (an absent page is reported where it is used)
        auto scales = [&](int t) -> const uint8_t* {
            const int32_t pg = table[t >> p.page_shift];
            if (static_cast<unsigned>(pg) >= static_cast<uint64_t>(p.num_pages)) return nullptr;
            return head + static_cast<uint64_t>(static_cast<uint32_t>(pg)) * page_stride + (t & (p.page_size - 1)) * kBlocks;
        };
        // what of a lane's word i is seen
        auto mask = [&](int t, int i) {  // D = 128: a token's four scales; D = 64: two tokens' two, in either half
            const int t0 = t + i * kTokens / 4, t1 = t + (i * kTokens + kTokens / 2) / 4;
            return (t0 >= first && t0 <= last ? 0x0000FFFFu : 0u) | (t1 >= first && t1 <= last ? 0xFFFF0000u : 0u);
        };
        const int from = (first & -kTokens) + kTokens * lane;
        const uint8_t* one = first <= last ? scales(first) : nullptr;
        const uint32_t kc = one ? __ldcg(one) : 0, vc = one ? __ldcg(one + v_at) : 0;
        bool far = first <= last && (kc - 16 > 223 || vc - 16 > 223);
        if (!far) {
            const uint32_t kb = (136 - kc & 0xFFu) * 0x01010101u, vb = (136 - vc & 0xFFu) * 0x01010101u;
            uint32_t out = 0;
#pragma unroll 1
            for (int t = from; t <= last; t += 32 * kTokens) {
                const uint8_t* at = scales(t);
                if (!at) continue;
                uint4 k = __ldcg(reinterpret_cast<const uint4*>(at)), v = __ldcg(reinterpret_cast<const uint4*>(at + v_at));
                if (t < first || t + kTokens - 1 > last) {
                    uint32_t* kw = reinterpret_cast<uint32_t*>(&k);
                    uint32_t* vw = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t see = mask(t, i);
                        kw[i] = (kw[i] & see) | (kc * 0x01010101u & ~see);
                        vw[i] = (vw[i] & see) | (vc * 0x01010101u & ~see);
                    }
                }
                out |= (k.x + kb ^ 0x80808080u) | (k.y + kb ^ 0x80808080u) | (k.z + kb ^ 0x80808080u) | (k.w + kb ^ 0x80808080u) |
                       (v.x + vb ^ 0x80808080u) | (v.y + vb ^ 0x80808080u) | (v.z + vb ^ 0x80808080u) | (v.w + vb ^ 0x80808080u);
            }
            far = (out & 0xF0F0F0F0u) != 0;
        }
        if (!__any_sync(0xFFFFFFFFu, far)) continue;
        // of V's blocks, of K's tokens (each token's largest): the largest, the smallest but 0 less 1, in either half
        uint32_t vtop = 0, vlow = 0xFFFFFFFFu, ktop = 0, klow = 0xFFFFFFFFu;
#pragma unroll 1
        for (int t = from; t <= last; t += 32 * kTokens) {
            const uint8_t* at = scales(t);
            if (!at) continue;
            const uint4 k4 = __ldcg(reinterpret_cast<const uint4*>(at)), v4 = __ldcg(reinterpret_cast<const uint4*>(at + v_at));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t see = mask(t, i);
                const uint32_t k = reinterpret_cast<const uint32_t*>(&k4)[i] & see, v = reinterpret_cast<const uint32_t*>(&v4)[i] & see;
                const uint32_t ve = v & 0x00FF00FFu, vo = v >> 8 & 0x00FF00FFu;
                vtop = __vmaxu2(vtop, __vmaxu2(ve, vo));
                vlow = __viaddmin_u16x2(vo, 0xFFFFFFFFu, __viaddmin_u16x2(ve, 0xFFFFFFFFu, vlow));
                uint32_t km = __vmaxu2(k & 0x00FF00FFu, k >> 8 & 0x00FF00FFu);
                if (D == 128) km = __vmaxu2(km, __byte_perm(km, km, 0x1032));
                ktop = __vmaxu2(ktop, km);
                klow = __viaddmin_u16x2(km, 0xFFFFFFFFu, klow);
            }
        }
        auto span = [](uint32_t top, uint32_t low) {  // negative where all are 0
            return static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16))) -
                   static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, min(low & 0xFFFFu, low >> 16))) - 1;
        };
        if (max(span(vtop, vlow), span(ktop, klow)) > kManySpan && lane == 0) mark_redo<D>(sm, n);
    }
}

// (of all warps, from wherever they are: their roles' code is not one place)
__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// Codes of a warp's 32 tokens of K or V on their way through shared memory, one block ahead; the pages' numbers
// two blocks ahead.
template <int D, bool IS_V>
struct CodeStream {
    static constexpr int kBlocks = D / 32;
    const AttendParams& p;
    ManyShared<D>& sm;
    int n = 0;  // units begun
    bool more;
    int block;        // of the request after the pending one
    int32_t page[2];  // its pages (of its first and second 16 tokens)
    uint32_t there;   // strips of the pending request that were copied, that are seen
    uint32_t seen;
    int first, last;  // the tokens of the pending request that any row sees, relative to its first
    bool fresh;       // it begins a unit
    int w, lane;

    __device__ __forceinline__ CodeStream(const AttendParams& p_, ManyShared<D>& sm_, int w_, int lane_)
        : p(p_), sm(sm_), w(w_), lane(lane_) {
        begin_unit();
        look();
    }
    __device__ __forceinline__ const Unit& unit() const { return sm.unit[(n - 1) % kManyUnits]; }
    __device__ __forceinline__ void begin_unit() {
        more = next_unit<D>(sm, n++, lane);
        if (more) block = unit().begin;
    }
    __device__ __forceinline__ void look() {
        page[0] = page[1] = -1;
        if (!more) return;
        const Unit& u0 = unit();
        const int t = block * 128 + 32 * w;
        const int32_t* table = p.tables + u0.t.b * p.table_width;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (t + 16 * u <= u0.t.sp.last_hi && t + 16 * u + 15 >= u0.t.sp.first_lo)
                page[u] = table[(t + 16 * u) >> p.page_shift];
    }
    // Starts the copies of the next block and looks further.
    __device__ __forceinline__ void request(uint8_t* raw) {
        if (more) {
            const Unit& u0 = unit();
            const int t0 = block * 128 + 32 * w;
            const PageLayout<D> lay{p.page_size};
            there = seen = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = t0 + 16 * u;
                if (t > u0.t.sp.last_hi || t + 15 < u0.t.sp.first_lo) continue;
                seen |= 1u << u;
                if (static_cast<unsigned>(page[u]) >= static_cast<uint64_t>(p.num_pages)) {
                    if (lane == 0) report_index();
                    continue;
                }
                there |= 1u << u;
                const int at = t & (p.page_size - 1);
                const uint8_t* src = p.cache + (static_cast<int64_t>(page[u]) * p.Hk + u0.kvh) * lay.bytes();
                const uint8_t* codes = src + (IS_V ? lay.v_codes() : 0) + at * lay.kRow + 16 * lane;
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    const int piece = lane + 32 * x;  // V's pieces swizzled as its readers want them
                    const int to = !IS_V ? piece
                                   : D == 128 ? (piece / 8) * 8 + ((piece % 8) ^ ((piece / 8 & 3) * 2))
                                              : (piece / 4) * 4 + ((piece % 4) ^ ((piece / 8 & 1) * 2));
                    cp_async16(smem_u32(raw) + u * 8 * D + 16 * to, codes + 512 * x);
                }
                if (lane < kBlocks)
                    cp_async16(smem_u32(raw) + 16 * D + 16 * kBlocks * u + 16 * lane,
                               src + (IS_V ? lay.v_scales() : lay.k_scales()) + at * kBlocks + 16 * lane);
            }
            first = u0.t.sp.first_lo - t0, last = u0.t.sp.last_hi - t0;
            fresh = block == u0.begin;
            if (++block == u0.end) begin_unit();
            look();
        }
        cp_async_commit();
    }
};

// 16 bytes of f16: eight codes times a power of two.
__device__ __forceinline__ uint4 widen_codes(uint32_t codes, uint32_t scale2) {
    uint32_t h[4];
    e2m1x8_to_f16(codes, h);
    const __half2 s = *reinterpret_cast<const __half2*>(&scale2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), s);
        h[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ uint4 widen_codes_bf16(uint32_t codes, uint32_t scale2) {
    uint32_t h[4];
    e2m1x8_to_f16(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = mul_bf16x2(e2m1_f16_to_bf16(h[i]), scale2);
    return make_uint4(h[0], h[1], h[2], h[3]);
}
// f16 2^(e - ref + kOperandLift) in both halves, 0 below the smallest normal (e <= ref); bf16 2^(e - ref).
__device__ __forceinline__ uint32_t operand_scale(uint32_t e, int ref) {
    return static_cast<uint32_t>(max(static_cast<int>(e) - ref + 15 + kOperandLift, 0)) * 0x04000400u;
}
__device__ __forceinline__ uint32_t operand_scale_bf16(uint32_t e, int ref) {
    return static_cast<uint32_t>(max(static_cast<int>(e) - ref + 127, 0)) * 0x00800080u;
}
__device__ __forceinline__ int byte_max(uint32_t w) {
    return max(max(w & 0xFFu, (w >> 8) & 0xFFu), max((w >> 16) & 0xFFu, w >> 24));
}

template <int D, bool WIDE>
__device__ __forceinline__ void many_keys(const AttendParams& p, ManyShared<D>& sm, int w, int lane) {
    constexpr int kBlocks = D / 32;
    uint8_t* raw = sm.raw[w];
    CodeStream<D, false> cs(p, sm, w, lane);
    bool pending = cs.more;
    cs.request(raw);
    // lane (token, chunk c of 8 elements a block): 8 tokens a step; the tokens of 8 neighbouring lanes differ by 4,
    // so that their 16-byte stores meet 8 different banks of the swizzled rows
    const int c = lane & 3, tok = ((lane >> 2) & 1) * 4 + (lane >> 3);
    for (int j = 0; pending; ++j) {
        uint32_t code[4][kBlocks], scale[4];
        cp_async_wait<0>();
        __syncwarp();
        int top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 8 * i + tok;
            const bool use = t >= cs.first && t <= cs.last && ((cs.there >> (i >> 1)) & 1u);
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(raw + t * 64 + 16 * c);
                code[i][0] = x.x, code[i][1] = x.y, code[i][2] = x.z, code[i][3] = x.w;
                scale[i] = *reinterpret_cast<const uint32_t*>(raw + 16 * D + 4 * t);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(raw + t * 32 + 8 * c);
                code[i][0] = x.x, code[i][1] = x.y;
                scale[i] = *reinterpret_cast<const uint16_t*>(raw + 16 * D + 2 * t);
            }
            if (!use) {  // whatever lay there: zeros
                scale[i] = 0;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) code[i][b] = 0;
            }
            if constexpr (!WIDE) top = max(top, byte_max(scale[i]));
        }
        const uint32_t gone = cs.seen & ~cs.there;
        __syncwarp();
        pending = cs.more;
        cs.request(raw);
        int ref = WIDE ? kKeyReference : static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(top)));
        const int stage = j & 1;
        if (j >= 2 && !warp_wait(&sm.k_free[stage], ((j >> 1) & 1) ^ 1, &sm.abort)) break;
        if (lane == 0) sm.k_ref[j & 3][w] = ref, sm.gone[j & 3][w] = static_cast<int>(gone);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 32 * w + 8 * i + tok;
            if constexpr (WIDE) {  // relative to the token's own largest scale
                ref = byte_max(scale[i]);
                if (c == 0) sm.k_factor[j & 3][row] = __uint_as_float(static_cast<uint32_t>(max(ref + 127 - kKeyReference, 1)) << 23);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t s2 = operand_scale((scale[i] >> (8 * b)) & 0xFFu, ref);
                const int chunk = (4 * (b & 1) + c) ^ (row & 7);
                *reinterpret_cast<uint4*>(sm.k[stage] + (b >> 1) * 16384 + row * 128 + chunk * 16) = widen_codes(code[i][b], s2);
            }
        }
        fence_proxy_async_smem();
        warp_arrive(&sm.k_full[stage], lane);
    }
    cp_async_wait<0>();
}

template <int D, bool WIDE>
__device__ __forceinline__ void many_values(const AttendParams& p, ManyShared<D>& sm, int w, int lane) {
    constexpr int kBlocks = D / 32, kWords = kBlocks / 2;
    uint8_t* raw = sm.raw[4 + w];
    CodeStream<D, true> cs(p, sm, w, lane);
    bool pending = cs.more;
    cs.request(raw);
    // lane (pair of tokens, elements 8c .. 8c + 7 of each block): 8 pairs a step; 8 neighbouring lanes are 4 pairs
    // by 2 chunks, whose 16-byte stores meet 8 different banks
    const int c = ((lane >> 2) & 1) + ((lane >> 3) & 1) * 2, pr = (lane & 3) + (lane >> 4) * 4;
    int ref = 0;
    uint32_t refs = 0;  // WIDE: of each block of elements
    for (int j = 0; pending; ++j) {
        uint32_t code[2][4 * kWords], scale[2][2];
        cp_async_wait<0>();
        __syncwarp();
        int top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pair = 8 * i + pr;
            if constexpr (D == 128) {
                const int s = (pair & 3) * 2;
                const uint4 x = *reinterpret_cast<const uint4*>(raw + pair * 128 + 16 * ((2 * c) ^ s));
                const uint4 y = *reinterpret_cast<const uint4*>(raw + pair * 128 + 16 * ((2 * c + 1) ^ s));
                code[i][0] = x.x, code[i][1] = x.y, code[i][2] = x.z, code[i][3] = x.w;
                code[i][4] = y.x, code[i][5] = y.y, code[i][6] = y.z, code[i][7] = y.w;
                const uint2 e = *reinterpret_cast<const uint2*>(raw + 16 * D + 8 * pair);
                scale[i][0] = e.x, scale[i][1] = e.y;
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(raw + pair * 64 + 16 * (c ^ ((pair >> 1 & 1) * 2)));
                code[i][0] = x.x, code[i][1] = x.y, code[i][2] = x.z, code[i][3] = x.w;
                const uint32_t e = *reinterpret_cast<const uint32_t*>(raw + 16 * D + 4 * pair);
                scale[i][0] = e & 0xFFFFu, scale[i][1] = e >> 16;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t = 2 * pair + r;
                if (t < cs.first || t > cs.last || !((cs.there >> i) & 1u)) {  // whatever lay there: zeros
                    scale[i][r] = 0;
#pragma unroll
                    for (int x = 0; x < kWords; ++x) code[i][r * kWords + x] = code[i][(2 + r) * kWords + x] = 0;
                }
                top = max(top, byte_max(scale[i][r]));
            }
        }
        if (cs.fresh) ref = 0, refs = 0;  // nothing of one unit's values reaches another's
        __syncwarp();
        pending = cs.more;
        cs.request(raw);
        top = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(top)));
        const int stage = j & 1;
        // all four warps go on or none does (kNoBlock in one of them: its wait gave up)
        constexpr int kNoBlock = 1 << 20;
        if (j >= 2 && !warp_wait(&sm.v_free[stage], ((j >> 1) & 1) ^ 1, &sm.abort)) top = kNoBlock;
        if (lane == 0) sm.v_top[w] = top;
        group_sync(2);
        top = max(max(sm.v_top[0], sm.v_top[1]), max(sm.v_top[2], sm.v_top[3]));
        group_sync(2);
        if (top == kNoBlock) break;
        if (top > ref) ref = min(top + 3, 254);  // room for three doublings before the next time
        int unit[kBlocks];  // WIDE: wide_reference of each block of elements
        if constexpr (WIDE) {
            uint2 tops = make_uint2(0, 0);  // blocks 0 and 2, 1 and 3
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                tops.x = __vmaxu2(tops.x, scale[i >> 1][i & 1] & 0x00FF00FFu);
                tops.y = __vmaxu2(tops.y, scale[i >> 1][i & 1] >> 8 & 0x00FF00FFu);
            }
            for (int x = 1; x < 32; x <<= 1) {
                tops.x = __vmaxu2(tops.x, __shfl_xor_sync(0xFFFFFFFFu, tops.x, x));
                tops.y = __vmaxu2(tops.y, __shfl_xor_sync(0xFFFFFFFFu, tops.y, x));
            }
            if (lane == 0) sm.v_tops[w] = tops;
            group_sync(2);
            for (int x = 0; x < 4; ++x) tops.x = __vmaxu2(tops.x, sm.v_tops[x].x), tops.y = __vmaxu2(tops.y, sm.v_tops[x].y);
            group_sync(2);
            const uint32_t old = refs;
            uint32_t units = 0;
            refs = 0;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t t = (b & 1 ? tops.y : tops.x) >> (16 * (b >> 1)) & 0xFFu, r = old >> (8 * b) & 0xFFu;
                const uint32_t now = t > r ? min(t + 3, 254u) : r;
                refs |= now << (8 * b);
                unit[b] = wide_reference(static_cast<int>(now));
                units |= static_cast<uint32_t>(unit[b]) << (8 * b);
            }
            if (lane == 0 && w == 0) sm.v_refs[j & 3] = units;
        }
        if (lane == 0 && w == 0) {
            sm.v_ref[j & 3] = ref;
            mbar_arrive(&sm.r_full[j & 3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 32 * w + 2 * (8 * i + pr) + r;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    // four codes of elements 8c .. and four of 8c + 4 ..
                    const uint32_t x = code[i][r * kWords + (b >> 1)], y = code[i][(2 + r) * kWords + (b >> 1)];
                    const uint32_t word = __byte_perm(x, y, b & 1 ? 0x7632 : 0x5410);
                    const uint32_t e = (scale[i][r] >> (8 * b)) & 0xFFu;
                    const int chunk = (4 * (b & 1) + c) ^ (row & 7);
                    *reinterpret_cast<uint4*>(sm.v[stage] + (b >> 1) * 16384 + row * 128 + chunk * 16) =
                        WIDE ? widen_codes_bf16(word, operand_scale_bf16(e, unit[b])) : widen_codes(word, operand_scale(e, ref));
                }
            }
        }
        fence_proxy_async_smem();
        warp_arrive(&sm.v_full[stage], lane);
    }
    cp_async_wait<0>();
}

// One warp: the matrix products of tile t, issued by one of its lanes.
template <int D, bool WIDE>
__device__ __forceinline__ void many_products(ManyShared<D>& sm, int t, int lane) {
    constexpr uint32_t kF32 = 1u << 4;  // fp32 sums, f16 operands
    constexpr uint32_t kScoreDesc = kF32 | ((64u >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t kBf16 = 1u << 7 | 1u << 10;
    constexpr uint32_t kValueDesc = kF32 | (WIDE ? kBf16 : 0u) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t kNext = ManyShared<D>::kTile >> 4, kHalf = 64 * 128 >> 4;
    const uint32_t tm = sm.tmem + 128 * t;
    const uint64_t qd = desc_sw128(smem_u32(sm.q[t])), k0 = desc_sw128(smem_u32(sm.k[0]));
    const uint64_t v0 = desc_mn_sw128(smem_u32(sm.v[0]), 16384);
    int j = 0, units = 0;
    for (; next_unit<D>(sm, units, lane); ++units) {
        const Unit& unit = sm.unit[units % kManyUnits];
        const int halves = 2 * (unit.end - unit.begin);
        if (!warp_wait(&sm.q_full[t], units & 1, &sm.abort)) return;
#pragma unroll 1
        for (int h = 0; h <= halves; ++h) {
            if (h < halves) {  // S = Q K^T of half h
                const int b = j + (h >> 1), half = h & 1;
                if (half == 0 && !warp_wait(&sm.k_full[b & 1], (b >> 1) & 1, &sm.abort)) return;
                tc_fence_after();
                const uint64_t kd = k0 + (b & 1) * kNext + half * kHalf;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                        tc_mma_f16(tm + 64 * half, qd + at, kd + at, kScoreDesc, k ? 1u : 0u);
                    }
                    mbar_arrive(&sm.s_full[t][half]);  // what this thread has seen (the block's references) goes on with it
                    tc_commit(&sm.s_full[t][half]);
                    if (half == 1) tc_commit(&sm.k_free[b & 1]);
                }
                __syncwarp();
            }
            if (h > 0) {  // O (+)= P V of the half before
                const int b = j + ((h - 1) >> 1), half = (h - 1) & 1;
                if (half == 0 && !warp_wait(&sm.v_full[b & 1], (b >> 1) & 1, &sm.abort)) return;
                if (!warp_wait(&sm.p_full[t][half], b & 1, &sm.abort)) return;
                tc_fence_after();
                const uint64_t vd = v0 + (b & 1) * kNext + half * kHalf;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f16_ts(tm + 256, tm + 64 * half + 8 * k, vd + (k * 2048 >> 4), kValueDesc, h == 1 && k == 0 ? 0u : 1u);
                    if constexpr (WIDE) {  // what bf16 left of the weights
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_f16_ts(tm + 256, tm + 64 * half + 32 + 8 * k, vd + (k * 2048 >> 4), kValueDesc, 1u);
                    }
                    tc_commit(&sm.o_done[t]);
                    if (h == halves) tc_commit(&sm.o_full[t]);
                    if (half == 1) tc_commit(&sm.v_free[b & 1]);
                }
                __syncwarp();
            }
        }
        j += halves >> 1;
    }
}

// A thread's query row: what it sees, where its result goes, its score factor; and the row itself to shared
// memory (zeros for rows past the tile's last).
struct QueryRow {
    int lo, hi;
    int64_t out;  // row of out, or < 0
    float factor;
};
template <int D>
__device__ __forceinline__ QueryRow load_query(const AttendParams& p, ManyShared<D>& sm, const Unit& u, int t, int tid) {
    QueryRow q = {0, -1, -1, 1.0f};
    const int r = 128 * t + tid;
    uint8_t* dst = sm.q[t] + tid * 128;
    if (r >= u.t.nrows) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint4*>(dst + (i >> 3) * 16384 + ((i & 7) ^ (tid & 7)) * 16) = make_uint4(0, 0, 0, 0);
    } else {
        const int rr = u.t.r0 + r, qi = rr / p.G, h = u.kvh * p.G + rr - qi * p.G;
        q.hi = u.t.s.pos0 + qi;
        q.lo = first_key(p, q.hi);
        q.out = (u.t.s.row0 + qi) * p.Hq + h;
        const uint16_t* src = p.q + (u.t.s.row0 + qi) * p.ldq + static_cast<int64_t>(h) * D;
        uint32_t top = 0;
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
            uint32_t w[16];
            load32(src + 32 * b, w);
#pragma unroll
            for (int k = 0; k < 16; ++k) top = max(top, max(w[k] << 16 & 0x7FFFFFFFu, w[k] & 0x7FFF0000u));
        }
        const uint32_t E = query_exponent(top);
        q.factor = score_factor(p.scale_log2, E);
        const float mul = query_multiplier(E);
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
            uint32_t w[16];
            load32(src + 32 * b, w);
            float2 f[16], m[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) f[k] = make_float2(bf_lo(w[k]), bf_hi(w[k])), m[k] = make_float2(mul, mul);
            scale_fwht32(f, m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 y = __floats2half2_rn(f[4 * i + k].x * kHadamardNorm, f[4 * i + k].y * kHadamardNorm);
                    h4[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *reinterpret_cast<uint4*>(dst + (b >> 1) * 16384 + ((4 * (b & 1) + i) ^ (tid & 7)) * 16) =
                    make_uint4(h4[0], h4[1], h4[2], h4[3]);
            }
        }
    }
    fence_proxy_async_smem();
    warp_arrive(&sm.q_full[t], tid & 31);
    return q;
}

template <int D, bool WIDE>
__device__ __forceinline__ void many_softmax(const AttendParams& p, ManyShared<D>& sm, int t, int tid) {
    const uint32_t lanes = static_cast<uint32_t>(tid & 96) << 16;  // the warp's 32 lanes of tensor memory
    const uint32_t ts = sm.tmem + 128 * t + lanes, to = sm.tmem + 256 + 128 * t + lanes;
    int j = 0, units = 0;
    float ref = 0.0f, bound = -INFINITY, sum = 0.0f;
    int vref = 0;
    uint32_t vunit = 0;  // WIDE: what the sums of each block of elements count units of
    int64_t slot = -1;
    QueryRow row = {0, -1, -1, 1.0f};
    for (;; ++units) {
        // this unit's queries (the last one's have been used: its last scores are there), then the last one's results
        const int64_t out = row.out, out_slot = slot;
        const bool more = next_unit<D>(sm, units, tid & 31);
        const Unit& unit = sm.unit[units % kManyUnits];
        if (more) {
            row = load_query<D>(p, sm, unit, t, tid);
            slot = unit.slot;
        }
        if (units > 0) {
            if (!warp_wait(&sm.o_full[t], (units - 1) & 1, &sm.abort)) return;
            tc_fence_after();
            const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
            float vs = vref > kOperandLift ? __uint_as_float(static_cast<uint32_t>(vref - kOperandLift) << 23) : 0.0f;
            const float m = bound == -INFINITY && sum == 0.0f ? -INFINITY : ref;  // (a row that is not finite: NaN)
            const int64_t at = out_slot * kManyRows + 128 * t + tid;
#pragma unroll 1
            for (int b = 0; b < D / 32; ++b) {
                float2 o[16];
                tmem_ld32(to + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(o));
                tmem_ld_wait();
                if constexpr (WIDE) vs = __uint_as_float((vunit >> (8 * b) & 0xFFu) << 23);
                const float2 i2 = make_float2(inv, inv), v2 = make_float2(vs, vs);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __fmul2_rn(__fmul2_rn(o[i], i2), v2);
                if (out < 0) continue;
                if (out_slot >= 0) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + 32 * b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[2 * i].x, o[2 * i].y, o[2 * i + 1].x, o[2 * i + 1].y);
                } else {
                    float2 n[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) n[i] = make_float2(kHadamardNorm, kHadamardNorm);
                    scale_fwht32(o, n);
                    uint4* dst = reinterpret_cast<uint4*>(p.out + out * D + 32 * b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_uint4(pack_bf16(o[4 * i].x, o[4 * i].y), pack_bf16(o[4 * i + 1].x, o[4 * i + 1].y),
                                            pack_bf16(o[4 * i + 2].x, o[4 * i + 2].y), pack_bf16(o[4 * i + 3].x, o[4 * i + 3].y));
                }
            }
            tc_fence_before();
            if (!WIDE && __any_sync(0xFFFFFFFFu, too_large(m))) mark_redo<D>(sm, units - 1);
            if (out >= 0) {
                if (out_slot >= 0)
                    p.part_ml[at] = make_float2(m, sum);
                else if (p.lse)
                    p.lse[out] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
            }
        }
        if (!more) return;
        ref = 0.0f, bound = -INFINITY, sum = 0.0f, vref = 0, vunit = 0;
        const int begin = unit.begin, halves = 2 * (unit.end - unit.begin);
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {  // 64 keys
            const int b = j + (h >> 1), half = h & 1;
            const uint32_t th = ts + 64 * half;
            if (half == 0 && !warp_wait(&sm.r_full[b & 3], (b >> 2) & 1, &sm.abort)) return;
            if (!warp_wait(&sm.s_full[t][half], b & 1, &sm.abort)) return;
            tc_fence_after();
            float f[2];
            uint32_t gone = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // score of a product: times 2^(k_ref - 127 - kOperandLift)
                const int e = max(sm.k_ref[b & 3][2 * half + i] - kOperandLift, 1);
                f[i] = fmaxf(row.factor * __uint_as_float(static_cast<uint32_t>(e) << 23), 1.17549435e-38f);
                gone |= static_cast<uint32_t>(sm.gone[b & 3][2 * half + i]) << (2 * i);
            }
            const int key0 = (begin * 2 + h) * 64, lo = row.lo - key0, hi = row.hi - key0;
            if (__any_sync(0xFFFFFFFFu, gone != 0 || lo > 0 || hi < 63)) {  // masked in place
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[32];
                    tmem_ld32(th + 32 * i, x);
                    // columns lo .. hi, without those whose page is not there
                    const int a = max(lo - 32 * i, 0), z = min(hi - 32 * i, 31);
                    uint32_t keep = a > z ? 0u : (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (31 - z));
                    keep &= ~(((gone >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((gone >> (2 * i)) & 2 ? 0xFFFF0000u : 0u));
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = (keep >> k) & 1 ? x[k] : 0xFF800000u;
                    tmem_st16(th + 32 * i, x);
                    tmem_st16(th + 32 * i + 16, x + 16);
                }
                tmem_st_wait();
            }
            float s[64];
            tmem_ld32(th, *reinterpret_cast<uint32_t(*)[32]>(s));
            tmem_ld32(th + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
            tmem_ld_wait();
            if constexpr (WIDE) {
#pragma unroll
                for (int k = 0; k < 64; ++k) s[k] *= sm.k_factor[b & 3][64 * half + k];
            }
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a = fmax3(s[32 * i], s[32 * i + 1], s[32 * i + 2]), z = fmax3(s[32 * i + 16], s[32 * i + 17], s[32 * i + 18]);
#pragma unroll
                for (int k = 3; k < 15; k += 2) {
                    a = fmax3(a, s[32 * i + k], s[32 * i + k + 1]);
                    z = fmax3(z, s[32 * i + 16 + k], s[32 * i + 16 + k + 1]);
                }
                a = fmax3(a, s[32 * i + 15], s[32 * i + 31]);
                m = fmaxf(m, fmaxf(a, z) * f[i]);
            }
            const int nv = sm.v_ref[b & 3];
            const uint32_t nunit = WIDE ? sm.v_refs[b & 3] : 0;
            if (__any_sync(0xFFFFFFFFu, m > bound || nv != vref || nunit != vunit)) {
                float scale = WIDE ? 1.0f : nv - vref < 127 ? __uint_as_float(static_cast<uint32_t>(127 - (nv - vref)) << 23) : 0.0f;
                vref = nv;
                if (m > bound - kSlack) {  // false while the row has seen nothing
                    const float old = ref;
                    ref = m - kLift;
                    const float shift = bound == -INFINITY ? 0.0f : exp2_approx(old - ref);
                    bound = m + kSlack;
                    sum = rescaled(sum, shift);
                    scale *= shift;
                }
                if (h > 0) {  // once the products of the half before are done (those of halves before that are: s_full)
                    if (!warp_wait(&sm.o_done[t], (h - 1) & 1, &sm.abort)) return;
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * i, o);
                        tmem_ld_wait();
                        float more = 1.0f, by = scale;
                        if constexpr (WIDE) {  // and by 2^(old unit - new unit), in two factors that are normal numbers
                            const int d = static_cast<int>(nunit >> (4 * i & 24) & 0xFFu) - static_cast<int>(vunit >> (4 * i & 24) & 0xFFu);
                            by *= __uint_as_float(static_cast<uint32_t>(127 - d / 2) << 23);
                            more = __uint_as_float(static_cast<uint32_t>(127 - (d - d / 2)) << 23);
                        }
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(rescaled(__uint_as_float(o[k]), by) * more);
                        tmem_st16(to + 16 * i, o);
                    }
                }
                vunit = nunit;
            }
            float2 add[2] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f2 = make_float2(f[i], f[i]), r2 = make_float2(-ref, -ref);
                uint32_t w[16], rest[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 e = make_float2(s[32 * i + 2 * k], s[32 * i + 2 * k + 1]);
                    if constexpr (WIDE)  // (the packed operations would be fused)
                        e = make_float2(__fsub_rn(__fmul_rn(e.x, f[i]), ref), __fsub_rn(__fmul_rn(e.y, f[i]), ref));
                    else
                        e = __ffma2_rn(e, f2, r2);
                    e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                    add[k & 1] = __fadd2_rn(add[k & 1], e);
                    if constexpr (WIDE) {
                        w[k] = pack_bf16(e.x, e.y);
                        rest[k] = pack_bf16(e.x - bf_lo(w[k]), e.y - bf_hi(w[k]));
                        continue;
                    }
                    const __half2 y = __floats2half2_rn(e.x, e.y);
                    w[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                tmem_st16(th + 16 * i, w);  // over scores that have been read
                if constexpr (WIDE) tmem_st16(th + 32 + 16 * i, rest);
            }
            sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.p_full[t][half], tid & 31);
        }
        j += halves >> 1;
    }
}

// One thread: all barriers as new (`again`: nothing arrives at the old ones any more).
template <int D>
__device__ __forceinline__ void many_init(ManyShared<D>& sm, bool again, uint32_t unit_readers) {
    auto init = [again](uint64_t* bar, uint32_t count) {
        if (again) mbar_inval(bar);
        mbar_init(bar, count);
    };
    for (int i = 0; i < 2; ++i) {
        init(&sm.k_full[i], 4), init(&sm.k_free[i], 2);
        init(&sm.v_full[i], 4), init(&sm.v_free[i], 2);
        init(&sm.q_full[i], 4), init(&sm.o_done[i], 1), init(&sm.o_full[i], 1);
        for (int h = 0; h < 2; ++h) init(&sm.s_full[i][h], 2), init(&sm.p_full[i][h], 4);
    }
    for (int i = 0; i < 4; ++i) init(&sm.r_full[i], 1);
    init(&sm.drained[0], 1), init(&sm.drained[1], 1);
    for (int i = 0; i < kManyUnits; ++i) init(&sm.unit_full[i], 1), init(&sm.unit_free[i], unit_readers);
    fence_mbar_init();
}

// All threads, each in its role, when the CTA's units are done: whether some are to be done again, with barriers as new.
template <int D>
__device__ __forceinline__ bool many_again(ManyShared<D>& sm) {
    tc_fence_before();
    cta_sync();
    if (!sm.redo_any || sm.abort) return false;
    if (threadIdx.x == 0) many_init(sm, true, kUnitReaders);
    cta_sync();
    tc_fence_after();
    return true;
}

template <int D, bool WIDE>
__device__ __forceinline__ void many_issue(const AttendParams& p, ManyShared<D>& sm, int warp, int lane) {
    if (warp == 17) many_units<D, WIDE>(p, sm, lane);
    if (!WIDE && warp == 19) many_ranges<D>(p, sm, lane);
    if (warp == 16 || warp == 18) {
        const int t = (warp - 16) >> 1;
        many_products<D, WIDE>(sm, t, lane);
        __syncwarp();
        if (elect_one()) {
            int gave_up = 0;  // nothing is in flight when tensor memory is given back, whatever happened
            tc_commit(&sm.drained[t]);
            mbar_wait(&sm.drained[t], 0, &gave_up);
        }
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kManyThreads, 1) attend_many_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ __align__(1024) uint8_t dynamic_many[];
    ManyShared<D>& sm = *reinterpret_cast<ManyShared<D>*>(
        dynamic_many + ((1024 - (smem_u32(dynamic_many) & 1023)) & 1023));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        many_init(sm, false, kUnitReaders + 1);  // and the warp that looks at the scales
        sm.abort = 0, sm.redo_any = 0;
    }
    if (threadIdx.x < sizeof(sm.redo) / 4) reinterpret_cast<uint32_t*>(sm.redo)[threadIdx.x] = 0;
    if (warp == 16) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    {
        const Place place = find_place<kManyThreads>(p, kManyShift, blockIdx.x, sm.place);
        if (threadIdx.x == 0) sm.start = place;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
        setmaxnreg_inc<kSoftmaxRegs>();
        many_softmax<D, false>(p, sm, warp >> 2, threadIdx.x & 127);
        if (many_again(sm)) many_softmax<D, true>(p, sm, warp >> 2, threadIdx.x & 127);
    } else if (warp < 12) {
        setmaxnreg_dec<kCodeRegs>();
        many_keys<D, false>(p, sm, warp - 8, lane);
        if (many_again(sm)) many_keys<D, true>(p, sm, warp - 8, lane);
    } else if (warp < 16) {
        setmaxnreg_dec<kCodeRegs>();
        many_values<D, false>(p, sm, warp - 12, lane);
        if (many_again(sm)) many_values<D, true>(p, sm, warp - 12, lane);
    } else {
        setmaxnreg_dec<kIssueRegs>();
        many_issue<D, false>(p, sm, warp, lane);
        if (many_again(sm)) many_issue<D, true>(p, sm, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(sm.tmem, 512);
}

// Joins the parts of the units that were cut: CTA (i, y) those of the unit that range i ends in.  SPREAD: row y, its
// parts spread over the warps (few rows of many parts); otherwise a warp a row (many rows of two or three).
template <int D, bool SPREAD>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kElems = D / 32, kWarps = SPREAD ? 4 : 1;  // elements of a lane, neighbours; warps of a row
    __shared__ float o_s[kWarps][D];
    __shared__ float2 ml_s[kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CutUnit u = p.cuts[blockIdx.x];
    const int r = SPREAD ? blockIdx.y : blockIdx.y * 4 + warp;
    if (u.parts == 0 || r >= u.nrows) return;
    // the first part is what its CTA's range ends in (slot 1), the others are what theirs begin with (slot 0)
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 2 * p.tile_rows + r;
    auto place_of = [&](int k) { return at + static_cast<int64_t>(k) * 2 * p.tile_rows + (k == 0 ? p.tile_rows : 0); };
    const int k0 = SPREAD ? warp : 0;
    float m = -INFINITY, total = 0.0f, o[kElems] = {};
    for (int base = k0; base < u.parts; base += 32 * kWarps) {  // up to 32 parts at a time, one a lane
        const int mine = base + kWarps * lane;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (mine < u.parts) ml = __ldcg(&p.part_ml[place_of(mine)]);
        float top = ml.x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        if (top > m) {
            const float shift = m == -INFINITY ? 0.0f : exp2_approx(m - top);
            total *= shift;
#pragma unroll
            for (int j = 0; j < kElems; ++j) o[j] *= shift;
            m = top;
        }
        const float w = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - m) * ml.y;
        const int n = min(32, (u.parts - base + kWarps - 1) / kWarps);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const float* src = p.part_o + place_of(base + kWarps * k) * D + kElems * lane;
            float x[kElems];
            if constexpr (kElems == 4)
                *reinterpret_cast<float4*>(x) = __ldcg(reinterpret_cast<const float4*>(src));
            else
                *reinterpret_cast<float2*>(x) = __ldcg(reinterpret_cast<const float2*>(src));
            total += wk;
#pragma unroll
            for (int j = 0; j < kElems; ++j) o[j] += wk == 0.0f ? 0.0f : wk * x[j];
        }
    }
    if constexpr (SPREAD) {
        if (lane == 0) ml_s[warp] = make_float2(m, total);
#pragma unroll
        for (int j = 0; j < kElems; ++j) o_s[warp][kElems * lane + j] = o[j];
        __syncthreads();
        if (warp) return;
        m = fmaxf(fmaxf(ml_s[0].x, ml_s[1].x), fmaxf(ml_s[2].x, ml_s[3].x));
        total = 0.0f;
#pragma unroll
        for (int j = 0; j < kElems; ++j) o[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float w = ml_s[k].x == -INFINITY ? 0.0f : exp2_approx(ml_s[k].x - m);
            total += w * ml_s[k].y;
#pragma unroll
            for (int j = 0; j < kElems; ++j) o[j] += w == 0.0f ? 0.0f : w * o_s[k][kElems * lane + j];
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
    const int qi = (u.r0 + r) / p.G;
    const int64_t row = (u.row0 + qi) * p.Hq + u.kvh * p.G + (u.r0 + r) - qi * p.G;
    uint16_t* dst = p.out + row * D + kElems * lane;
#pragma unroll
    for (int j = 0; j < kElems; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = pack_bf16(o[j], o[j + 1]);
    if (p.lse && lane == 0) p.lse[row] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
}

// ------------------------------------------------------------------------------------ host side

constexpr int64_t kMaxKeys = int64_t{1} << 30;  // of a sequence: positions and block ends stay in 32 bits

// How a call is split, from what the host knows (not the sequences' lengths).
// attend_few_kernel takes up to 16 query rows of a unit always; up to kFewMost for heads of 64, and for heads of 128 where
// the sequences' tables (or windows) and kv heads together have room for kFewKeys keys: its 32-row tiles are bound by
// latency, the tiles of 256 of attend_many_kernel by the empty rows.  Device times of a call, few against many, 1 to 64
// sequences of 300 to 16000 keys, 1 and 8 kv heads, 20 and 32 rows, equal and ragged lengths, a window of 1024:
//   heads of 64    few faster in 55 of 76 cases, up to 2.3 times (24 sequences of 300 keys, 8 kv heads: 21.5 / 37.6 us),
//                  many in the others up to 1.14 times (one sequence of 4000: 26.7 / 23.8 us)
//   heads of 128   8 kv heads, 4 sequences of 4000: 44.7 / 44.9 us, 12: 83.7 / 87.3, 24: 120 / 143, 64: 253 / 340; 4 of 16000: 88 / 98;
//                  1 kv head, 24 of 16000: 80 / 79, 64: 133 / 175; below some 2^19 keys many is faster (64 sequences of 4000,
//                  1 kv head: 73 / 66; 1 to 24 of 300: 37 / 26).  What the host does not see are ragged lengths: 24 sequences
//                  of 500 to 4000 keys, 8 kv heads, 118 / 96 us, are taken for full ones.
// 64 rows (24 sequences of 4000 keys, tiles of 32 read the keys twice): 202 / 144 us.
constexpr int kFewMost = 32;
constexpr int64_t kFewKeys = int64_t{1} << 19;
// Keys of a sequence's table up to which few rows are not cut (one query, 64 heads on 8: 48 sequences of 500 keys 14.8
// against 23.5 us, 32 of 1000 keys 19.9 against 23.9 us, one of 1000 keys 13.4 against 12.5 us).
constexpr int64_t kWholeKeys = 1024;
struct AttendPlan {
    int tile_rows, row_tiles, ctas, unit_cost;
    int64_t units;
    size_t bytes;
};
static AttendPlan plan_attend(int64_t B, int Hq, int Hk, int D, int64_t max_q, int64_t keys, int64_t window) {
    AttendPlan a = {};
    const int64_t rows = max_q * (Hq / Hk);
    const int64_t seen = window && window < keys - max_q ? window + max_q : keys;
    const bool few32 = rows <= kFewMost && (D == 64 || (seen > 0 && B * Hk >= (kFewKeys + seen - 1) / seen));
    a.tile_rows = rows <= 8 ? 8 : rows <= 16 ? 16 : few32 ? 32 : kManyRows;
    a.row_tiles = static_cast<int>((rows + a.tile_rows - 1) / a.tile_rows);
    if (B > kMaxDim / (static_cast<int64_t>(Hk) * a.row_tiles)) return a;  // units are counted in 31 bits
    a.units = B * Hk * a.row_tiles;
    if (a.tile_rows == kManyRows) {
        a.ctas = sm_count();
        a.unit_cost = 4;
    } else {
        // Cut while there are few units.  Many fill the GPU whole, and need no joining (256 sequences of 4000 keys, 64
        // heads on 8: 232 / 251 us; of 500 to 4000 keys, four queries, 32 on 8: 253 / 288) unless one is far longer than
        // all others, which the host does not see (300 sequences of 200 keys and one of 100000: 601 / 84 us).
        const int resident = sm_count() * few_resident(a.tile_rows / 8);
        a.ctas = a.units >= 4 * resident || keys <= kWholeKeys ? 0 : resident;
        a.unit_cost = 16;
    }
    a.bytes = static_cast<size_t>(a.ctas) * (2 * a.tile_rows * (static_cast<size_t>(D) * 4 + 8) + sizeof(CutUnit));
    a.bytes = (a.bytes + 255) / 256 * 256 + 256;
    return a;
}

template <int D, int NT>
static int launch_few(const AttendParams& p, unsigned blocks, cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(FewShared<D, NT>);
    static_assert(few_resident(NT) * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    static int cache[64] = {0};
    const int ready = cached_per_device(cache, [] {
        return cudaFuncSetAttribute(attend_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess
                   ? 1
                   : -1;
    });
    if (!ready) return MACAQ_ECUDA;
    return launch_dependent_smem(attend_few_kernel<D, NT>, dim3(blocks), kFewThreads, kSmem, stream, p);
}

template <int D>
static int launch_many(const AttendParams& p, cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(ManyShared<D>) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
    // setmaxnreg.inc takes registers from those the CTA was launched with: with fewer it would wait forever
    static int cache[64] = {0};
    const int ready = cached_per_device(cache, [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, attend_many_kernel<D>) == cudaSuccess && fa.numRegs >= kManyLaunchRegs &&
                       cudaFuncSetAttribute(attend_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
                           cudaSuccess
                   ? 1
                   : -1;
    });
    if (!ready) return MACAQ_ECUDA;
    return launch_dependent_smem(attend_many_kernel<D>, dim3(p.ctas), kManyThreads, kSmem, stream, p);
}

template <int D>
static int launch_attend(const AttendParams& p, int64_t units, cudaStream_t stream) {
    const auto n = static_cast<unsigned>(p.ctas ? p.ctas : units);
    const int st = p.tile_rows == kManyRows ? launch_many<D>(p, stream)
                   : p.tile_rows == 8  ? launch_few<D, 1>(p, n, stream)
                   : p.tile_rows == 16 ? launch_few<D, 2>(p, n, stream)
                                       : launch_few<D, 4>(p, n, stream);
    if (st != MACAQ_OK || p.ctas < 2) return st;
    if (p.tile_rows == kManyRows)
        return launch_dependent(attend_join_kernel<D, false>, dim3(p.ctas - 1, kManyRows / 4), 128, stream, p);
    return launch_dependent(attend_join_kernel<D, true>, dim3(p.ctas - 1, p.tile_rows), 128, stream, p);
}

}  // namespace macaq

extern "C" size_t macaq_kv4_attention_workspace_bytes(int64_t T, int64_t B, int Hq, int Hk, int head_dim, int64_t max_q) {
    if (!head_dim_ok(head_dim) || T < 0 || T > kMaxDim || B < 0 || B > kMaxDim || Hk < 1 || Hq < Hk || Hq > kMaxHeads ||
        Hq % Hk != 0 || max_q < 1 || max_q > kMaxDim / kMaxHeads)
        return 0;
    if (T == 0 || B == 0) return 256;
    // whatever the tables' width
    const size_t a = plan_attend(B, Hq, Hk, head_dim, max_q, 0, 0).bytes;
    const size_t z = plan_attend(B, Hq, Hk, head_dim, max_q, kMaxKeys, 0).bytes;
    return a && z ? (a > z ? a : z) : 0;
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
    const AttendPlan plan = plan_attend(B, Hq, Hk, head_dim, max_q, table_width * page_size, window);
    AttendParams p = {};
    p.q = q, p.T = T, p.ldq = ldq, p.Hq = Hq, p.Hk = Hk, p.G = Hq / Hk, p.cache = cache, p.num_pages = num_pages;
    p.page_size = page_size, p.page_shift = __builtin_ctz(page_size), p.tables = tables, p.table_width = table_width;
    p.kv_lens = kv_lens, p.cu_q = cu_q, p.B = static_cast<int>(B), p.max_q = static_cast<int>(max_q);
    p.scale_log2 = scale * kLog2e, p.window = static_cast<int>(window < kMaxDim ? window : 0), p.out = out, p.lse = lse;
    p.tile_rows = plan.tile_rows, p.row_tiles = plan.row_tiles, p.ctas = plan.ctas;
    p.unit_cost = plan.unit_cost;
    p.cuts = static_cast<CutUnit*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.cuts + p.ctas);
    p.part_o = reinterpret_cast<float*>(p.part_ml + static_cast<int64_t>(p.ctas) * 2 * p.tile_rows);
    const auto s = static_cast<cudaStream_t>(stream);
    return head_dim == 64 ? launch_attend<64>(p, plan.units, s) : launch_attend<128>(p, plan.units, s);
}
