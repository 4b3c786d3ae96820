// Paged 8-bit key/value cache: writing new tokens, and attention of a few new
// queries per sequence over it.
//
// A page holds page_size tokens of every key/value head as OCP E4M3 codes, with
// one fp32 scale per page, head and tensor: the value is scale * code.
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// One block per (touched page, head, K or V).  The page's scale is the power of
// two 2^e with the smallest e >= kMinScaleExp such that the largest finite new
// magnitude is at most 448 * 2^e, or the scale it has where older tokens are in
// it and that one is large enough; where it has to grow, the older codes are
// rounded again to the new scale (exact for a power of two, but for codes that
// fall below E4M3's normal range).  Dividing by a power of two is exact, so a
// new code carries one rounding, to nearest even, saturating at 448.
// Bound by reading the new tokens, which stay in registers between the two looks at them
// (read twice they cost a quarter more), and by issue: magnitudes are compared two at a time
// as integers, and the quotient's correction is left out where the scale is a power of two
// (without both a quarter more again).  4 prompts of up to 8192 tokens, 8 heads, d = 128: 23
// us among other calls, 5.8 TB/s, 20 in a row; d = 64 16 in a row, 4.2 TB/s; one token for 32
// sequences 3 us in a row.
constexpr int kAppendThreads = 128;
constexpr int kMinScaleExp = -100;

// Smallest power of two s >= 2^kMinScaleExp with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float append_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>(max(e, kMinScaleExp) + 127) << 23);
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads, 8) cache_append_kernel(const CacheAppendParams p) {
    constexpr int TPR = D / 8;  // threads per token: 8 elements each
    constexpr int RPP = kAppendThreads / TPR;
    pdl_wait();
    const int hk = blockIdx.y, b = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int page = p.c.page_size;
    const int len = p.c.seq_lens[b];
    const int m = p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
    if (blockIdx.x == 0 && hk == 0 && !is_v && threadIdx.x == 0) check_len(p.c, p.st, b);
    if (m == 0 || len <= 0) return;
    const int first = len - m;  // position of new token 0 (negative: it is not written)
    const int pg = max(first, 0) / page + static_cast<int>(blockIdx.x);
    if (pg >= p.c.max_pages) return;  // behind the table; below it positions stay far inside 32 bits
    const int lo = max(first, pg * page), hi = min(len, pg * page + page);  // new positions in this page
    if (lo >= hi) return;
    const int pid = __ldg(p.c.table + b * p.c.table_stride + pg);
    if (static_cast<unsigned>(pid) >= static_cast<unsigned>(p.c.num_pages)) {
        if (threadIdx.x == 0) record_device_error(p.st, ATTN_DEVERR_PAGE, 0x303);
        return;
    }
    const Strides cs = is_v ? p.c.vs : p.c.ks, xs = is_v ? p.vs : p.ks;
    const int c8 = threadIdx.x % TPR * 8, rr = threadIdx.x / TPR;
    uint8_t* codes = (is_v ? p.c.v_pages : p.c.k_pages) + pid * cs.b + hk * cs.h + c8;
    const uint16_t* x = static_cast<const uint16_t*>(is_v ? p.v : p.k) + b * xs.b + hk * xs.h + c8;
    float* scale = (is_v ? p.c.v_scale : p.c.k_scale) + static_cast<long long>(pid) * p.Hk + hk;
    const float was = *scale;

    // The first kHeld tokens of each thread stay in registers between the two looks at them.
    constexpr int kHeld = 8;
    uint4 held[kHeld];
    const int n = hi - lo;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        held[k] = make_uint4(0u, 0u, 0u, 0u);
        if (rr + k * RPP < n) held[k] = __ldcs(reinterpret_cast<const uint4*>(x + (lo + rr + k * RPP - first) * xs.n));
    }
    // Magnitudes of bf16 order as their bit patterns: two at a time, one integer maximum a warp.
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    auto largest = [&](auto halves) -> uint32_t {  // of the block's new values, each word's halves given by `halves`
        uint32_t m = 0u;
        auto look = [&](const uint4& w) {
            for (uint32_t u : {w.x, w.y, w.z, w.w}) m = __vmaxu2(m, halves(u & 0x7FFF7FFFu));
        };
#pragma unroll
        for (int k = 0; k < kHeld; ++k) look(held[k]);
        for (int t = rr + kHeld * RPP; t < n; t += RPP) look(*reinterpret_cast<const uint4*>(x + (lo + t - first) * xs.n));
        const uint32_t wm = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu));
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = wm;
        __syncthreads();  // and every thread has read the old scale
        return max(max(warp_max[0], warp_max[1]), max(warp_max[2], warp_max[3]));
    };
    uint32_t top = largest([](uint32_t u) { return u; });
    if (top >= 0x7F80u) {  // infinities or NaN: the largest finite magnitude counts
        __syncthreads();
        top = largest([](uint32_t u) { return u & ~__vcmpgeu2(u, 0x7F807F80u); });
    }
    const float amax = __uint_as_float(top << 16);
    const int old = lo - pg * page;  // tokens that the page holds already
    const bool keep = old > 0 && was >= __uint_as_float((kMinScaleExp + 127) << 23) && amax <= 448.f * was;
    const float s = keep ? was : append_scale(amax);
    if (old > 0 && !keep) {
        const float f = was > 0.f ? was / s : 0.f;
        for (int t = rr; t < old; t += RPP) {
            uint2* at = reinterpret_cast<uint2*>(codes + t * cs.n);
            uint2 w = *at;
            uint32_t r[2] = {w.x, w.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a0, a1, a2, a3;
                uint32_t h01, h23;
                e4m3x4_to_f16(r[i], h01, h23);
                asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                    : "=f"(a0), "=f"(a1) : "r"(h01));
                asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                    : "=f"(a2), "=f"(a3) : "r"(h23));
                r[i] = pack_e4m3x4(a0 * f, a1 * f, a2 * f, a3 * f);
            }
            *at = make_uint2(r[0], r[1]);
        }
    }
    // x / s rounded once: a power of two's inverse is exact; for another scale (one that was
    // there) the remainder of the product puts it right, as it would not change the former.  Beyond 448 the code saturates.
    const float inv = 1.f / s;
    auto quotient = [&](float v) {
        const float q = v * inv;
        return fabsf(q) <= 448.f ? fmaf(fmaf(-q, s, v), inv, q) : q;
    };
    auto put_all = [&](auto code) {
        auto put = [&](int t, const uint4& w) {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                c[i] = pack_e4m3x4(code(bf16lo(u[2 * i])), code(bf16hi(u[2 * i])), code(bf16lo(u[2 * i + 1])),
                                   code(bf16hi(u[2 * i + 1])));
            *reinterpret_cast<uint2*>(codes + (old + t) * cs.n) = make_uint2(c[0], c[1]);
        };
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (rr + k * RPP < n) put(rr + k * RPP, held[k]);
        for (int t = rr + kHeld * RPP; t < n; t += RPP)
            put(t, *reinterpret_cast<const uint4*>(x + (lo + t - first) * xs.n));
    };
    if ((__float_as_uint(s) & 0x7FFFFFu) == 0u) put_all([&](float v) { return v * inv; });
    else put_all(quotient);
    if (threadIdx.x == 0 && !keep) *scale = s;
}

// ---------------------------------------------------------------------------
// Attention of a few queries: work shared out evenly
// ---------------------------------------------------------------------------
// An item is (sequence, key/value head, tile of p.rows query rows); the rows of a
// key/value head are its H/Hk query heads of every new query, row = t * H/Hk + g.
// An item's blocks of kBlock tokens are laid end to end over all items, and CTA c
// of G takes the c-th of G equal shares of that line, whatever the lengths of the
// sequences are: lengths stay on the device.  A share can begin and end inside
// an item; such unfinished segments go to the workspace and a second kernel joins
// them.  At most two per CTA: slot 2c for a segment that does not start its item,
// slot 2c + 1 for one that starts it and does not reach its end.  (Where there is a CTA
// for every item and the longest item is at most a quarter above an equal share, each
// CTA takes one item whole.)
constexpr int kTok = 16;    // tokens of a tile: M of a score product, K of an output product
constexpr int kBlock = 32;  // tokens of a block: two tiles, which may lie in different pages
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// A share has at least this many blocks: with fewer, joining costs more than the
// shorter walk gives.
constexpr int kMinShare = 4;

struct Share {
    long long total, share;
    int whole;          // > 0: every item counts as that many blocks and is one share
    int b;              // sequence that holds the start of the share; -1: there is none
    long long b_first;  // blocks before that sequence
};

struct ShareSmem {
    long long work[kWarps], b_first;
    int items[kWarps], longest[kWarps], b;
};

__device__ __forceinline__ int row_tiles(const CacheFwdParams& p, const CacheSeq& s) {
    return (s.q_len * (p.H / p.Hk) + p.rows - 1) / p.rows;
}
// Blocks of a sequence's items (whole: see Share).
__device__ __forceinline__ long long seq_work(const CacheFwdParams& p, const CacheSeq& s, int whole) {
    return static_cast<long long>(whole > 0 ? whole : s.n) * (row_tiles(p, s) * p.Hk);
}

// Shares of a line of `total` blocks in which all_items items lie; their start is still to be found.
__device__ __forceinline__ Share equal_shares(const CacheFwdParams& p, long long total, int all_items, int longest) {
    Share s;
    s.total = total;
    s.share = max(div_mostly32(total + p.grid - 1, p.grid), static_cast<long long>(kMinShare));
    s.whole = all_items <= p.grid && 4ll * longest <= 5ll * s.share ? longest : 0;
    if (s.whole > 0) {
        s.share = s.whole;
        s.total = static_cast<long long>(all_items) * s.whole;
    }
    return s;
}

// Lays the items of all sequences end to end and finds the sequence at the start
// of share c (a slice of the sequences per thread).
__device__ Share find_share(const CacheFwdParams& p, int c, ShareSmem* sm) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    long long work = 0;
    int items = 0, longest = 0;
    for (int b = b0; b < b1; ++b) {
        const CacheSeq q = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b);
        if (blockIdx.x == 0) check_len(p.c, p.st, b);
        work += seq_work(p, q, 0);
        items = min(items + row_tiles(p, q) * p.Hk, 1 << 20);
        if (q.q_len > 0) longest = max(longest, q.n);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long work_to = work;
    int items_to = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, work_to, o);
        const int n = __shfl_up_sync(0xffffffffu, items_to, o);
        if (lane >= o) work_to += w, items_to += n;
    }
    if (lane == 31) {
        sm->work[warp] = work_to;
        sm->items[warp] = items_to;
        sm->longest[warp] = longest;
    }
    if (threadIdx.x == 0) sm->b = -1;
    __syncthreads();
    long long total = 0;
    int all_items = 0, items_before = items_to - items;
    long long work_before = work_to - work;
    longest = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) work_before += sm->work[w], items_before += sm->items[w];
        total += sm->work[w];
        all_items += sm->items[w];
        longest = max(longest, sm->longest[w]);
    }
    Share s = equal_shares(p, total, all_items, longest);
    if (s.whole > 0) {
        work = static_cast<long long>(items) * s.whole;
        work_before = static_cast<long long>(items_before) * s.whole;
    }
    const long long x = c * s.share;
    if (x < s.total && work_before <= x && x < work_before + work) {
        for (int b = b0; b < b1; ++b) {
            const long long w = seq_work(p, cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b), s.whole);
            if (x < work_before + w) {
                sm->b = b;
                sm->b_first = work_before;
                break;
            }
            work_before += w;
        }
    }
    __syncthreads();
    s.b = sm->b;
    s.b_first = sm->b_first;
    return s;
}

// The same by each warp for itself, without a barrier: 26.8 us for 28.6 and 39.2 for 41.1
// (16 x 4096 tokens, 24 and 64 rows) with up to 64 sequences; with more the block's threads
// share the reading of the lengths (1024 sequences: 88 us, each warp for itself 107).
constexpr int kFewSeqs = 64;
__device__ __forceinline__ Share find_share_few(const CacheFwdParams& p, int c) {
    const int lane = threadIdx.x & 31, per = (p.B + 31) >> 5;
    const int b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
    long long work = 0;
    int items = 0, longest = 0;
    for (int b = b0; b < b1; ++b) {
        const CacheSeq q = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b);
        if (blockIdx.x == 0 && threadIdx.x < 32) check_len(p.c, p.st, b);
        const int n = row_tiles(p, q) * p.Hk;
        work += static_cast<long long>(q.n) * n;
        items = min(items + n, 1 << 20);
        if (q.q_len > 0) longest = max(longest, q.n);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    long long work_to = work;
    int items_to = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, work_to, o);
        const int n = __shfl_up_sync(0xffffffffu, items_to, o);
        if (lane >= o) work_to += w, items_to += n;
    }
    Share s = equal_shares(p, __shfl_sync(0xffffffffu, work_to, 31), __shfl_sync(0xffffffffu, items_to, 31), longest);
    long long before = work_to - work;
    if (s.whole > 0) {
        work = static_cast<long long>(items) * s.whole;
        before = static_cast<long long>(items_to - items) * s.whole;
    }
    const long long x = c * s.share;
    int found = -1;
    if (x < s.total && before <= x && x < before + work) {
        for (int b = b0; b < b1; ++b) {
            const long long w = seq_work(p, cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b), s.whole);
            if (x < before + w) {
                found = b;
                break;
            }
            before += w;
        }
    }
    const unsigned who = __ballot_sync(0xffffffffu, found >= 0);
    const int src = who ? __ffs(who) - 1 : 0;
    s.b = __shfl_sync(0xffffffffu, found, src);
    s.b_first = __shfl_sync(0xffffffffu, before, src);
    return s;
}

// Row r (0 .. p.rows - 1) of row tile rt of a sequence: query and head of the group.
struct RowAt {
    int t, h;
    bool there;
};
__device__ __forceinline__ RowAt row_at(const CacheFwdParams& p, int q_len, int hk, int rt, int r) {
    const int G = p.H / p.Hk, row = rt * p.rows + r;
    RowAt a;
    a.t = row / G;
    a.h = hk * G + row - a.t * G;
    a.there = a.t < q_len;
    return a;
}

// ---------------------------------------------------------------------------
// Attention of a few queries: the kernel
// ---------------------------------------------------------------------------
// Bound by reading the codes once: 64 sequences of up to 8192 tokens, 32/8 heads, d = 128,
// one query each: 124 us, 6.4 TB/s.  (With 40 rows a key/value head, 16 x 4096 tokens: 32 us
// for 7.5 of reading; three row tiles, latency in 8 warps an SM.)  Each warp walks every
// kWarps-th block of a segment on its own, with its own running maximum, sums and output;
// the codes come by asynchronous copies into a ring of its own, so no barrier stands in
// the loop.  Codes become
// f16 exactly and go to f16 matrix products with fp32 sums; Q rows are brought to
// f16 by a power of two each.  A page's scales enter in fp32: the key scale
// multiplies the scores, the value scale is added, as its log2, to the exponent,
// so that the weights given to the products are 2^(score + log2 sv - m) with the
// running maximum m taken over score + log2 sv, and the sum of the probabilities
// takes them back by 1 / sv (kScaleReach).  m is raised, and the output rescaled, only when
// a score passes it by more than kWeightSlack; a weight is lost to f16's underflow below
// 2^-31 of the largest.
//
// What belongs to a tile and not to a lane (its page's address and scales, whether
// all of it is seen) is worked out by one lane per tile for 16 blocks at a time and
// handed round by shuffles: done by every lane for every tile it took more than
// half of all instructions.
//
// Both products have the keys' side as A: S^T (16 tokens x 8 rows) = K Q^T and
// O^T (16 d x 8 rows) += V^T P^T, so that the 8 rows of a group of query heads fill
// the narrow side of the product and codes turned into f16 serve all NT groups of 8
// rows (with Q as A, 8 rows took as long as 16).  P^T goes from the layout of a
// result to that of B by an 8x8 transposition between lanes.
//
// Fragment layouts (g = lane / 4, q = lane % 4).  Contraction indices, and the order
// of d in the output, may be permuted.  K: lane (g, q) holds tokens g and g + 8 and
// the 16 consecutive d from 64 c + 16 q, of which word s gives the k-pairs
// (2q, 2q + 1) and (2q + 8, 2q + 9) of product (c, s).  V: lane (g, q) holds tokens
// 2q, 2q + 1, 2q + 8, 2q + 9 and the D/8 consecutive d from g D/8, of which 2j and
// 2j + 1 are rows g and g + 8 of product j.
//
// The copies take whole rows, 512 consecutive bytes an instruction where rows follow
// each other (each lane copying its own fragments' bytes reached 5.3 TB/s, whole rows
// 7.0), and the 16-byte pieces of a row are placed so that neither fragment's reads
// meet in a bank (chunk_at).
template <int D, int NT>
struct DecodeTraits {
    static constexpr int ROWS = 8 * NT;
    // Registers (the output takes NT D/4 a lane) admit this many CTAs of four warps to
    // an SM, and the rings share its memory.  NT = 2: with three CTAs an SM d = 64 takes
    // 33 us for 37 (32 x 4096 tokens, 8 heads, 12 rows), d = 128 spills: 37 us for 35
    // (16 x 4096, 4 heads, 40 rows).
    static constexpr int CTAS_PER_SM = NT == 1 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);
    static constexpr int STAGES = NT == 1 ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : 3);  // blocks in a warp's ring
    static constexpr int KC = D / 64;  // 16-byte pieces of a token's K row per lane
    static constexpr int VB = D / 8;   // bytes of a token's V row per lane
    static constexpr int NJ = D / 16;  // products of a tile's output
    static constexpr int ROW = D;             // bytes of a token's row
    static constexpr int LPR = ROW / 16;      // lanes that copy a row, 16 bytes each
    static constexpr int RPI = 32 / LPR;      // rows that one copy instruction of the warp takes
    static constexpr int K_BYTES = kTok * ROW, TILE = 2 * K_BYTES;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int O_PITCH = D + 4;  // floats between rows of a warp's output in shared memory
    static constexpr int WARP_BYTES = RING > ROWS * O_PITCH * 4 ? RING : ROWS * O_PITCH * 4;
    static constexpr int SMEM = kWarps * WARP_BYTES + kWarps * ROWS * 8 + static_cast<int>(sizeof(ShareSmem));
};

// Byte offset in a tile of 16-byte piece c of row r.  D = 128: pieces of a row are
// permuted by a XOR; a quarter warp then finds its eight pieces (K: four pieces of
// two neighbouring rows; V: two neighbouring pieces of rows 0, 2, 4, 6 or 1, 3, 5, 7)
// in eight different places of 16 bytes.  D = 64: the same over pairs of rows.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
    if constexpr (D == 128) return r * 128 + ((c ^ (r & 6) ^ ((r & 1) << 2)) << 4);
    else return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, DecodeTraits<D, NT>::CTAS_PER_SM) cache_decode_kernel(const CacheFwdParams p) {
    using T = DecodeTraits<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    uint8_t* my = smem + warp * T::WARP_BYTES;
    const uint32_t my_u = smem_u32(my);
    float2* stat = reinterpret_cast<float2*>(smem + kWarps * T::WARP_BYTES);  // [kWarps][ROWS]
    ShareSmem* ssm = reinterpret_cast<ShareSmem*>(stat + kWarps * T::ROWS);

    pdl_launch_dependents();
    pdl_wait();
    const Share sh = p.B <= kFewSeqs ? find_share_few(p, blockIdx.x) : find_share(p, blockIdx.x, ssm);
    if (sh.b < 0) {  // more CTAs than shares
        if (threadIdx.x == 0) p.border[blockIdx.x].c_first = -1;
        return;
    }
    const long long x_begin = blockIdx.x * sh.share;
    const long long x_end = min(x_begin + sh.share, sh.total);
    long long x = x_begin;
    int b = sh.b;
    long long b_first = sh.b_first;
    const int G = p.H / p.Hk;

    while (x < x_end) {
        CacheSeq s = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b);
        for (long long w; x >= b_first + (w = seq_work(p, s, sh.whole));) {  // next sequence with work
            b_first += w;
            s = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, ++b);
        }
        // segment [v0, v1) of the item's n blocks
        const int rts = row_tiles(p, s);
        const int counts = sh.whole > 0 ? sh.whole : s.n;
        const int item = static_cast<int>(div_mostly32(x - b_first, counts));
        const int v0 = static_cast<int>((x - b_first) - static_cast<long long>(item) * counts);
        const int v1 = static_cast<int>(min(static_cast<long long>(s.n), v0 + (x_end - x)));
        const int hk = item / rts, rt = item - hk * rts;
        const int first_pos = s.len - s.q_len;  // may be negative: rows before the first token see nothing
        if (x == x_begin && threadIdx.x == 0) {
            CacheBorder bd;
            bd.b = b;
            bd.item = item;
            bd.q_len = s.q_len;
            bd.c_first = v0 > 0 ? static_cast<int>(div_mostly32(x - v0, sh.share)) + 1 : -1;
            bd.c_last = static_cast<int>(div_mostly32(x - v0 + s.n - 1, sh.share));
            p.border[blockIdx.x] = bd;
        }

        // ---- Q rows on their way while the first blocks are found ----
        uint4 qw[NT][T::KC][2];  // row g of each group of 8
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const RowAt a = row_at(p, s.q_len, hk, rt, 8 * n + g);
            const uint16_t* qrow = static_cast<const uint16_t*>(p.q) + b * p.qs.b + a.h * p.qs.h + a.t * p.qs.n + q * 16;
#pragma unroll
            for (int c = 0; c < T::KC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qw[n][c][e] = a.there ? *reinterpret_cast<const uint4*>(qrow + c * 64 + e * 8)
                                          : make_uint4(0u, 0u, 0u, 0u);
        }

        const int crow = lane / T::LPR, cchunk = lane % T::LPR;  // this lane's piece of a copy instruction
        const uint8_t* kbase = p.c.k_pages + hk * p.c.ks.h + crow * p.c.ks.n + cchunk * 16;
        const uint8_t* vbase = p.c.v_pages + hk * p.c.vs.h + crow * p.c.vs.n + cchunk * 16;
        const long long kn = p.c.ks.n, vn = p.c.vs.n;
        const int n_my = (v1 - v0 - warp + kWarps - 1) / kWarps;  // blocks of this warp
        // token of the sequence seen by some query
        auto seen = [&](int j) { return j < s.len && (j >= s.key_lo || j < p.sinks); };

        // ---- tiles of 16 blocks at a time, one per lane: lane 2i + u holds tile u of block i ----
        long long koff = 0, voff = 0;          // byte offsets of the tile's first token, for the copies
        uint32_t loadable = 0;                 // tiles all of whose tokens some query sees
        float sk_next = 1.f, sv_next = 1.f;    // scales, one batch ahead of their use
        uint32_t whole_next = 0;
        auto batch = [&](int i0) {
            const int i = i0 + (lane >> 1);
            int tok = 0;
            bool all = false, whole = false;
            koff = voff = 0;
            sk_next = sv_next = 1.f;
            if (i < n_my) {
                tok = cache_block(s, v0 + warp + kWarps * i) * kBlock + (lane & 1) * kTok;
                if (tok < s.len && (tok + kTok > s.key_lo || tok < p.sinks)) {
                    const int pid = cache_page(p.c, p.st, b, tok);
                    const int slot = tok & (p.c.page_size - 1);
                    koff = pid * p.c.ks.b + slot * kn;
                    voff = pid * p.c.vs.b + slot * vn;
                    const long long at = static_cast<long long>(pid) * p.Hk + hk;
                    sk_next = __ldg(p.c.k_scale + at);
                    sv_next = __ldg(p.c.v_scale + at);
                    all = tok + kTok <= s.len && (tok >= s.key_lo || tok + kTok <= p.sinks);
                    // every query sees all of the tile
                    whole = tok + kTok - 1 <= first_pos &&
                            (p.left < 0 || tok >= s.len - 1 - p.left || tok + kTok <= p.sinks);
                }
            }
            loadable = __ballot_sync(0xffffffffu, all);
            whole_next = __ballot_sync(0xffffffffu, whole);
        };
        auto issue = [&](int i, int stage) {
            if (i < n_my) {
                if ((i & 15) == 0) batch(i);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int src = (2 * i + u) & 31;
                    const uint8_t* kp = kbase + __shfl_sync(0xffffffffu, koff, src);
                    const uint8_t* vp = vbase + __shfl_sync(0xffffffffu, voff, src);
                    const uint32_t dst = my_u + stage * T::STAGE + u * T::TILE;
                    if ((loadable >> src) & 1u) {
#pragma unroll
                        for (int k = 0; k < kTok; k += T::RPI) cp_async16(dst + chunk_at<D>(crow + k, cchunk), kp + k * kn);
#pragma unroll
                        for (int k = 0; k < kTok; k += T::RPI)
                            cp_async16(dst + T::K_BYTES + chunk_at<D>(crow + k, cchunk), vp + k * vn);
                    } else {  // tokens that no query sees are not read: zeros stand for them
                        const int tok = cache_block(s, v0 + warp + kWarps * i) * kBlock + u * kTok;
#pragma unroll
                        for (int k = 0; k < kTok; k += T::RPI) {
                            const bool there = seen(tok + crow + k);
                            const int at = chunk_at<D>(crow + k, cchunk);
                            cp_async16(dst + at, there ? kp + k * kn : kbase, there);
                            cp_async16(dst + T::K_BYTES + at, there ? vp + k * vn : vbase, there);
                        }
                    }
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < T::STAGES - 1; ++i) issue(i, i);

        // ---- Q: row g of each group of 8 as f16, times a power of two ----
        uint32_t qb[NT][T::KC * 4][2];
        float rq[NT][2];  // rows 2q and 2q + 1: scale * log2 e over that power
        int pos[NT][2];   // and their positions
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 (&w)[T::KC][2] = qw[n];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < T::KC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    for (uint32_t u : {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w})
                        amax = fmaxf(amax, fmaxf(fabsf(bf16lo(u)), fabsf(bf16hi(u))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float f = f16_row_scale(amax);
#pragma unroll
            for (int c = 0; c < T::KC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t u[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // elements 8e + 2k, 8e + 2k + 1 of the lane's 16: product 2e + k/2
                        qb[n][c * 4 + 2 * e + (k >> 1)][k & 1] = pack_f16x2(bf16lo(u[k]) * f, bf16hi(u[k]) * f);
                }
            const float rf = p.cs * __uint_as_float((254u << 23) - __float_as_uint(f));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rq[n][e] = __shfl_sync(0xffffffffu, rf, (2 * q + e) * 4);
                pos[n][e] = first_pos + row_at(p, s.q_len, hk, rt, 8 * n + 2 * q + e).t;
            }
        }

        float o[NT][T::NJ][4];  // (row 2q, 2q + 1 at d 2j; row 2q, 2q + 1 at d 2j + 1) of the lane's D/8
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < T::NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
        float sk = 1.f, lsv = 0.f, isv = 1.f;  // of this lane's tile of the batch in use
        uint32_t whole = 0, far = 0;           // far: tiles whose value scale is beyond kScaleReach
        auto row_sees = [&](int ps, int j) { return j <= ps && (p.left < 0 || j >= ps - p.left || j < p.sinks); };

        int stage = 0;
        auto next_batch = [&]() {  // batch i / 16, whose loads went out with its first copies
            sk = sk_next;
            lsv = lg2_approx(sv_next);
            isv = rcp_approx(sv_next);
            whole = whole_next;
            far = __ballot_sync(0xffffffffu, !(fabsf(lsv) <= kScaleReach));
        };
        // apart_tag: a second copy of the code for walks with far value scales, whose sums (of 2^u)
        // are in stat, so that the first has nothing more to hold
        auto step = [&](auto apart_tag, int i) {
            constexpr bool apart = decltype(apart_tag)::value;
            cp_async_wait<T::STAGES - 2>();
            __syncwarp();  // block i is there for every lane, and block i - 1 has been read
            issue(i + T::STAGES - 1, stage == 0 ? T::STAGES - 1 : stage - 1);
            const uint8_t* src = my + stage * T::STAGE;
            stage = stage + 1 == T::STAGES ? 0 : stage + 1;

            // ---- scores of 2 x 16 tokens and NT x 8 rows ----
            float sf[2][NT][4];  // tokens g, g, g + 8, g + 8; rows 2q, 2q + 1, 2q, 2q + 1
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sf[u][n][e] = 0.f;
#pragma unroll
            for (int c = 0; c < T::KC; ++c) {
                uint4 w[2][2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        w[u][k] = *reinterpret_cast<const uint4*>(src + u * T::TILE + chunk_at<D>(8 * k + g, 4 * c + q));
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        auto word = [&](const uint4& x) { return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w; };
                        uint32_t ka[4];
                        e4m3x4_to_f16(word(w[u][0]), ka[0], ka[2]);
                        e4m3x4_to_f16(word(w[u][1]), ka[1], ka[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(sf[u][n], ka, qb[n][c * 4 + k][0], qb[n][c * 4 + k][1]);
                    }
            }
            const int src0 = (2 * i) & 31;
            const bool all_seen = ((whole >> src0) & 3u) == 3u;
            const int tok = cache_block(s, v0 + warp + kWarps * i) * kBlock;
            if (!all_seen) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!row_sees(pos[n][e & 1], tok + u * kTok + g + 8 * (e >> 1))) sf[u][n][e] = -INFINITY;
            }
            float t_sk[2], t_lsv[2], t_isv[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                t_sk[u] = __shfl_sync(0xffffffffu, sk, src0 + u);
                t_lsv[u] = __shfl_sync(0xffffffffu, lsv, src0 + u);
                t_isv[u] = __shfl_sync(0xffffffffu, isv, src0 + u);
            }
            if constexpr (apart) {  // ---- the sums ----
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float2* const at = stat + warp * T::ROWS + 8 * n + 2 * q + r;
                        const float2 us = *at;
                        const float f0 = score_factor(rq[n][r], t_sk[0]), f1 = score_factor(rq[n][r], t_sk[1]);
                        const float s0 = sf[0][n][r] * f0, s1 = sf[0][n][2 + r] * f0;
                        const float s2 = sf[1][n][r] * f1, s3 = sf[1][n][2 + r] * f1;
                        float u = fmaxf(fmaxf(s0, s1), fmaxf(s2, s3));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, x));
                        u = fmaxf(u, us.x);
                        const float sub = u == -INFINITY ? 0.f : u;
                        float sum = ex2_approx(s0 - sub) + ex2_approx(s1 - sub) + ex2_approx(s2 - sub) + ex2_approx(s3 - sub);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                        __syncwarp();
                        if (g == 0) *at = make_float2(u, fmaf(us.y, us.x == u ? 1.f : ex2_approx(us.x - u), sum));
                        __syncwarp();
                    }
            }
            // ---- score + log2 sv, and the running maximum ----
            bool passes = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float f = score_factor(rq[n][r], t_sk[u]);
                        sf[u][n][r] = fmaf(sf[u][n][r], f, t_lsv[u]);
                        sf[u][n][2 + r] = fmaf(sf[u][n][2 + r], f, t_lsv[u]);
                    }
                    const float mx = fmaxf(fmaxf(sf[0][n][r], sf[0][n][2 + r]), fmaxf(sf[1][n][r], sf[1][n][2 + r]));
                    passes |= mx > m[n][r] + kWeightSlack;
                }
            if (__any_sync(0xffffffffu, passes)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float mx = fmaxf(fmaxf(sf[0][n][r], sf[0][n][2 + r]), fmaxf(sf[1][n][r], sf[1][n][2 + r]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                        mx = fmaxf(m[n][r], mx);
                        const float alpha = mx == m[n][r] ? 1.f : ex2_approx(m[n][r] - mx);  // 0 while m is -inf
                        m[n][r] = mx;
                        l[n][r] *= alpha;
#pragma unroll
                        for (int j = 0; j < T::NJ; ++j) {
                            o[n][j][r] *= alpha;
                            o[n][j][2 + r] *= alpha;
                        }
                    }
            }
            // ---- weights: f16 (half a step, 2^-11 relative), finer than the bf16 output ----
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float sub0 = kWeightShift - (m[n][0] == -INFINITY ? 0.f : m[n][0]);
                const float sub1 = kWeightShift - (m[n][1] == -INFINITY ? 0.f : m[n][1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float e0 = ex2_approx(sf[u][n][0] + sub0), e1 = ex2_approx(sf[u][n][1] + sub1);
                    const float e2 = ex2_approx(sf[u][n][2] + sub0), e3 = ex2_approx(sf[u][n][3] + sub1);
                    l[n][0] = fmaf(e0 + e2, t_isv[u], l[n][0]);
                    l[n][1] = fmaf(e1 + e3, t_isv[u], l[n][1]);
                    pb[u][n][0] = transpose_b16(pack_f16x2(e0, e1));
                    pb[u][n][1] = transpose_b16(pack_f16x2(e2, e3));
                }
            }

            // ---- output += V^T weights, tile by tile ----
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t vw[4][T::VB / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = 2 * q + (k & 1) + 8 * (k >> 1);
                    const uint8_t* at = src + u * T::TILE + T::K_BYTES +
                                        (T::VB == 16 ? chunk_at<D>(row, g) : chunk_at<D>(row, g >> 1) + (g & 1) * 8);
                    if constexpr (T::VB == 16) {
                        const uint4 w = *reinterpret_cast<const uint4*>(at);
                        vw[k][0] = w.x, vw[k][1] = w.y, vw[k][2] = w.z, vw[k][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(at);
                        vw[k][0] = w.x, vw[k][1] = w.y;
                    }
                }
                auto each_pv = [&](const uint32_t (&w)[4][T::VB / 4], auto product) {  // product j, its A words
#pragma unroll
                    for (int k = 0; k < T::VB / 4; ++k) {
                        uint32_t va[4], vb[4];
                        e4m3x4_to_f16(__byte_perm(w[0][k], w[1][k], 0x5140), va[0], va[1]);
                        e4m3x4_to_f16(__byte_perm(w[2][k], w[3][k], 0x5140), va[2], va[3]);
                        product(2 * k, va);
                        e4m3x4_to_f16(__byte_perm(w[0][k], w[1][k], 0x7362), vb[0], vb[1]);
                        e4m3x4_to_f16(__byte_perm(w[2][k], w[3][k], 0x7362), vb[2], vb[3]);
                        product(2 * k + 1, vb);
                    }
                };
                bool nan_v = false;  // a NaN code that some query of the tile must not see (0 * NaN is NaN)
                if (!all_seen && s.q_len > 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < T::VB / 4; ++n) nan_v |= __vcmpeq4(vw[k][n] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
                }
                if (__any_sync(0xffffffffu, nan_v)) {
                    // query by query, with only the tokens that it sees and only its rows:
                    // rows of other queries take nothing of such a product, 0 * NaN is in it
                    const int t_lo = rt * T::ROWS / G, t_hi = min(s.q_len - 1, (rt * T::ROWS + T::ROWS - 1) / G);
#pragma unroll 1
                    for (int t = t_lo; t <= t_hi; ++t) {
                        const int ps = first_pos + t;
                        uint32_t wt[4][T::VB / 4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool vis = row_sees(ps, tok + u * kTok + 2 * q + (k & 1) + 8 * (k >> 1));
#pragma unroll
                            for (int n = 0; n < T::VB / 4; ++n) wt[k][n] = vis ? vw[k][n] : 0u;
                        }
                        each_pv(wt, [&](int j, const uint32_t (&va)[4]) {
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float t4[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(t4, va, pb[u][n][0], pb[u][n][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (pos[n][e & 1] == ps) o[n][j][e] += t4[e];
                            }
                        });
                    }
                } else {
                    each_pv(vw, [&](int j, const uint32_t (&va)[4]) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(o[n][j], va, pb[u][n][0], pb[u][n][1]);
                    });
                }
            }
        };
        int i = 0;
        for (; i < n_my; ++i) {
            if ((i & 15) == 0) next_batch();
            if (((far >> (2 * i & 31)) & 3u) != 0u) break;
            step(std::false_type{}, i);
        }
        const bool apart = i < n_my;
        if (apart) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {  // what the walk has summed so far
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], x);
                    if (g == 0)
                        stat[warp * T::ROWS + 8 * n + 2 * q + r] =
                            make_float2(l[n][r] != 0.f ? m[n][r] - kWeightShift : -INFINITY, l[n][r]);
                }
            __syncwarp();
            for (bool first = true; i < n_my; ++i, first = false) {
                if ((i & 15) == 0 && !first) next_batch();
                step(std::true_type{}, i);
            }
        }
        cp_async_wait<0>();

        // ---- join the warps ----
        __syncwarp();  // every lane is done with its ring
        float* ow = reinterpret_cast<float*>(my);
        if (apart) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 us = stat[warp * T::ROWS + 8 * n + 2 * q + r];
                    float half;
                    plain_units(m[n][r], l[n][r], us.x, us.y, half);
                    if (g != 0) l[n][r] = 0.f;  // the lanes' sums are added up
#pragma unroll
                    for (int j = 0; j < T::NJ; ++j) {
                        o[n][j][r] *= half;
                        o[n][j][r] *= half;
                        o[n][j][2 + r] *= half;
                        o[n][j][2 + r] *= half;
                    }
                }
            __syncwarp();  // stat is written again
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], x);
                const int row = 8 * n + 2 * q + r;
                if (g == 0) stat[warp * T::ROWS + row] = make_float2(m[n][r], l[n][r]);
#pragma unroll
                for (int j = 0; j < T::NJ; j += 2)
                    *reinterpret_cast<float4*>(ow + row * T::O_PITCH + g * T::VB + 2 * j) =
                        make_float4(o[n][j][r], o[n][j][2 + r], o[n][j + 1][r], o[n][j + 1][2 + r]);
            }
        __syncthreads();
        const bool finished = v0 == 0 && v1 == s.n;
        const int slot = 2 * blockIdx.x + (v0 == 0 ? 1 : 0);
        constexpr int TPR = kThreads / T::ROWS, CPT = D / TPR;  // threads a row, columns a thread
        const int r = threadIdx.x / TPR, c0 = threadIdx.x % TPR * CPT;
        const RowAt a = row_at(p, s.q_len, hk, rt, r);
        if (a.there) {
            float mm = -INFINITY, ll = 0.f, wgt[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[w * T::ROWS + r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 st = stat[w * T::ROWS + r];
                wgt[w] = st.x == -INFINITY ? 0.f : ex2_approx(st.x - mm);
                ll += st.y * wgt[w];
            }
            float acc[CPT];
#pragma unroll
            for (int e = 0; e < CPT; ++e) acc[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* from = reinterpret_cast<const float*>(smem + w * T::WARP_BYTES) + r * T::O_PITCH + c0;
#pragma unroll
                for (int e = 0; e < CPT; e += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(from + e);
                    acc[e] += wgt[w] * y.x;
                    acc[e + 1] += wgt[w] * y.y;
                    acc[e + 2] += wgt[w] * y.z;
                    acc[e + 3] += wgt[w] * y.w;
                }
            }
            if (finished) {
                const float inv = ll != 0.f ? 1.f / ll : 0.f;  // NaN stays NaN
                uint32_t pk[CPT / 2];
#pragma unroll
                for (int e = 0; e < CPT; e += 2) pk[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                uint16_t* dst = static_cast<uint16_t*>(p.o) + b * p.os.b + a.h * p.os.h + a.t * p.os.n + c0;
#pragma unroll
                for (int e = 0; e < CPT / 4; ++e) *reinterpret_cast<uint2*>(dst + 4 * e) = make_uint2(pk[2 * e], pk[2 * e + 1]);
                if (c0 == 0)
                    p.lse[(static_cast<long long>(b) * p.H + a.h) * p.T + a.t] =
                        ll != 0.f ? (mm - kWeightShift + log2f(ll)) * kLn2 : INFINITY;
            } else {
                float* dst = p.part + (static_cast<long long>(slot) * T::ROWS + r) * D + c0;
#pragma unroll
                for (int e = 0; e < CPT; e += 4)
                    *reinterpret_cast<float4*>(dst + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
                if (c0 == 0) p.stat[slot * T::ROWS + r] = make_float2(mm, ll);
            }
        }
        __syncthreads();  // shared memory is free for the next segment
        x += sh.whole > 0 ? sh.whole : v1 - v0;
    }
}

// Joins an item's unfinished segments (of either cache attention kernel), in the
// order of the keys: with M the largest of their maxima, O = sum 2^(m_i - M) O_i /
// sum 2^(m_i - M) l_i.  Blocks (c - 1, *) stand for the border before share c; the
// borders inside an item divide its rows among them.  A row is joined by one warp
// where it has few segments, else by the whole block, the segments divided among the
// warps.  Bound by latency (the border, then statistics and rows of all segments at
// once): 6 us by itself for 456 shares of 8 rows, most of it behind the kernel before it.
constexpr int kJoinWarps = 8;
constexpr int kJoinFew = 16;  // segments that one warp joins alone

// Running join of segments [i0, i1) of row r: maximum, sum and the lane's D/32 columns.
template <int D>
struct Joined {
    static constexpr int E = D / 32;
    float m = -INFINITY, l = 0.f, o[E] = {};
    __device__ void add(float sm, float sl, const float (&y)[E]) {
        if (sm == -INFINITY && sl == 0.f) return;  // a segment in which the row sees no key: no output either
        const float n = fmaxf(m, sm);
        const float a = m == -INFINITY ? 0.f : ex2_approx(m - n), w = sm == -INFINITY ? 0.f : ex2_approx(sm - n);
        m = n;
        l = l * a + sl * w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + y[e] * w;
    }
};

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_kernel(const CacheFwdParams p) {
    constexpr int E = D / 32;
    __shared__ float o_sm[kJoinWarps][D];
    __shared__ float2 stat_sm[kJoinWarps];
    const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const CacheBorder bd = p.border[c];
    if (bd.c_first < 0) return;  // the share begins with its item
    const int G = p.H / p.Hk, rts = (bd.q_len * G + p.rows - 1) / p.rows;
    const int hk = bd.item / rts, rt = bd.item - hk * rts;
    const int rows = min(p.rows, bd.q_len * G - rt * p.rows);
    const int n = bd.c_last - bd.c_first + 2;  // segments: of CTAs c_first - 1 (which starts the item) .. c_last
    auto join = [&](int r, int i0, int i1, auto at_once) {  // so many segments' loads go out together
        constexpr int U = decltype(at_once)::value;
        Joined<D> x;
        for (int i = i0; i < i1; i += U) {
            float2 st[U];
            float y[U][E];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                st[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int e = 0; e < E; ++e) y[u][e] = 0.f;
                if (i + u < i1) {
                    const long long k = 2 * (bd.c_first - 1 + i + u) + (i + u == 0 ? 1 : 0);
                    st[u] = p.stat[k * p.rows + r];
                    const float* src = p.part + (k * p.rows + r) * D + lane * E;
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 v = *reinterpret_cast<const float2*>(src + e);
                        y[u][e] = v.x;
                        y[u][e + 1] = v.y;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) x.add(st[u].x, st[u].y, y[u]);
        }
        return x;
    };
    auto write = [&](int r, const Joined<D>& x) {
        const RowAt a = row_at(p, bd.q_len, hk, rt, r);
        const float inv = x.l != 0.f ? 1.f / x.l : 0.f;
        uint16_t* dst = static_cast<uint16_t*>(p.o) + bd.b * p.os.b + a.h * p.os.h + a.t * p.os.n + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(x.o[e] * inv, x.o[e + 1] * inv);
        if (lane == 0)
            p.lse[(static_cast<long long>(bd.b) * p.H + a.h) * p.T + a.t] =
                x.l != 0.f ? (x.m - kWeightShift + log2f(x.l)) * kLn2 : INFINITY;
    };
    const int mine = (c - bd.c_first) * static_cast<int>(gridDim.y) + blockIdx.y, borders = (n - 1) * static_cast<int>(gridDim.y);
    if (n <= kJoinFew) {
        for (int r = mine + borders * warp; r < rows; r += borders * kJoinWarps)
            write(r, join(r, 0, n, std::integral_constant<int, 4>{}));
        return;
    }
    const int per = (n + kJoinWarps - 1) / kJoinWarps;
    for (int r = mine; r < rows; r += borders) {
        const Joined<D> x = join(r, min(n, warp * per), min(n, warp * per + per), std::integral_constant<int, 8>{});
#pragma unroll
        for (int e = 0; e < E; ++e) o_sm[warp][lane * E + e] = x.o[e];
        if (lane == 0) stat_sm[warp] = make_float2(x.m, x.l);
        __syncthreads();
        if (warp == 0) {
            Joined<D> z;
            for (int w = 0; w < kJoinWarps; ++w) {
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = o_sm[w][lane * E + e];
                z.add(stat_sm[w].x, stat_sm[w].y, y);
            }
            write(r, z);
        }
        __syncthreads();
    }
}

template <int D, int NT>
cudaError_t launch_decode_impl(CacheFwdParams p, int sms, cudaStream_t stream) {
    using T = DecodeTraits<D, NT>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t attr = once_per_device(ready, [] {
        return cudaFuncSetAttribute(cache_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    });
    if (attr != cudaSuccess) return attr;
    p.rows = T::ROWS;
    p.grid = sms * T::CTAS_PER_SM < kCacheGridMax ? sms * T::CTAS_PER_SM : kCacheGridMax;
    const cudaError_t e = launch_dependent(cache_decode_kernel<D, NT>, dim3(static_cast<unsigned>(p.grid)), kThreads,
                                           T::SMEM, stream, p);
    return e != cudaSuccess ? e : launch_cache_join(p, 1, stream);
}

template <int D>
cudaError_t launch_decode_d(const CacheFwdParams& p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(p.T) * (p.H / p.Hk);
    if (rows <= 8) return launch_decode_impl<D, 1>(p, sms, stream);
    return launch_decode_impl<D, 2>(p, sms, stream);
}

}  // namespace

cudaError_t launch_cache_join(const CacheFwdParams& p, int blocks, cudaStream_t stream) {
    if (p.grid == 1) return cudaSuccess;  // no border
    const dim3 grid(static_cast<unsigned>(p.grid - 1), static_cast<unsigned>(blocks));
    if (p.D == 64) return launch_dependent(cache_join_kernel<64>, grid, 32 * kJoinWarps, 0, stream, p);
    if (p.D == 128) return launch_dependent(cache_join_kernel<128>, grid, 32 * kJoinWarps, 0, stream, p);
    return cudaErrorInvalidValue;
}

cudaError_t launch_cache_decode(const CacheFwdParams& p, cudaStream_t stream) {
    if (p.D == 64) return launch_decode_d<64>(p, stream);
    if (p.D == 128) return launch_decode_d<128>(p, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream) {
    const int pages = (p.T + p.c.page_size - 2) / p.c.page_size + 1;  // pages that T tokens can touch
    const dim3 grid(static_cast<unsigned>(pages), static_cast<unsigned>(p.Hk), static_cast<unsigned>(2 * p.B));
    if (p.D == 64) return launch_dependent(cache_append_kernel<64>, grid, kAppendThreads, 0, stream, p);
    if (p.D == 128) return launch_dependent(cache_append_kernel<128>, grid, kAppendThreads, 0, stream, p);
    return cudaErrorInvalidValue;
}

}  // namespace attn
