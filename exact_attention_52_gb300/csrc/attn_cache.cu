// Paged 8-bit key/value cache: writing new tokens, and attention of a few new
// queries per sequence over it.
//
// A page holds page_size tokens of every key/value head as OCP E4M3 codes, with
// one fp32 scale per page, head and tensor: the value is scale * code.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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
constexpr int kAppendThreads = 128;
constexpr int kMinScaleExp = -100;

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;  // NaN compares false
}

// Smallest power of two s >= 2^kMinScaleExp with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float append_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>(max(e, kMinScaleExp) + 127) << 23);
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheAppendParams p) {
    constexpr int TPR = D / 8;  // threads per token: 8 elements each
    constexpr int RPP = kAppendThreads / TPR;
    const int hk = blockIdx.y, b = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int page = p.c.page_size, cap = p.c.max_pages * page;
    const int len = p.c.seq_lens[b];
    const int m = p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
    if (m == 0 || len <= 0) return;
    const int first = len - m;  // position of new token 0 (negative: it is not written)
    const int pg = max(first, 0) / page + static_cast<int>(blockIdx.x);
    const int lo = max(first, pg * page), hi = min(len, pg * page + page);  // new positions in this page
    if (lo >= hi) return;
    if (lo >= cap) {
        if (threadIdx.x == 0) record_device_error(p.st, ATTN_DEVERR_PAGE, 0x302);
        return;
    }
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

    float amax = 0.f;
    for (int pos = lo + rr; pos < hi; pos += RPP) {
        const uint4 w = *reinterpret_cast<const uint4*>(x + (pos - first) * xs.n);
        for (uint32_t u : {w.x, w.y, w.z, w.w}) amax = fmaxf(amax, fmaxf(finite_abs(bf16lo(u)), finite_abs(bf16hi(u))));
    }
    // Magnitudes order as their bit patterns: one integer maximum per warp.
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = wm;
    __syncthreads();  // and every thread has read the old scale
    amax = __uint_as_float(max(max(warp_max[0], warp_max[1]), max(warp_max[2], warp_max[3])));
    const int old = lo - pg * page;  // tokens that the page holds already
    const bool keep = old > 0 && amax <= 448.f * was;
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
    for (int pos = lo + rr; pos < hi; pos += RPP) {
        const uint4 w = *reinterpret_cast<const uint4*>(x + (pos - first) * xs.n);
        const uint32_t a = pack_e4m3x4(bf16lo(w.x) / s, bf16hi(w.x) / s, bf16lo(w.y) / s, bf16hi(w.y) / s);
        const uint32_t c = pack_e4m3x4(bf16lo(w.z) / s, bf16hi(w.z) / s, bf16lo(w.w) / s, bf16hi(w.w) / s);
        *reinterpret_cast<uint2*>(codes + (pos - pg * page) * cs.n) = make_uint2(a, c);
    }
    if (threadIdx.x == 0 && !keep) *scale = s;
}

// ---------------------------------------------------------------------------
// Attention of a few queries: work shared out evenly
// ---------------------------------------------------------------------------
// An item is (sequence, key/value head, tile of kRows query rows); the rows of a
// key/value head are its H/Hk query heads of every new query, row = t * H/Hk + g.
// An item's blocks of kBlock tokens are laid end to end over all items, and CTA c
// of G takes the c-th of G equal shares of that line, whatever the lengths of the
// sequences are: lengths stay on the device.  A share can begin and end inside
// an item; such unfinished segments go to the workspace and a second kernel joins
// them.  At most two per CTA: slot 2c for a segment that does not start its item,
// or starts it and does not reach its end in slot 2c + 1.
constexpr int kRows = 16;   // query rows of a tile: M of one mma
constexpr int kBlock = 16;  // tokens of a block: K of one mma
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;  // blocks in flight per warp
constexpr int kCtasPerSm = 3;
// A share has at least this many blocks: with fewer, joining costs more than the
// shorter walk gives.
constexpr int kMinShare = 16;

struct Share {
    long long total, share;
    int b;              // sequence that holds the start of the share
    long long b_first;  // blocks before that sequence
};

struct ShareSmem {
    long long warp_sum[kWarps], b_first;
    int b;
};

__device__ __forceinline__ long long seq_work(const CacheFwdParams& p, const CacheSeq& s) {
    const int rt = (s.q_len * (p.H / p.Hk) + kRows - 1) / kRows;
    return static_cast<long long>(s.n) * rt * p.Hk;
}

// Lays the items of all sequences end to end and finds the sequence at the start
// of share c (B sequences, a slice of them per thread).
__device__ Share find_share(const CacheFwdParams& p, int c, ShareSmem* sm) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += seq_work(p, cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sm->warp_sum[warp] = incl;
    if (threadIdx.x == 0) sm->b = -1;
    __syncthreads();
    Share s;
    s.total = 0;
    long long before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm->warp_sum[w];
        s.total += sm->warp_sum[w];
    }
    s.share = max((s.total + p.grid - 1) / p.grid, static_cast<long long>(kMinShare));
    const long long x = c * s.share;
    if (x < s.total && before <= x && x < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const long long w = seq_work(p, cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b));
            if (x < before + w) {
                sm->b = b;
                sm->b_first = before;
                break;
            }
            before += w;
        }
    }
    __syncthreads();
    s.b = sm->b;
    s.b_first = sm->b_first;
    return s;
}

// Row r (0 .. kRows - 1) of row tile rt of a sequence: query and head of the group.
struct RowAt {
    int t, h;
    bool there;
};
__device__ __forceinline__ RowAt row_at(const CacheFwdParams& p, int q_len, int hk, int rt, int r) {
    const int G = p.H / p.Hk, row = rt * kRows + r;
    RowAt a;
    a.t = row / G;
    a.h = hk * G + row % G;
    a.there = a.t < q_len;
    return a;
}

// ---------------------------------------------------------------------------
// Attention of a few queries: the kernel
// ---------------------------------------------------------------------------
// Bound by reading the codes once.  Each warp walks every kWarps-th block of a
// segment on its own, with its own running maximum, sums and output: a lane
// copies exactly the bytes that it will turn into its fragments (asynchronous
// copies into a ring of its own, kStages - 1 blocks ahead), so no barrier stands
// in the loop.  Codes become f16 exactly and go to f16 matrix products with fp32
// sums; Q rows are brought to f16 by a power of two each.  A page's scales enter
// in fp32: the key scale multiplies the scores, the value scale is added, as its
// log2, to the exponent, so that the weights given to the products are
// 2^(score + log2 sv - m) with the running maximum m taken over score + log2 sv,
// and the sum of the probabilities takes them back by 1 / sv.  The weights are
// scaled by 2^kShift, f16's room above 1, so that one is lost to underflow only
// below 2^-40 of the largest.
//
// Fragment layouts (g = lane / 4, q = lane % 4).  Contraction indices may be
// permuted if both operands are: in K, lane (g, q) holds token g and the 16
// consecutive d from 64 c + 16 q, of which word s gives the k-pairs (2q, 2q + 1)
// and (2q + 8, 2q + 9) of product (c, s).  In V, lane (g, q) holds tokens 2q,
// 2q + 1, 2q + 8, 2q + 9 and the D/8 consecutive d from g D/8, the j-th of which
// is column g of n-tile j: column n of n-tile j is d = n D/8 + j.
constexpr int kShift = 15;

template <int D>
struct DecodeTraits {
    static constexpr int KC = D / 64;  // 16-byte pieces of a token's K row per lane
    static constexpr int VB = D / 8;   // bytes of a token's V row per lane
    static constexpr int NJ = D / 8;   // n-tiles of the output
    static constexpr int K_BYTES = 2 * KC * 512, V_BYTES = 4 * 32 * VB;
    static constexpr int STAGE = K_BYTES + V_BYTES + 16;  // + the page's two scales
    static constexpr int RING = kStages * STAGE;
    static constexpr int O_PITCH = D + 4;  // floats between rows of a warp's output in shared memory
    static constexpr int WARP_BYTES = RING > kRows * O_PITCH * 4 ? RING : kRows * O_PITCH * 4;
    static constexpr int SMEM = kWarps * WARP_BYTES + kWarps * kRows * 8 + static_cast<int>(sizeof(ShareSmem));
};

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) cache_decode_kernel(const CacheFwdParams p) {
    using T = DecodeTraits<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    uint8_t* my = smem + warp * T::WARP_BYTES;
    const uint32_t my_u = smem_u32(my);
    float2* stat = reinterpret_cast<float2*>(smem + kWarps * T::WARP_BYTES);  // [kWarps][kRows]
    ShareSmem* ssm = reinterpret_cast<ShareSmem*>(stat + kWarps * kRows);

    const Share sh = find_share(p, blockIdx.x, ssm);
    pdl_launch_dependents();
    if (sh.b < 0) return;  // more CTAs than shares
    long long x = blockIdx.x * sh.share;
    const long long x_end = min(x + sh.share, sh.total);
    int b = sh.b;
    long long b_first = sh.b_first;
    const int G = p.H / p.Hk;

    while (x < x_end) {
        CacheSeq s = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, b);
        for (long long w; x >= b_first + (w = seq_work(p, s));) {  // next sequence with work
            b_first += w;
            s = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, ++b);
        }
        // segment [v0, v1) of the item's n blocks
        const int rts = (s.q_len * G + kRows - 1) / kRows;
        const int item = static_cast<int>((x - b_first) / s.n);
        const int v0 = static_cast<int>((x - b_first) - static_cast<long long>(item) * s.n);
        const int v1 = static_cast<int>(min(static_cast<long long>(s.n), v0 + (x_end - x)));
        const int hk = item / rts, rt = item % rts;
        const int first_pos = s.len - s.q_len;  // may be negative: rows before the first token see nothing

        // ---- Q rows g and g + 8 as f16, each times a power of two ----
        uint32_t qa[T::KC * 4][4];
        float rq[2];
        int pos[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const RowAt a = row_at(p, s.q_len, hk, rt, g + 8 * i);
            pos[i] = first_pos + a.t;
            uint4 w[T::KC][2];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < T::KC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[c][e] = make_uint4(0u, 0u, 0u, 0u);
                    if (a.there)
                        w[c][e] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + b * p.qs.b +
                                                                  a.h * p.qs.h + a.t * p.qs.n + c * 64 + q * 16 + e * 8);
                    for (uint32_t u : {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w})
                        amax = fmaxf(amax, fmaxf(fabsf(bf16lo(u)), fabsf(bf16hi(u))));
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float f = f16_row_scale(amax);
            rq[i] = p.cs * __uint_as_float((254u << 23) - __float_as_uint(f));
#pragma unroll
            for (int c = 0; c < T::KC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t u[4] = {w[c][e].x, w[c][e].y, w[c][e].z, w[c][e].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // elements 8e + 2k, 8e + 2k + 1 of the lane's 16: product 2e + k/2
                        qa[c * 4 + 2 * e + (k >> 1)][i + 2 * (k & 1)] = pack_f16x2(bf16lo(u[k]) * f, bf16hi(u[k]) * f);
                }
        }

        float o[T::NJ][4];
#pragma unroll
        for (int j = 0; j < T::NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        const uint8_t* kbase = p.c.k_pages + hk * p.c.ks.h + g * p.c.ks.n + q * 16;
        const uint8_t* vbase = p.c.v_pages + hk * p.c.vs.h + 2 * q * p.c.vs.n + g * T::VB;
        const int slot_mask = p.c.page_size - 1;
        // token of the sequence seen by some query
        auto seen = [&](int j) { return j < s.len && (j >= s.key_lo || j < p.sinks); };
        auto issue = [&](int v, int stage) {
            if (v < v1) {
                const int tok = cache_block(s, v) * kBlock;
                const int pid = tok < s.len ? cache_page(p.c, p.st, b, tok) : 0;
                const uint32_t dst = my_u + stage * T::STAGE;
                const uint8_t* kp = kbase + pid * p.c.ks.b + (tok & slot_mask) * p.c.ks.n;
                const uint8_t* vp = vbase + pid * p.c.vs.b + (tok & slot_mask) * p.c.vs.n;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bool there = seen(tok + 8 * u + g);
#pragma unroll
                    for (int c = 0; c < T::KC; ++c)
                        cp_async16(dst + (u * T::KC + c) * 512 + lane * 16, kp + 8 * u * p.c.ks.n + c * 64, there);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = (k & 1) + 8 * (k >> 1);
                    const bool there = seen(tok + 2 * q + t);
                    const uint32_t to = dst + T::K_BYTES + (k * 32 + lane) * T::VB;
                    if constexpr (T::VB == 16) cp_async16(to, vp + t * p.c.vs.n, there);
                    else cp_async8(to, vp + t * p.c.vs.n, there);
                }
                if (lane < 2)
                    cp_async4(dst + T::K_BYTES + T::V_BYTES + 4 * lane,
                              (lane ? p.c.v_scale : p.c.k_scale) + static_cast<long long>(pid) * p.Hk + hk, true);
            }
            cp_async_commit();
        };

#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(v0 + warp + kWarps * i, i);
        int stage = 0;
        for (int v = v0 + warp; v < v1; v += kWarps) {
            issue(v + kWarps * (kStages - 1), stage == 0 ? kStages - 1 : stage - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();  // the scales were copied by lanes 0 and 1
            const uint8_t* src = my + stage * T::STAGE;
            const float2 sc = *reinterpret_cast<const float2*>(src + T::K_BYTES + T::V_BYTES);

            // ---- scores of 16 rows and 16 tokens ----
            float sf[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sf[u][e] = 0.f;
#pragma unroll
                for (int c = 0; c < T::KC; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(src + (u * T::KC + c) * 512 + lane * 16);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(ww[k], b0, b1);
                        mma_f16(sf[u], qa[c * 4 + k], b0, b1);
                    }
                }
            }
            const int tok = cache_block(s, v) * kBlock;
            const float lsv = lg2_approx(sc.y);
            const float f[2] = {rq[0] * sc.x, rq[1] * sc.x};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) sf[u][e] = fmaf(sf[u][e], f[e >> 1], lsv);
            // every query sees all 16 tokens, or each score is checked
            const bool whole = tok + kBlock - 1 <= first_pos &&
                               (p.left < 0 || tok >= s.len - 1 - p.left || tok + kBlock <= p.sinks);
            auto row_sees = [&](int ps, int j) { return j <= ps && (p.left < 0 || j >= ps - p.left || j < p.sinks); };
            if (!whole) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!row_sees(pos[e >> 1], tok + 8 * u + 2 * q + (e & 1))) sf[u][e] = -INFINITY;
            }
            // ---- running maximum: raised (and the output rescaled) only when a score passes it ----
            float mx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mx[i] = fmaxf(fmaxf(sf[0][2 * i], sf[0][2 * i + 1]), fmaxf(sf[1][2 * i], sf[1][2 * i + 1]));
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float n = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                    n = fmaxf(m[i], fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2)));
                    const float alpha = n == m[i] ? 1.f : ex2_approx(m[i] - n);  // 0 while m is -inf
                    m[i] = n;
                    l[i] *= alpha;
#pragma unroll
                    for (int j = 0; j < T::NJ; ++j) {
                        o[j][2 * i] *= alpha;
                        o[j][2 * i + 1] *= alpha;
                    }
                }
            }
            const float inv_sv = 1.f / sc.y;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float sub = (m[i] == -INFINITY ? 0.f : m[i]) - kShift;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sf[u][2 * i + e] = ex2_approx(sf[u][2 * i + e] - sub);
                        sum += sf[u][2 * i + e];
                    }
                l[i] = fmaf(sum, inv_sv, l[i]);
            }
            // weights rounded to f16 (2^-12 relative): finer than the bf16 output
            const uint32_t pa[4] = {pack_f16x2(sf[0][0], sf[0][1]), pack_f16x2(sf[0][2], sf[0][3]),
                                    pack_f16x2(sf[1][0], sf[1][1]), pack_f16x2(sf[1][2], sf[1][3])};

            // ---- output += weights V ----
            uint32_t vw[4][T::VB / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint8_t* at = src + T::K_BYTES + (k * 32 + lane) * T::VB;
                if constexpr (T::VB == 16) {
                    const uint4 w = *reinterpret_cast<const uint4*>(at);
                    vw[k][0] = w.x, vw[k][1] = w.y, vw[k][2] = w.z, vw[k][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(at);
                    vw[k][0] = w.x, vw[k][1] = w.y;
                }
            }
            auto add_pv = [&](const uint32_t (&a)[4], const uint32_t (&w)[4][T::VB / 4]) {
#pragma unroll
                for (int i = 0; i < T::VB / 4; ++i) {
                    const uint32_t x01 = __byte_perm(w[0][i], w[1][i], 0x5140), x23 = __byte_perm(w[0][i], w[1][i], 0x7362);
                    const uint32_t y01 = __byte_perm(w[2][i], w[3][i], 0x5140), y23 = __byte_perm(w[2][i], w[3][i], 0x7362);
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    e4m3x4_to_f16(x01, a0, a1);
                    e4m3x4_to_f16(x23, a2, a3);
                    e4m3x4_to_f16(y01, b0, b1);
                    e4m3x4_to_f16(y23, b2, b3);
                    mma_f16(o[4 * i], a, a0, b0);
                    mma_f16(o[4 * i + 1], a, a1, b1);
                    mma_f16(o[4 * i + 2], a, a2, b2);
                    mma_f16(o[4 * i + 3], a, a3, b3);
                }
            };
            bool nan_v = false;  // a NaN code that some query of the tile must not see (0 * NaN is NaN)
            if (!whole && s.q_len > 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < T::VB / 4; ++i) nan_v |= __vcmpeq4(vw[k][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
            }
            if (__any_sync(0xffffffffu, nan_v)) {
                // query by query, with only the rows and the tokens that belong to it
                const int t_lo = rt * kRows / G, t_hi = min(s.q_len - 1, (rt * kRows + kRows - 1) / G);
                for (int t = t_lo; t <= t_hi; ++t) {
                    const int ps = first_pos + t;
                    uint32_t wt[4][T::VB / 4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool vis = row_sees(ps, tok + 2 * q + (k & 1) + 8 * (k >> 1));
#pragma unroll
                        for (int i = 0; i < T::VB / 4; ++i) wt[k][i] = vis ? vw[k][i] : 0u;
                    }
                    // a row of another query gets zero weights; 0 * NaN of this query's
                    // values would reach it, so its output is kept
                    const uint32_t at[4] = {pos[0] == ps ? pa[0] : 0u, pos[1] == ps ? pa[1] : 0u,
                                            pos[0] == ps ? pa[2] : 0u, pos[1] == ps ? pa[3] : 0u};
                    float kept[T::NJ][4];
#pragma unroll
                    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) kept[j][e] = o[j][e];
                    add_pv(at, wt);
#pragma unroll
                    for (int j = 0; j < T::NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (pos[e >> 1] != ps) o[j][e] = kept[j][e];
                }
            } else {
                add_pv(pa, vw);
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();

        // ---- join the warps ----
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        __syncwarp();  // every lane is done with its ring
        float* ow = reinterpret_cast<float*>(my);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (q == 0) stat[warp * kRows + g + 8 * i] = make_float2(m[i], l[i]);
#pragma unroll
            for (int n = 0; n < 2; ++n)  // columns 2q and 2q + 1: D/8 consecutive d each
#pragma unroll
                for (int j = 0; j < T::NJ; j += 4)
                    *reinterpret_cast<float4*>(ow + (g + 8 * i) * T::O_PITCH + (2 * q + n) * T::VB + j) =
                        make_float4(o[j][2 * i + n], o[j + 1][2 * i + n], o[j + 2][2 * i + n], o[j + 3][2 * i + n]);
        }
        __syncthreads();
        const bool finished = v0 == 0 && v1 == s.n;
        const int slot = 2 * blockIdx.x + (v0 == 0 ? 1 : 0);
        constexpr int CPT = D / 8;  // columns per thread: 8 threads a row
        const int r = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * CPT;
        const RowAt a = row_at(p, s.q_len, hk, rt, r);
        if (a.there) {
            float mm = -INFINITY, ll = 0.f, wgt[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[w * kRows + r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 st = stat[w * kRows + r];
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
                for (int e = 0; e < CPT / 8; ++e)
                    st_global_v4(dst + 8 * e, pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                if (c0 == 0)
                    p.lse[(static_cast<long long>(b) * p.H + a.h) * p.T + a.t] =
                        ll != 0.f ? (mm - kShift + log2f(ll)) * kLn2 : INFINITY;
            } else {
                float* dst = p.part + (static_cast<long long>(slot) * kRows + r) * D + c0;
#pragma unroll
                for (int e = 0; e < CPT; e += 4)
                    *reinterpret_cast<float4*>(dst + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
                if (c0 == 0) p.stat[slot * kRows + r] = make_float2(mm, ll);
            }
        }
        __syncthreads();  // shared memory is free for the next segment
        x += v1 - v0;
    }
}

// Joins an item's unfinished segments, in the order of the keys: with M the
// largest of their maxima, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  Block
// (c, r) looks at the border between shares c and c + 1; the first border inside
// an item joins row r of the whole item.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_join_kernel(const CacheFwdParams p) {
    __shared__ ShareSmem ssm;
    __shared__ float acc_sm[kWarps][D];
    __shared__ float2 stat_sm[kWarps];
    const int c = blockIdx.x + 1, r = blockIdx.y;
    const Share sh = find_share(p, c, &ssm);
    pdl_wait();
    if (sh.b < 0) return;
    const CacheSeq s = cache_seq<kBlock>(p.c, p.q_lens, p.T, p.left, p.sinks, sh.b);
    const long long x = c * sh.share;
    const int G = p.H / p.Hk, rts = (s.q_len * G + kRows - 1) / kRows;
    const int item = static_cast<int>((x - sh.b_first) / s.n);
    const long long i0 = sh.b_first + static_cast<long long>(item) * s.n, i1 = i0 + s.n;
    if (x == i0 || x - sh.share > i0) return;  // no border here, or not the item's first
    const RowAt a = row_at(p, s.q_len, item / rts, item % rts, r);
    if (!a.there) return;
    // segments: share c - 1 (it starts the item), c, c + 1, ... up to the one with block i1 - 1
    const int c_last = static_cast<int>((i1 - 1) / sh.share);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto slot = [&](int k) { return 2 * k + (k == c - 1 ? 1 : 0); };
    constexpr int E = D / 32;
    float M = -INFINITY;
    for (int k = c - 1 + static_cast<int>(threadIdx.x); k <= c_last; k += kThreads)
        M = fmaxf(M, p.stat[slot(k) * kRows + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) stat_sm[warp].x = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stat_sm[w].x);
    __syncthreads();
    float acc[E], l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int n = c_last - (c - 1) + 1, per = (n + kWarps - 1) / kWarps;
#pragma unroll 4
    for (int i = warp * per; i < min(n, warp * per + per); ++i) {
        const int k = slot(c - 1 + i);
        const float2 st = p.stat[k * kRows + r];
        const float w = st.x == -INFINITY ? 0.f : ex2_approx(st.x - M);
        const float* src = p.part + (static_cast<long long>(k) * kRows + r) * D + lane * E;
        l += w * st.y;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 y = *reinterpret_cast<const float2*>(src + e);
            acc[e] += w * y.x;
            acc[e + 1] += w * y.y;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc_sm[warp][lane * E + e] = acc[e];
    if (lane == 0) stat_sm[warp].y = l;
    __syncthreads();
    if (warp != 0) return;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        l += stat_sm[w].y;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += acc_sm[w][lane * E + e];
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint16_t* dst = static_cast<uint16_t*>(p.o) + sh.b * p.os.b + a.h * p.os.h + a.t * p.os.n + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
        p.lse[(static_cast<long long>(sh.b) * p.H + a.h) * p.T + a.t] =
            l != 0.f ? (M - kShift + log2f(l)) * kLn2 : INFINITY;
}

template <int D>
cudaError_t launch_decode_impl(const CacheFwdParams& p, cudaStream_t stream) {
    static const cudaError_t attr = cudaFuncSetAttribute(
        cache_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecodeTraits<D>::SMEM);
    if (attr != cudaSuccess) return attr;
    cache_decode_kernel<D><<<p.grid, kThreads, DecodeTraits<D>::SMEM, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.grid == 1) return e;
    const int rows = p.T * (p.H / p.Hk);  // rows of a tile that exist
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid - 1), static_cast<unsigned>(rows < kRows ? rows : kRows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<D>, p);
}

}  // namespace

int cache_decode_ctas_per_sm() { return kCtasPerSm; }

cudaError_t launch_cache_decode(const CacheFwdParams& p, cudaStream_t stream) {
    if (p.D == 64) return launch_decode_impl<64>(p, stream);
    if (p.D == 128) return launch_decode_impl<128>(p, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream) {
    const int pages = (p.T + p.c.page_size - 2) / p.c.page_size + 1;  // pages that T tokens can touch
    const dim3 grid(static_cast<unsigned>(pages), static_cast<unsigned>(p.Hk), static_cast<unsigned>(2 * p.B));
    if (p.D == 64) cache_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(p);
    else if (p.D == 128) cache_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(p);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace attn
