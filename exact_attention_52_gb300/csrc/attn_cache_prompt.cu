// Attention of many new queries per sequence (chunks of a prompt) over the paged
// 8-bit cache, on the fifth-generation tensor cores.
//
// An item is (sequence, two adjacent 128-row query tiles, key/value head); the rows
// of a key/value head are its H/Hk query heads of every new query, row = t * H/Hk +
// g, so that grouped heads fill the tiles and share the keys.  The item's key tiles
// of 128 tokens stream through a shared-memory ring:
//
//   warps 9-11  converters: read the codes of a key or value tile page by page,
//               turn them into f16 (exact) and write them where the tensor core
//               expects them (128-byte swizzle)
//   warp 8      MMA issuer: S_g = Q_g K_j^T and O_g += P_g V_j, accumulators in
//               tensor memory, order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
//   warps 0-3   softmax of query tile 0 (one thread per row), which also bring the
//   warps 4-7   tile's Q rows to f16; the same for query tile 1
//
// Bound by the tensor cores: 2048 cycles of products a key tile and item, in which
// the converters' 64 KB of f16 take about 430 issue slots each.  Codes are turned
// into f16 and not used as E4M3 operands, because then Q and the weights would have
// to be E4M3 too (2^-4 relative).  A page's scales enter in fp32 as in the kernel
// for few queries: score * key scale, + log2 of the value scale in the exponent, and
// 1 / value scale in the sum.
//
// The work is shared out as there: items laid end to end by their key tiles, an
// equal share for each CTA, unfinished segments joined by a second kernel.  Whole
// items would leave SMs idle in the last of few rounds (512 equal items on 152 SMs:
// 16 %).
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kPairRows = 2 * kTile;
constexpr int kPromptThreads = 384;
constexpr int kConvWarps = 3;
constexpr int kScaleRing = 8;
constexpr float kShift = 4.f;           // weights are 2^(score - m + kShift), f16
constexpr float kRedoBound = 32768.f;   // a row's tile sum that makes it take its own maximum

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }
__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

enum : uint32_t {
    SITE_Q = 0x401, SITE_KV_EMPTY = 0x402, SITE_KV_FULL = 0x403, SITE_P_FULL = 0x404, SITE_S_FULL = 0x405,
    SITE_O_FULL = 0x406, SITE_DRAIN = 0x407, SITE_SCALE = 0x408,
};

constexpr uint32_t kFmtF16 = 0;

template <int D>
struct PromptTraits {
    static constexpr int NBLK = D / 64;             // 128-byte column blocks of an f16 row
    static constexpr int BLK_BYTES = kTile * 128;
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int KV_SLOTS = D == 128 ? 5 : 8;
    static constexpr int SMEM_Q = 2 * TILE_BYTES;
    static constexpr int OFF_KV = SMEM_Q;
    static constexpr int OFF_SCALE = OFF_KV + KV_SLOTS * TILE_BYTES;  // float4 [kScaleRing][8]
    static constexpr int OFF_BAR = OFF_SCALE + kScaleRing * 8 * 16;
    // q_full[2], kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], scale_full[8], done
    static constexpr int NBARS = 2 + 2 * KV_SLOTS + 6 + kScaleRing + 1;
    static constexpr int OFF_SHARE = OFF_BAR + NBARS * 8 + 16;
    static constexpr int SMEM_BYTES = OFF_SHARE + 256;
    static constexpr uint32_t COL_S0 = 0, COL_S1 = 128, COL_O0 = 256, COL_O1 = 256 + D;
    static constexpr uint32_t IDESC_S = make_idesc(kFmtF16, kTile, kTile, false, false);
    static constexpr uint32_t IDESC_PV = make_idesc(kFmtF16, kTile, D, false, true);
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// A pair of query tiles of a sequence and the key tiles it walks: the n_sink first
// ones of the sequence, then those from lo on; query tile g uses the first n_g of n.
struct PromptUnit {
    int len, q_len, rows;
    int first_pos;  // position of query 0 (negative: rows before the first token see nothing)
    int key_lo;     // first key of the window of the pair's first query
    int n_sink, lo, n, n0, n1;
    __device__ int tile(int v) const { return v < n_sink ? v : lo + v - n_sink; }
};

__device__ PromptUnit prompt_unit(const CacheFwdParams& p, int b, int pair) {
    PromptUnit u;
    const int G = p.H / p.Hk, cap = p.c.max_pages * p.c.page_size;
    u.len = min(max(p.c.seq_lens[b], 0), cap);
    u.q_len = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
    u.rows = u.q_len * G;
    u.first_pos = u.len - u.q_len;
    u.n = u.n0 = u.n1 = u.n_sink = u.lo = u.key_lo = 0;
    const int r0 = pair * kPairRows;
    if (r0 >= u.rows) return u;  // no such pair: no work
    const int pos_lo = max(0, u.first_pos + r0 / G);
    u.key_lo = p.left < 0 ? 0 : max(0, pos_lo - p.left);
    u.lo = u.key_lo / kTile;
    u.n_sink = min((min(p.sinks, u.key_lo) + kTile - 1) / kTile, u.lo);
    auto tiles = [&](int row_hi) {  // up to the key tile of the last position of rows .. row_hi
        const int pos = u.first_pos + min(u.rows - 1, row_hi) / G;
        return pos < 0 ? 0 : u.n_sink + pos / kTile - u.lo + 1;
    };
    u.n0 = tiles(r0 + kTile - 1);
    u.n1 = r0 + kTile < u.rows ? tiles(r0 + kPairRows - 1) : 0;
    u.n = max(1, max(u.n0, u.n1));
    return u;
}

// A CTA's share: blocks [x, x_end) of the line on which the units' items lie end to
// end (each unit once per key/value head), starting in unit `unit`, before which lie
// unit_first blocks.  unit < 0: nothing.
struct PromptShare {
    long long share, x, x_end, unit_first;
    int unit;
};

struct PromptShareSmem {
    long long warp_sum[kPromptThreads / 32], unit_first;
    int unit;
};

__device__ __forceinline__ long long div_mostly32(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

__device__ PromptShare prompt_share(const CacheFwdParams& p, int pairs, PromptShareSmem* sm) {
    constexpr int W = kPromptThreads / 32;
    const int units = p.B * pairs, per = (units + kPromptThreads - 1) / kPromptThreads;
    const int u0 = min(units, static_cast<int>(threadIdx.x) * per), u1 = min(units, u0 + per);
    auto work = [&](int u) { return static_cast<long long>(prompt_unit(p, u / pairs, u % pairs).n) * p.Hk; };
    long long mine = 0;
    for (int u = u0; u < u1; ++u) mine += work(u);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sm->warp_sum[warp] = incl;
    if (threadIdx.x == 0) sm->unit = -1;
    __syncthreads();
    long long total = 0, before = incl - mine;
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sm->warp_sum[w];
        total += sm->warp_sum[w];
    }
    PromptShare s;
    s.share = max(div_mostly32(total + p.grid - 1, p.grid), 1ll);
    s.x = blockIdx.x * s.share;
    s.x_end = min(s.x + s.share, total);
    if (s.x < total && before <= s.x && s.x < before + mine) {
        for (int u = u0; u < u1; ++u) {
            const long long w = work(u);
            if (s.x < before + w) {
                sm->unit = u;
                sm->unit_first = before;
                break;
            }
            before += w;
        }
    }
    __syncthreads();
    s.unit = sm->unit;
    s.unit_first = sm->unit_first;
    return s;
}

// Walks the segments of a share, for every role alike.
struct PromptWalk {
    PromptShare s;
    int pairs;
    PromptUnit u;
    int b, pair, hk, v0, v1, a0, a1;  // segment [v0, v1); query tile g is live in its first a_g tiles
    __device__ PromptWalk(const PromptShare& share, int pairs_) : s(share), pairs(pairs_) {}
    __device__ bool next(const CacheFwdParams& p) {
        if (s.unit < 0 || s.x >= s.x_end) return false;
        u = prompt_unit(p, s.unit / pairs, s.unit % pairs);
        for (long long w; s.x >= s.unit_first + (w = static_cast<long long>(u.n) * p.Hk);) {
            s.unit_first += w;
            ++s.unit;
            u = prompt_unit(p, s.unit / pairs, s.unit % pairs);
        }
        b = s.unit / pairs;
        pair = s.unit - b * pairs;
        hk = static_cast<int>(div_mostly32(s.x - s.unit_first, u.n));
        v0 = static_cast<int>((s.x - s.unit_first) - static_cast<long long>(hk) * u.n);
        v1 = static_cast<int>(min(static_cast<long long>(u.n), v0 + (s.x_end - s.x)));
        a0 = max(0, min(v1, u.n0) - v0);
        a1 = max(0, min(v1, u.n1) - v0);
        s.x += v1 - v0;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1) cache_prompt_kernel(const CacheFwdParams p, const int pairs) {
    using T = PromptTraits<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* sKV = smem + T::OFF_KV;
    float4* scales = reinterpret_cast<float4*>(smem + T::OFF_SCALE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + T::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t b_q = bar0;  // + 8 g
    auto b_kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto b_kv_empty = [&](int s) { return bar0 + 8u * (2 + T::KV_SLOTS + s); };
    const uint32_t b_s_full = bar0 + 8u * (2 + 2 * T::KV_SLOTS);  // + 8 g
    const uint32_t b_p_full = b_s_full + 16u, b_o_full = b_p_full + 16u, b_scale = b_o_full + 16u;
    const uint32_t b_done = b_scale + 8u * kScaleRing;

    if ((smem_u32(smem) & 1023u) != 0) {  // swizzle atoms need 1024-byte alignment
        if (threadIdx.x == 0) record_device_error(p.st, ATTN_DEVERR_SMEM_ALIGN, 0x4FF);
        return;
    }
    if (threadIdx.x == 0) {
        for (int g = 0; g < 2; ++g) {
            mbar_init(b_q + 8u * g, 4);       // one arrival per softmax warp
            mbar_init(b_s_full + 8u * g, 1);
            mbar_init(b_p_full + 8u * g, 4);
            mbar_init(b_o_full + 8u * g, 1);
        }
        for (int s = 0; s < T::KV_SLOTS; ++s) {
            mbar_init(b_kv_full(s), kConvWarps);
            mbar_init(b_kv_empty(s), 1);
        }
        for (int s = 0; s < kScaleRing; ++s) mbar_init(b_scale + 8u * s, 1);
        mbar_init(b_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const PromptShare share = prompt_share(p, pairs, reinterpret_cast<PromptShareSmem*>(smem + T::OFF_SHARE));
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    PromptWalk w(share, pairs);
    const int G = p.H / p.Hk;

    if (warp >= 9) {
        // ================= converters =================
        const int cw = warp - 9;
        constexpr int LPR = D / 16, RPI = 32 / LPR;                // lanes a row, rows an instruction
        constexpr int GROUPS = kTile / RPI, PER = (GROUPS + kConvWarps - 1) / kConvWarps;
        const int crow = lane / LPR, cc = lane % LPR;
        const long long kn = p.c.ks.n, vn = p.c.vs.n;
        int idx = 0;   // ring position, over all segments
        int tile_no = 0;  // key tiles converted
        bool ok = true;
        while (ok && w.next(p)) {
            const uint8_t* kbase = p.c.k_pages + w.hk * p.c.ks.h + cc * 16;
            const uint8_t* vbase = p.c.v_pages + w.hk * p.c.vs.h + cc * 16;
            // lanes 0-7 (repeated above): the tile's eight groups of 16 tokens
            long long koff = 0, voff = 0;
            float sk = 1.f, sv = 1.f;
            int tok0 = 0;
            auto find = [&](int v) {  // pages of the walk's v-th key tile
                tok0 = w.u.tile(v) * kTile;
                const int tok = tok0 + (lane & 7) * 16;
                koff = voff = 0;
                sk = sv = 1.f;
                if (tok < w.u.len && (tok + 16 > w.u.key_lo || tok < p.sinks)) {
                    const int pid = cache_page(p.c, p.st, w.b, tok), slot = tok & (p.c.page_size - 1);
                    koff = pid * p.c.ks.b + slot * kn;
                    voff = pid * p.c.vs.b + slot * vn;
                    const long long at = static_cast<long long>(pid) * p.Hk + w.hk;
                    sk = __ldg(p.c.k_scale + at);
                    sv = __ldg(p.c.v_scale + at);
                }
            };
            uint4 kb[PER], vb[PER];
            auto load = [&](uint4 (&buf)[PER], const uint8_t* base, long long off, long long n) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int grp = cw + kConvWarps * i;
                    const int row = grp * RPI + crow;
                    const long long o16 = __shfl_sync(0xffffffffu, off, (grp * RPI) >> 4);
                    const int tok = tok0 + row;
                    buf[i] = make_uint4(0u, 0u, 0u, 0u);  // tokens that no query sees are zeros
                    if (grp < GROUPS && tok < w.u.len && (tok >= w.u.key_lo || tok < p.sinks))
                        buf[i] = __ldg(reinterpret_cast<const uint4*>(base + o16 + (row & 15) * n));
                }
            };
            auto convert = [&](const uint4 (&buf)[PER], bool keys) -> bool {
                const int slot = idx % T::KV_SLOTS, round = idx / T::KV_SLOTS;
                if (round > 0 && !wait_warp(b_kv_empty(slot), (round - 1) & 1, abort_flag, p.st, SITE_KV_EMPTY))
                    return false;
                if (keys && cw == 0) {  // the tile's scales: their entry is free now (see the softmax)
                    if (lane < 8)
                        scales[(tile_no % kScaleRing) * 8 + lane] = make_float4(sk, lg2_approx(sv), rcp_approx(sv), 0.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_scale + 8u * (tile_no % kScaleRing));
                }
                uint8_t* dst = sKV + slot * T::TILE_BYTES;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int grp = cw + kConvWarps * i;
                    if (grp >= GROUPS) break;
                    const int row = grp * RPI + crow;
                    const uint32_t in[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e4m3x4_to_f16(in[k], h[2 * k], h[2 * k + 1]);
                    // 16-byte pieces 2c and 2c + 1 of the row's 128-byte block; lanes of the
                    // second block write them the other way round, so that a quarter warp's
                    // eight pieces lie in different banks
                    uint8_t* at = dst + (cc >> 2) * T::BLK_BYTES + row * 128;
                    const int c = (cc & 3) * 2, flip = (cc >> 2) & 1;
                    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                    *reinterpret_cast<uint4*>(at + (((c + flip) ^ (row & 7)) << 4)) = flip ? hi : lo;
                    *reinterpret_cast<uint4*>(at + (((c + 1 - flip) ^ (row & 7)) << 4)) = flip ? lo : hi;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_kv_full(slot));
                ++idx;
                return true;
            };
            find(w.v0);
            load(kb, kbase, koff, kn);
            for (int v = w.v0; v < w.v1 && ok; ++v) {
                load(vb, vbase, voff, vn);
                ok = convert(kb, true);
                if (!ok) break;
                ++tile_no;
                if (v + 1 < w.v1) {
                    find(v + 1);
                    load(kb, kbase, koff, kn);
                }
                ok = convert(vb, false);
            }
        }
    } else if (warp == 8) {
        // ================= MMA issuer (the whole warp; one elected lane issues) =================
        const SmemDesc dq0 = sw128_desc_words(smem_u32(smem), 16, 1024);                  // Q, K-major
        const SmemDesc dk0 = sw128_desc_words(smem_u32(sKV), 16, 1024);                   // K tiles, K-major
        const SmemDesc dv0 = sw128_desc_words(smem_u32(sKV), T::BLK_BYTES, 1024);         // V tiles, MN-major
        int ring = 0;                // ring position of the segment's first K tile
        int pdone[2] = {0, 0};       // P tiles of query tile g consumed in earlier segments
        int qdone[2] = {0, 0};       // segments in which query tile g was live
        auto slot_desc = [&](SmemDesc base, int i) {
            return desc_add(base, static_cast<uint32_t>((i % T::KV_SLOTS) * T::TILE_BYTES));
        };
        auto wait_kv = [&](int i) {
            return wait_warp(b_kv_full(i % T::KV_SLOTS), (i / T::KV_SLOTS) & 1, abort_flag, p.st, SITE_KV_FULL);
        };
        auto issue_s = [&](int g, int j) {
            const SmemDesc qa = desc_add(dq0, static_cast<uint32_t>(g * T::TILE_BYTES));
            const SmemDesc kd = slot_desc(dk0, ring + 2 * j);
#pragma unroll
            for (int q = 0; q < D / 64; ++q)
                mma_ss_warp4<false, 0, 2, 4, 6, 0, 2, 4, 6>(tmem + (g ? T::COL_S1 : T::COL_S0),
                                                            desc_add(qa, q * T::BLK_BYTES), desc_add(kd, q * T::BLK_BYTES),
                                                            T::IDESC_S, q > 0 ? 1u : 0u);
            mma_commit_warp(b_s_full + 8u * g);
        };
        auto issue_pv = [&](int g, int j) {
            const SmemDesc vd = slot_desc(dv0, ring + 2 * j + 1);
            constexpr uint32_t VS = 16 * 8;  // V rows of one instruction (16), in 16-byte units
#pragma unroll
            for (int q = 0; q < 2; ++q)
                mma_ts_warp4<false, 0, 8, 16, 24, 0, VS, 2 * VS, 3 * VS>(
                    tmem + (g ? T::COL_O1 : T::COL_O0), tmem + (g ? T::COL_S1 : T::COL_S0) + 32 * q,
                    desc_add(vd, static_cast<uint32_t>(4 * q * 16 * 128)), T::IDESC_PV, (j > 0 || q > 0) ? 1u : 0u);
        };
        auto run = [&]() -> bool {
            const int a[2] = {w.a0, w.a1}, steps = w.v1 - w.v0;
            if (!wait_kv(ring)) return false;
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (a[g] > 0) {
                    if (!wait_warp(b_q + 8u * g, qdone[g] & 1, abort_flag, p.st, SITE_Q)) return false;
                    tc_fence_after();
                    issue_s(g, 0);
                }
            mma_commit_warp(b_kv_empty(ring % T::KV_SLOTS));
            for (int j = 0; j < steps; ++j) {
                if (!wait_kv(ring + 2 * j + 1)) return false;                       // V_j
                if (j + 1 < steps && !wait_kv(ring + 2 * j + 2)) return false;      // K_{j+1}
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (j >= a[g]) continue;
                    if (!wait_warp(b_p_full + 8u * g, (pdone[g] + j) & 1, abort_flag, p.st, SITE_P_FULL)) return false;
                    tc_fence_after();
                    issue_pv(g, j);
                    if (j + 1 < a[g]) issue_s(g, j + 1);
                    else mma_commit_warp(b_o_full + 8u * g);
                }
                mma_commit_warp(b_kv_empty((ring + 2 * j + 1) % T::KV_SLOTS));
                if (j + 1 < steps) mma_commit_warp(b_kv_empty((ring + 2 * j + 2) % T::KV_SLOTS));
            }
            return true;
        };
        while (w.next(p)) {
            if (!run()) break;
            ring += 2 * (w.v1 - w.v0);
            pdone[0] += w.a0;
            pdone[1] += w.a1;
            qdone[0] += w.a0 > 0;
            qdone[1] += w.a1 > 0;
        }
        mma_commit_warp(b_done);  // every product has finished before tensor memory is freed
        wait_drain(b_done, 0, p.st, SITE_DRAIN);
    } else {
        // ================= softmax: one thread per row of query tile g =================
        const int g = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + (g ? T::COL_S1 : T::COL_S0) + lane_off;
        const uint32_t tO = tmem + (g ? T::COL_O1 : T::COL_O0) + lane_off;
        const uint32_t b_sf = b_s_full + 8u * g, b_pf = b_p_full + 8u * g, b_of = b_o_full + 8u * g;
        uint8_t* q_row = smem + g * T::TILE_BYTES + row * 128;
        int s_seen = 0, o_seen = 0, tile_no = 0;
        bool ok = true;
        while (ok && w.next(p)) {
            const int n = g ? w.a1 : w.a0;
            const int r = w.pair * kPairRows + g * kTile + row;  // row of the key/value head
            const bool row_ok = r < w.u.rows;
            const int t = row_ok ? r / G : 0, h = w.hk * G + (row_ok ? r - t * G : 0);
            const int pos = row_ok ? w.u.first_pos + t : -1;
            const int key_min = p.left < 0 ? 0 : pos - p.left;
            float rq = 0.f;
            if (n > 0) {
                // Q row to f16, times a power of two.  The tile's place is free: the
                // previous segment's last S_g, read here, came after every product on it.
                uint4 x[D / 8];
                float amax = 0.f;
                const uint16_t* src = static_cast<const uint16_t*>(p.q) + w.b * p.qs.b + h * p.qs.h + t * p.qs.n;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    x[c] = row_ok ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    for (uint32_t u : {x[c].x, x[c].y, x[c].z, x[c].w})
                        amax = fmaxf(amax, fmaxf(fabsf(bf16lo(u)), fabsf(bf16hi(u))));
                const float f = f16_row_scale(amax);
                rq = p.cs * __uint_as_float((254u << 23) - __float_as_uint(f));
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    auto cv = [&](uint32_t u) { return pack_f16x2(bf16lo(u) * f, bf16hi(u) * f); };
                    *reinterpret_cast<uint4*>(q_row + (c >> 3) * T::BLK_BYTES + (((c & 7) ^ (row & 7)) << 4)) =
                        make_uint4(cv(x[c].x), cv(x[c].y), cv(x[c].z), cv(x[c].w));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_q + 8u * g);
            }

            float m_used = -INFINITY;  // running maximum of score + log2 sv (log2 units), possibly stale
            float l_sum = 0.f;         // sum of 2^(score - m_used + kShift) (value scales taken back out)
            for (int j = 0; j < n; ++j) {
                // Scales of key tile j.  Its entry is written again for tile j + 8, once that
                // tile's K slot is free: the one of V(j + 5) (five slots) or K(j + 4) (eight),
                // read by products that follow this warp's arrival for tile j + 3 at least.
                const int tn = tile_no + j;
                if (!wait_warp(b_scale + 8u * (tn % kScaleRing), (tn / kScaleRing) & 1, abort_flag, p.st, SITE_SCALE) ||
                    !wait_warp(b_sf, (s_seen + j) & 1, abort_flag, p.st, SITE_S_FULL)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4* sc = scales + (tn % kScaleRing) * 8;
                uint32_t s[4][32];
                auto load_s = [&]() {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
                    const int kv0 = w.u.tile(w.v0 + j) * kTile;
                    const int c_lo = key_min - kv0, c_hi = pos - kv0, c_sink = p.sinks - kv0;
                    if ((c_lo > 0 && c_sink < c_lo) || c_hi < kTile - 1) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int k = c * 32 + i;
                                if ((k < c_lo && k >= c_sink) || k > c_hi) s[c][i] = f2u(-INFINITY);
                            }
                    }
                };
                load_s();
                float alpha = 1.f;
                bool rescale_o = false;
                auto update_max = [&](float tau) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int grp = 0; grp < 8; ++grp) {
                        const float4 e = sc[grp];
                        const uint32_t* x = s[grp >> 1] + (grp & 1) * 16;
                        float a = fmax3(u2f(x[0]), u2f(x[1]), u2f(x[2]));
#pragma unroll
                        for (int i = 3; i < 15; i += 2) a = fmax3(a, u2f(x[i]), u2f(x[i + 1]));
                        mx = fmaxf(mx, fmaf(fmaxf(a, u2f(x[15])), rq * e.x, e.y));
                    }
                    if (mx > m_used + tau) {
                        alpha = ex2_approx(m_used - mx);  // 0 while m_used is -inf
                        l_sum *= alpha;
                        m_used = mx;
                        rescale_o = j > 0;
                    }
                };
                if (__any_sync(0xffffffffu, m_used == -INFINITY)) update_max(0.f);

                uint32_t pk[2][32];
                float tile_sum, tile_l;
                auto exp_pass = [&]() {
                    const float sub = kShift - (m_used == -INFINITY ? 0.f : m_used);
                    tile_sum = tile_l = 0.f;
#pragma unroll
                    for (int grp = 0; grp < 8; ++grp) {
                        const float4 e = sc[grp];  // the same address in every lane
                        const float f = rq * e.x, add = e.y + sub;
                        const uint32_t* x = s[grp >> 1] + (grp & 1) * 16;
                        float a0 = 0.f, a1 = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float x0, x1;
                            ffma2(x0, x1, u2f(x[i]), u2f(x[i + 1]), f, f, add, add);
                            x0 = ex2_approx(x0);
                            x1 = ex2_approx(x1);
                            // weights rounded to f16 (half a step, 2^-11 relative), finer than the bf16 output
                            pk[grp >> 2][(grp & 3) * 8 + i / 2] = pack_f16x2(x0, x1);
                            fadd2(a0, a1, a0, a1, x0, x1);
                        }
                        tile_sum += a0 + a1;
                        tile_l = fmaf(a0 + a1, e.z, tile_l);
                    }
                };
                exp_pass();
                if (__any_sync(0xffffffffu, !(tile_sum <= kRedoBound))) {
                    // scores rose above m_used: redo the tile with its own maximum
                    load_s();
                    update_max(0.f);
                    exp_pass();
                }
                tmem_st32(tS, pk[0]);
                tmem_st32(tS + 32, pk[1]);
                l_sum += tile_l;
                if (__any_sync(0xffffffffu, rescale_o)) {
                    // PV_g(j-1) has completed: S_g(j) was committed after it
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * alpha);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_pf);
            }
            s_seen += n;
            tile_no += w.v1 - w.v0;
            if (ok && n > 0) {
                ok = wait_warp(b_of, o_seen & 1, abort_flag, p.st, SITE_O_FULL);
                ++o_seen;
                tc_fence_after();
            }
            if (!ok) break;
            const bool finished = w.v0 == 0 && w.v1 == w.u.n;
            // without a live key tile: O = 0 and LSE = +inf, or a segment that takes no part
            const float inv = n > 0 && l_sum != 0.f ? 1.f / l_sum : 0.f;  // NaN stays NaN
            const long long part_row =
                (2ll * blockIdx.x + (w.v0 == 0 ? 1 : 0)) * kPairRows + g * kTile + row;
            uint16_t* orow = static_cast<uint16_t*>(p.o) + w.b * p.os.b + h * p.os.h + t * p.os.n;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                if (!row_ok) continue;
                if (finished) {
                    uint32_t pkd[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) pkd[i] = pack_bf16x2(u2f(o[2 * i]) * inv, u2f(o[2 * i + 1]) * inv);
                    st_global_row64<false>(reinterpret_cast<uint8_t*>(orow + 32 * c), pkd);
                } else {
                    float* dst = p.part + part_row * D + 32 * c;
#pragma unroll
                    for (int v = 0; v < 8; ++v) st_global_v4(dst + 4 * v, o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
            }
            if (row_ok) {
                if (finished)
                    p.lse[(static_cast<long long>(w.b) * p.H + h) * p.T + t] =
                        l_sum != 0.f ? (m_used - kShift + log2f(l_sum)) * kLn2 : INFINITY;
                else
                    p.stat[part_row] = make_float2(l_sum != 0.f ? m_used : -INFINITY, l_sum);
            }
            tc_fence_before();  // O_g may be overwritten once this warp arrives on q_full and p_full
        }
    }

    // what the joining kernel finds at the border before this share
    if (threadIdx.x == 0) {
        CacheBorder bd;
        bd.c_first = -1;
        bd.b = bd.item = bd.q_len = bd.c_last = 0;
        PromptWalk f(share, pairs);
        const long long x = share.x;
        if (f.next(p) && f.v0 > 0) {
            bd.b = f.b;
            bd.item = f.pair * p.Hk + f.hk;
            bd.q_len = f.u.q_len;
            bd.c_first = static_cast<int>(div_mostly32(x - f.v0, share.share)) + 1;
            bd.c_last = static_cast<int>(div_mostly32(x - f.v0 + f.u.n - 1, share.share));
        }
        p.border[blockIdx.x] = bd;
    }
    // ---- teardown: all tensor-memory traffic of this CTA is complete ----
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins unfinished segments row by row (one warp a row), in the order of the keys:
// with M the largest of their maxima, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// The borders inside an item, and gridDim.y blocks each, divide its rows.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache_prompt_join_kernel(const CacheFwdParams p) {
    constexpr int E = D / 32, W = kJoinThreads / 32;
    const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const CacheBorder bd = p.border[c];
    if (bd.c_first < 0) return;
    const int G = p.H / p.Hk, pair = bd.item / p.Hk, hk = bd.item - pair * p.Hk;
    const int rows = min(kPairRows, bd.q_len * G - pair * kPairRows);
    const int n = bd.c_last - bd.c_first + 2, borders = n - 1;
    const int first = ((c - bd.c_first) * static_cast<int>(gridDim.y) + blockIdx.y) * W + warp;
    for (int r = first; r < rows; r += borders * static_cast<int>(gridDim.y) * W) {
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int i = 0; i < n; ++i) {
            const long long at = (2ll * (bd.c_first - 1 + i) + (i == 0 ? 1 : 0)) * kPairRows + r;
            const float2 st = p.stat[at];
            if (st.x == -INFINITY && st.y == 0.f) continue;  // no key of it seen
            const float* src = p.part + at * D + lane * E;
            const float x = fmaxf(m, st.x), a = m == -INFINITY ? 0.f : ex2_approx(m - x), f = ex2_approx(st.x - x);
            m = x;
            l = l * a + st.y * f;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 y = *reinterpret_cast<const float2*>(src + e);
                o[e] = o[e] * a + y.x * f;
                o[e + 1] = o[e + 1] * a + y.y * f;
            }
        }
        const int row = pair * kPairRows + r, t = row / G, h = hk * G + row - t * G;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint16_t* dst = static_cast<uint16_t*>(p.o) + bd.b * p.os.b + h * p.os.h + t * p.os.n + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
        if (lane == 0)
            p.lse[(static_cast<long long>(bd.b) * p.H + h) * p.T + t] =
                l != 0.f ? (m - kShift + log2f(l)) * kLn2 : INFINITY;
    }
}

template <int D>
cudaError_t launch_prompt_impl(CacheFwdParams p, cudaStream_t stream) {
    using T = PromptTraits<D>;
    static const cudaError_t attr = cudaFuncSetAttribute(
        cache_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES);
    if (attr != cudaSuccess) return attr;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.rows = kPairRows;
    p.grid = sms < kPromptGridMax ? sms : kPromptGridMax;
    const long long rows = static_cast<long long>(p.T) * (p.H / p.Hk);
    const int pairs = static_cast<int>((rows + kPairRows - 1) / kPairRows);
    if ((e = dbg_set_word(p.st.word, stream)) != cudaSuccess) return e;
    cache_prompt_kernel<D><<<p.grid, kPromptThreads, T::SMEM_BYTES, stream>>>(p, pairs);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.grid == 1) return e;
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.grid - 1), 8);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_prompt_join_kernel<D>, p);
}

}  // namespace

cudaError_t launch_cache_prompt(const CacheFwdParams& p, cudaStream_t stream) {
    if (p.D == 64) return launch_prompt_impl<64>(p, stream);
    if (p.D == 128) return launch_prompt_impl<128>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
