// Attention of many new queries per sequence (chunks of a prompt) over the paged
// 8-bit cache, on the fifth-generation tensor cores.
//
// An item is (sequence, two adjacent 128-row query tiles, key/value head); the rows
// of a key/value head are its H/Hk query heads of every new query, row = t * H/Hk +
// g, so that grouped heads fill the tiles and share the keys.  The item's key tiles
// of 128 tokens stream through a shared-memory ring:
//
//   warps 12-15 converters: read the codes of a key or value tile page by page,
//               turn them into f16 (exact) and write them where the tensor core
//               expects them (128-byte swizzle)
//   warp 8      MMA issuer: S_g = Q_g K_j^T and O_g += P_g V_j, accumulators in
//               tensor memory, order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
//   warps 0-3   softmax of query tile 0 (one thread per row), which also bring the
//   warps 4-7   tile's Q rows to f16; the same for query tile 1
//   warps 9-11  next to nothing (warps come in fours for the register split)
//
// Bound by the chain S -> softmax -> PV of the two query tiles: a key tile's step takes
// about 3700 cycles, of which 2048 are products and 1650 the pass of one tile's softmax;
// the products' operands (S 128 bytes a cycle, PV 64) and the converters' writes together
// fill what shared memory gives.  2 x 2048 queries over 16384 keys (32/8 heads): d = 128
// 596 us, 1.2 PFLOP/s; d = 64 485 us, 0.74 (the same softmax, half the products).  Codes are
// turned into f16 and not used as E4M3 operands, because then Q and the weights would have to
// be E4M3 too (2^-4 relative).  A page's scales enter in fp32 as in the kernel for few
// queries: score * key scale, + log2 of the value scale in the exponent, and 1 / value scale in
// the sum (kScaleReach).
//
// The work is shared out as there: items laid end to end by their key tiles, an
// equal share for each CTA, unfinished segments joined by a second kernel.  Whole
// items would leave SMs idle in the last of few rounds (512 equal items on 152 SMs:
// 16 %).
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

// sum of 32 weights from which on they are formed again (a weight in f16 ends at 2^16)
constexpr float kWeightMax = 32768.f;
constexpr int kPairRows = 2 * kTile;
constexpr int kPromptThreads = 512;
constexpr int kConvWarps = 4;
constexpr int kAhead = 3;  // tiles
// Registers a thread: the launch's 128 are dealt out again, more for the softmax, less
// for the MMA issuer's four warps.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 152, kMmaRegs = 80, kConvRegs = 128;
static_assert(2 * kSoftmaxRegs + kMmaRegs + kConvRegs <= 4 * kLaunchRegs, "more registers than the launch has");
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

enum : uint32_t {
    SITE_Q = 0x401, SITE_KV_EMPTY = 0x402, SITE_KV_FULL = 0x403, SITE_P_FULL = 0x404, SITE_S_FULL = 0x405,
    SITE_O_FULL = 0x406, SITE_DRAIN = 0x407, SITE_SCALE = 0x408, SITE_MERGE = 0x409,
};

constexpr uint32_t kFmtF16 = 0;

template <int D>
struct PromptTraits {
    static constexpr int NBLK = D / 64;             // 128-byte column blocks of an f16 row
    static constexpr int BLK_BYTES = kTile * 128;
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int KV_SLOTS = D == 128 ? 5 : 8;
    static constexpr int SCALES = D == 128 ? 4 : 8;  // ring of the key tiles' scales
    static constexpr int SMEM_Q = 2 * TILE_BYTES;
    static constexpr int OFF_KV = SMEM_Q;
    static constexpr int OFF_SCALE = OFF_KV + KV_SLOTS * TILE_BYTES;  // float4 [SCALES][8]
    static constexpr int OFF_BAR = OFF_SCALE + SCALES * 8 * 16;
    // q_full[2], kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], scale_full[SCALES], done,
    // merge, merged
    static constexpr int NBARS = 2 + 2 * KV_SLOTS + 6 + SCALES + 3;
    static constexpr int OFF_WALK = (OFF_BAR + NBARS * 8 + 16 + 15) & ~15;  // a walk per warp; the share's scratch before
    static constexpr int SMEM_BYTES = OFF_WALK + 14 * 128;  // warps 0-9 and 12-15
    static constexpr uint32_t COL_S0 = 0, COL_S1 = 128, COL_O0 = 256, COL_O1 = 256 + D;
    static constexpr uint32_t IDESC_S = make_idesc(kFmtF16, kTile, kTile, false, false);
    static constexpr uint32_t IDESC_PV = make_idesc(kFmtF16, kTile, D, false, true);
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// wait_warp without its out-of-line half: ptxas deals out registers to parts of a
// kernel only where they call nothing.
__device__ __forceinline__ bool wait_in_line(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             const DevStatus& st, uint32_t site) {
    return wait_warp_loop(bar, parity, abort_flag, st.word, st.wait_limit_ns, site);
}

// A pair of query tiles of a sequence and the n key tiles it walks: the n_sink first
// ones of the sequence, then those from lo on.  Query tile g uses the first n_g of
// them; or, where the pair has rows for one query tile only (dual), the two softmax
// groups take its key tiles in turn: alone, a query tile's chain of products and
// softmax would leave the tensor cores idle most of the time.
struct PromptUnit {
    int len, q_len, rows;
    int first_pos;  // position of query 0 (negative: rows before the first token see nothing)
    int pos_lo, pos_hi;  // positions of the pair's first and last row
    int key_lo;     // first key of the window of the pair's first query
    int n_sink, lo, dual, n, n0, n1;
    __host__ __device__ int tile(int t) const { return t < n_sink ? t : lo + t - n_sink; }
    // Every row of the pair sees every token of key tile t.  Those of a walk that it does not
    // are the few at the diagonal, the window's edge and the last sink.
    __host__ __device__ bool all_see(int t, int left, int sinks) const {
        const int kv0 = tile(t) * kTile;
        return kv0 + kTile - 1 <= pos_lo && (left < 0 || kv0 >= pos_hi - left || kv0 + kTile <= sinks);
    }
};

__host__ __device__ inline PromptUnit prompt_unit(const CacheFwdParams& p, int b, int pair) {
    PromptUnit u;
    const int G = p.H / p.Hk, cap = p.c.max_pages * p.c.page_size;
    u.len = min(max(p.c.seq_lens[b], 0), cap);
    u.q_len = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
    u.rows = u.q_len * G;
    u.first_pos = u.len - u.q_len;
    u.n = u.n0 = u.n1 = u.n_sink = u.lo = u.key_lo = u.dual = u.pos_lo = u.pos_hi = 0;
    const int r0 = pair * kPairRows;
    if (r0 >= u.rows) return u;  // no such pair: no work
    u.pos_lo = u.first_pos + r0 / G;
    u.pos_hi = u.first_pos + min(u.rows - 1, r0 + kPairRows - 1) / G;
    u.key_lo = p.left < 0 ? 0 : max(0, max(0, u.pos_lo) - p.left);
    u.lo = u.key_lo / kTile;
    u.n_sink = min((min(p.sinks, u.key_lo) + kTile - 1) / kTile, u.lo);
    auto tiles = [&](int row_hi) {  // up to the key tile of the last position of rows .. row_hi
        const int pos = u.first_pos + min(u.rows - 1, row_hi) / G;
        return pos < 0 ? 0 : u.n_sink + pos / kTile - u.lo + 1;
    };
    u.dual = r0 + kTile >= u.rows;
    u.n0 = tiles(r0 + kTile - 1);
    u.n1 = u.dual ? u.n0 : tiles(r0 + kPairRows - 1);
    u.n = max(1, u.n1);  // one that no row sees stands for none
    return u;
}

// The same of a launch's part of the sequences.  A group's prefix: the rows of all its sequences
// are one sequence's, all of them behind its last key.  32 sequences of 8 rows behind 131072 tokens, 4
// heads, d = 128: 82 us, 0.82 PFLOP/s, 3400 cycles a key tile and 31000 before the first and behind the
// last; 64 of 4 rows behind 8192, 8 heads: 30 us, of which 8 are key tiles.
template <CachePart PART>
__device__ __forceinline__ PromptUnit unit_of(const CacheFwdParams& p, int b, int pair) {
    static_assert(PART != kRest, "the rest of a sequence is for the kernel of few queries");
    if constexpr (PART == kPrefix) {
        PromptUnit u;
        u.len = group_len(p, b);
        u.q_len = max(0, group_end(p, b) - group_begin(p, b)) * p.T;
        u.rows = u.q_len * (p.H / p.Hk);
        u.first_pos = u.pos_lo = u.pos_hi = u.len - 1;
        const int r0 = pair * kPairRows;
        u.n = u.n0 = u.n1 = r0 < u.rows ? u.len / kTile : 0;
        u.dual = r0 + kTile >= u.rows;
        u.n_sink = u.lo = u.key_lo = 0;
        return u;
    }
    return prompt_unit(p, b, pair);
}

// Tiles [first, end) of a segment [v0, v1), tile t0 of its CTA the first, that lie among the
// CTA's tiles lo .. hi (none: INT_MAX, -1).
struct TileSpan {
    int first, end;
};
__host__ __device__ __forceinline__ TileSpan segment_span(int lo, int hi, int t0, int v0, int v1) {
    if (hi < lo || hi < t0 || lo - t0 >= v1 - v0) return {v0, v0};
    return {v0 + (lo > t0 ? lo - t0 : 0), v0 + (hi - t0 < v1 - v0 ? hi - t0 + 1 : v1 - v0)};
}

// A CTA's share: key tiles [x, x_end) of the line on which the units' items lie end to
// end (each unit once per key/value head), starting in unit `unit`, before which lie
// unit_first key tiles.  unit < 0: nothing.
struct PromptShare {
    long long share, x, x_end, unit_first;
    int unit;
};

struct PromptShareSmem {
    long long warp_sum[kPromptThreads / 32], unit_first;
    int unit;
};

__device__ PromptShare prompt_share(const CacheFwdParams& p, int pairs, PromptShareSmem* sm) {
    constexpr int W = kPromptThreads / 32;
    const int units = p.B * pairs, per = (units + kPromptThreads - 1) / kPromptThreads;
    const int u0 = min(units, static_cast<int>(threadIdx.x) * per), u1 = min(units, u0 + per);
    auto work = [&](int u) { return static_cast<long long>(prompt_unit(p, u / pairs, u % pairs).n) * p.Hk; };
    long long mine = 0;
    for (int u = u0; u < u1; ++u) {
        if (blockIdx.x == 0 && u % pairs == 0) check_len(p.c, p.st, u / pairs);
        mine += work(u);
    }
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

// The same for the prefixes' launch, by each warp for itself, without a barrier; a group's units are
// numbered as if each had as many as all rows fill.
__device__ __forceinline__ PromptShare prefix_share(const CacheFwdParams& p, int pairs) {
    const int lane = threadIdx.x & 31, per = (p.groups + 31) >> 5;
    const int g0 = min(p.groups, lane * per), g1 = min(p.groups, g0 + per);
    auto unit_work = [&](const PromptUnit& u) { return static_cast<long long>(u.n) * p.Hk; };
    auto work = [&](int g) {
        const PromptUnit u = unit_of<kPrefix>(p, g, 0);
        return unit_work(u) * ((u.rows + kPairRows - 1) / kPairRows);
    };
    long long mine = 0;
    for (int g = g0; g < g1; ++g) mine += work(g);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    PromptShare s;
    s.share = max(div_mostly32(total + p.grid - 1, p.grid), 1ll);
    s.x = blockIdx.x * s.share;
    s.x_end = min(s.x + s.share, total);
    long long before = incl - mine;
    int found = -1;
    if (s.x < total && before <= s.x && s.x < incl) {
        for (int g = g0; g < g1; ++g) {
            const long long w = work(g);
            if (s.x < before + w) {
                const long long each = unit_work(unit_of<kPrefix>(p, g, 0));
                const int pair = static_cast<int>(div_mostly32(s.x - before, each));
                found = g * pairs + pair;
                before += pair * each;
                break;
            }
            before += w;
        }
    }
    const unsigned who = __ballot_sync(0xffffffffu, found >= 0);
    const int src = who ? __ffs(who) - 1 : 0;
    s.unit = __shfl_sync(0xffffffffu, found, src);
    s.unit_first = __shfl_sync(0xffffffffu, before, src);
    return s;
}

// Walks the segments of a share, for every role alike.  Each warp keeps its own walk
// in shared memory: its fields are read a few times a tile, and the softmax has no
// registers for them.
struct PromptWalk {
    PromptShare s;
    PromptUnit u;
    int pairs, b, pair, hk;
    int known;   // u is that of (b, pair)
    int v0, v1;  // key tiles [v0, v1) of the item
    int a0, a1;  // those that softmax group g takes: the first a_g, or (dual) v0 + g, v0 + g + 2, ...
};
// By a whole warp; every lane works out the same step.
template <CachePart PART>
__device__ __forceinline__ bool next_segment(const CacheFwdParams& p, PromptWalk* walk) {
    PromptWalk w = *walk;
    __syncwarp();
    if (w.s.unit < 0 || w.s.x >= w.s.x_end) return false;
    if (!w.known) w.u = unit_of<PART>(p, w.b, w.pair);
    w.known = 1;
    for (long long n; w.s.x >= w.s.unit_first + (n = static_cast<long long>(w.u.n) * p.Hk);) {
        w.s.unit_first += n;
        // (the units of a group behind its last rows are passed over at once)
        if (++w.pair == w.pairs || (PART == kPrefix && n == 0)) {
            w.pair = 0;
            ++w.b;
        }
        w.u = unit_of<PART>(p, w.b, w.pair);
    }
    w.hk = static_cast<int>(div_mostly32(w.s.x - w.s.unit_first, w.u.n));
    w.v0 = static_cast<int>((w.s.x - w.s.unit_first) - static_cast<long long>(w.hk) * w.u.n);
    w.v1 = static_cast<int>(min(static_cast<long long>(w.u.n), w.v0 + (w.s.x_end - w.s.x)));
    w.a0 = max(0, min(w.v1, w.u.n0) - w.v0);
    w.a1 = max(0, min(w.v1, w.u.n1) - w.v0);
    if (w.u.dual) {
        w.a1 = w.a0 / 2;
        w.a0 -= w.a1;
    }
    w.s.x += w.v1 - w.v0;
    if ((threadIdx.x & 31) == 0) *walk = w;
    __syncwarp();
    return true;
}

template <int D, CachePart PART>
__global__ void __launch_bounds__(kPromptThreads, 1) cache_prompt_kernel(const CacheFwdParams p, const int pairs) {
    using T = PromptTraits<D>;
    pdl_wait();
    if (PART == kPrefix && blockIdx.x == 0 && threadIdx.x == 0) open_rest(p);
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* sKV = smem + T::OFF_KV;
    float4* scales = reinterpret_cast<float4*>(smem + T::OFF_SCALE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + T::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // first and last key tile of this CTA with a NaN value that not every row of its pair sees
    int* nan_tiles = reinterpret_cast<int*>(tmem_slot + 2);
    const uint32_t bar0 = smem_u32(bars);
    const uint32_t b_q = bar0;  // + 8 g
    auto b_kv_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto b_kv_empty = [&](int s) { return bar0 + 8u * (2 + T::KV_SLOTS + s); };
    const uint32_t b_s_full = bar0 + 8u * (2 + 2 * T::KV_SLOTS);  // + 8 g
    const uint32_t b_p_full = b_s_full + 16u, b_o_full = b_p_full + 16u, b_scale = b_o_full + 16u;
    const uint32_t b_done = b_scale + 8u * T::SCALES;
    const uint32_t b_merge = b_done + 8u, b_merged = b_done + 16u;  // dual items: group 1's part is there / has been read

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
        for (int s = 0; s < T::SCALES; ++s) mbar_init(b_scale + 8u * s, kConvWarps);
        mbar_init(b_done, 1);
        mbar_init(b_merge, 4);
        mbar_init(b_merged, 4);
        *abort_flag = 0;
        nan_tiles[0] = INT_MAX;
        nan_tiles[1] = -1;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    static_assert(sizeof(PromptWalk) <= 128 && sizeof(PromptShareSmem) <= 256, "walk slots");
    PromptWalk* const walk = reinterpret_cast<PromptWalk*>(smem + T::OFF_WALK + (warp < 10 ? warp : warp - 2) * 128);
    {
        PromptShare share;
        if constexpr (PART == kPrefix) share = prefix_share(p, pairs);
        else share = prompt_share(p, pairs, reinterpret_cast<PromptShareSmem*>(smem + T::OFF_WALK));
        __syncthreads();  // the scratch has been read
        if (lane == 0 && (warp < 10 || warp >= 12)) {
            walk->s = share;
            walk->pairs = pairs;
            walk->b = share.unit / pairs;
            walk->pair = share.unit - walk->b * pairs;
            walk->known = 0;
        }
        __syncwarp();
    }
    const PromptWalk& w = *walk;
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    const int G = p.H / p.Hk;

    if (warp >= 12) {
        // ================= converters: 16-token groups 2 cw and 2 cw + 1 of every tile =================
        regs_dec<kConvRegs>();
        const int cw = warp - 12;
        constexpr int RPI = 512 / D, NI = 16 / RPI;  // rows a warp instruction loads, and those a group
        // Lane -> row of an instruction and 16-code piece of it: a quarter warp takes two
        // neighbouring rows, four pieces of one 128-byte block each, so that the f16 pieces it
        // writes lie in eight different banks.
        const int crow = D == 128 ? (lane >> 2) & 3 : lane >> 2;
        const int cc = D == 128 ? (lane & 3) | (lane >> 4 << 2) : lane & 3;
        const long long kn = p.c.ks.n, vn = p.c.vs.n;
        // f16 pieces 2c and 2c + 1 in row crow of this warp's part of a tile
        const uint32_t row_at = (cc >> 2) * T::BLK_BYTES + cw * 32 * 128 + crow * 128, c2 = (cc & 3) * 2;
        const uint32_t at0 = row_at + ((c2 ^ crow) << 4), at1 = row_at + (((c2 + 1) ^ crow) << 4);
        int idx = 0;      // ring position, over all segments
        int tile_no = 0;  // key tiles converted
        bool ok = true;
        while (ok && next_segment<PART>(p, walk)) {
            const uint8_t* kbase = p.c.k_pages + w.hk * p.c.ks.h + crow * kn + cc * 16;
            const uint8_t* vbase = p.c.v_pages + w.hk * p.c.vs.h + crow * vn + cc * 16;
            const int len = w.u.len, key_lo = w.u.key_lo;
            // Sequence whose table is read: of a group the first one that has queries (a slot of a
            // batch that has none may hold any table; a group without queries reads page 0, to no end).
            int seq = PART == kPrefix ? group_begin(p, w.b) : w.b;
            auto first_tok = [&](int t) { return w.u.tile(t) * kTile + cw * 32; };
            // some query sees a token of the group from tok on
            auto needed = [&](int tok) { return tok < len && (PART == kPrefix || tok + 16 > key_lo || tok < p.sinks); };
            // Page numbers of both groups of 16 tiles at a time, lane 2i + g holding group g of
            // tile i, fetched 16 tiles before their use (shared memory leaves the L1 no room:
            // each look at the table goes to the L2).
            auto fetch = [&](int t) {
                const int x = t + (lane >> 1), tok = x < w.v1 ? first_tok(x) + 16 * (lane & 1) : len;
                return needed(tok) && (PART != kPrefix || seq >= 0) ? __ldg(p.c.table + seq * p.c.table_stride + (tok >> p.c.page_shift)) : 0;
            };
            auto checked = [&](int pid) {
                if (static_cast<unsigned>(pid) < static_cast<unsigned>(p.c.num_pages)) return pid;
                record_device_error(p.st, ATTN_DEVERR_PAGE, 0x401);
                return 0;
            };
            // codes of both groups; tokens that no query sees are not read and count as zeros
            auto load = [&](uint4 (&buf)[2 * NI], const uint8_t* base, const Strides& st, int tok0, const int (&pid)[2]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = tok0 + 16 * i;
                    const uint8_t* src = base + pid[i] * st.b + (tok & (p.c.page_size - 1)) * st.n;
                    if (PART == kPrefix || (tok + 16 <= len && (tok >= key_lo || tok + 16 <= p.sinks))) {
#pragma unroll
                        for (int k = 0; k < NI; ++k) buf[i * NI + k] = __ldg(reinterpret_cast<const uint4*>(src + k * RPI * st.n));
                    } else {
#pragma unroll
                        for (int k = 0; k < NI; ++k) {
                            const int x = tok + k * RPI + crow;
                            buf[i * NI + k] = make_uint4(0u, 0u, 0u, 0u);
                            if (x < len && (x >= key_lo || x < p.sinks))
                                buf[i * NI + k] = __ldg(reinterpret_cast<const uint4*>(src + k * RPI * st.n));
                        }
                    }
                }
            };
            auto claim = [&]() {
                const int round = idx / T::KV_SLOTS;
                return round == 0 || wait_in_line(b_kv_empty(idx % T::KV_SLOTS), (round - 1) & 1, abort_flag, p.st, SITE_KV_EMPTY);
            };
            auto convert = [&](const uint4 (&buf)[2 * NI], int t, bool values) {
                const int slot = idx % T::KV_SLOTS;
                uint8_t* dst = sKV + slot * T::TILE_BYTES;
                uint32_t nan[4] = {0u, 0u, 0u, 0u};  // a byte's top bit: a NaN code (7F or FF) in its column
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < NI; ++k) {
                        const uint4 x = buf[i * NI + k];
                        uint32_t h[8];
                        e4m3x4_to_f16(x.x, h[0], h[1]);
                        e4m3x4_to_f16(x.y, h[2], h[3]);
                        e4m3x4_to_f16(x.z, h[4], h[5]);
                        e4m3x4_to_f16(x.w, h[6], h[7]);
                        if (values && PART == kWhole) {  // (every row sees all of a prefix)
                            nan[0] |= (x.x & 0x7F7F7F7Fu) + 0x01010101u;
                            nan[1] |= (x.y & 0x7F7F7F7Fu) + 0x01010101u;
                            nan[2] |= (x.z & 0x7F7F7F7Fu) + 0x01010101u;
                            nan[3] |= (x.w & 0x7F7F7F7Fu) + 0x01010101u;
                        }
                        const uint32_t more = (i * 16 + k * RPI) * 128, sw = ((k * RPI) & 7) << 4;  // swizzle of the row
                        *reinterpret_cast<uint4*>(dst + more + (at0 ^ sw)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(dst + more + (at1 ^ sw)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                // A weight of 0 times NaN is NaN: right where every row sees the tile, and elsewhere
                // NaN values stand as 0 in the products, and the rows that see one get it at the end
                // of the segment.
                if (values && PART == kWhole) {
                    if (__any_sync(0xffffffffu, ((nan[0] | nan[1] | nan[2] | nan[3]) & 0x80808080u) != 0u) &&
                        !w.u.all_see(t, p.left, p.sinks)) {
#pragma unroll 1
                        for (int i = 0; i < 4 * NI; ++i) {
                            const int k = (i >> 1) % NI;
                            uint32_t* at = reinterpret_cast<uint32_t*>(dst + ((i >> 1) / NI * 16 + k * RPI) * 128 +
                                                                       ((i & 1 ? at1 : at0) ^ (((k * RPI) & 7) << 4)));
#pragma unroll 1
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t h = at[e];
                                at[e] = ((h & 0x7FFFu) > 0x7C00u ? 0u : h & 0xFFFFu) |
                                        ((h & 0x7FFF0000u) > 0x7C000000u ? 0u : h & 0xFFFF0000u);
                            }
                        }
                        if (lane == 0) {
                            atomicMin(nan_tiles, tile_no - 1);
                            atomicMax(nan_tiles + 1, tile_no - 1);
                        }
                        __syncwarp();
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_kv_full(slot));
                ++idx;
            };
            // lanes 0 and 1: the scales of group `lane`
            float sk = 1.f, sv = 1.f;
            auto load_scales = [&](int tok0, const int (&pid)[2]) {
                const int i = lane & 1;
                sv = 1.f;
                if (lane < 2 && needed(tok0 + 16 * i)) {
                    const long long at = static_cast<long long>(i ? pid[1] : pid[0]) * p.Hk + w.hk;
                    sk = __ldg(p.c.k_scale + at);
                    sv = __ldg(p.c.v_scale + at);
                }
            };
            // Loads run ahead of their use: V of the tile before K is converted, K of the next
            // one before V is.
            uint4 kb[2 * NI], vb[2 * NI];
            int pages = fetch(w.v0), pages_next = fetch(w.v0 + 16), pid[2];
            if constexpr (PART == kPrefix) {
                if (query_count(p, seq) == 0) {
                    const int end = group_end(p, w.b);
                    do ++seq;
                    while (seq < end && query_count(p, seq) == 0);
                    if (seq == end) seq = -1;
                    pages = fetch(w.v0);
                    pages_next = fetch(w.v0 + 16);
                }
            }
            pages = checked(pages);
            auto take_pages = [&](int i) {  // of the segment's i-th tile
                if (i > 0 && (i & 15) == 0) {
                    pages = checked(pages_next);
                    pages_next = fetch(w.v0 + i + 16);
                }
                pid[0] = __shfl_sync(0xffffffffu, pages, 2 * (i & 15));
                pid[1] = __shfl_sync(0xffffffffu, pages, 2 * (i & 15) + 1);
            };
            const int tiles = w.v1 - w.v0;
            // A prefix's keys are read once, by this CTA: they are called into the L2 kAhead tiles before
            // their use.  The loads themselves are a half tile ahead, which covers the L2's latency and
            // not the memory's (32 sequences behind 131072 tokens: 105 us for 115).
            auto call_in = [&](int i) {  // lane: one of the warp's 32 tokens of the segment's i-th tile
                if (i >= tiles) return;
                const int from = (i & ~15) == ((i - kAhead > 0 ? i - kAhead : 0) & ~15) ? pages : pages_next;
                const int pg = __shfl_sync(0xffffffffu, from, 2 * (i & 15) + (lane >> 4)), tok = first_tok(w.v0 + i) + lane;
                if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.c.num_pages)) return;
                const long long slot = tok & (p.c.page_size - 1);
                prefetch_l2(p.c.k_pages + pg * p.c.ks.b + w.hk * p.c.ks.h + slot * p.c.ks.n);
                prefetch_l2(p.c.v_pages + pg * p.c.vs.b + w.hk * p.c.vs.h + slot * p.c.vs.n);
            };
            if constexpr (PART == kPrefix) {
                for (int i = 1; i <= kAhead; ++i) call_in(i);
            }
            int tok0 = first_tok(w.v0);
            if (tiles > 0) {
                take_pages(0);
                load(kb, kbase, p.c.ks, tok0, pid);
                load_scales(tok0, pid);
            }
            for (int i = 0; i < tiles; ++i) {
                load(vb, vbase, p.c.vs, tok0, pid);
                if constexpr (PART == kPrefix) {
                    if (i > 0) call_in(i + kAhead);
                }
                if (!(ok = claim())) break;
                // the scales' entry of the tile is free now as well (see the softmax)
                if (lane < 2) {
                    const float lsv = lg2_approx(sv);
                    scales[(tile_no % T::SCALES) * 8 + 2 * cw + lane] =
                        make_float4(sk, lsv, rcp_approx(sv), fabsf(lsv) <= kScaleReach ? 0.f : 1.f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(b_scale + 8u * (tile_no % T::SCALES));
                convert(kb, w.v0 + i, false);
                ++tile_no;
                if (i + 1 < tiles) {
                    tok0 = first_tok(w.v0 + i + 1);
                    take_pages(i + 1);
                    load(kb, kbase, p.c.ks, tok0, pid);
                    load_scales(tok0, pid);
                }
                if (!(ok = claim())) break;
                convert(vb, w.v0 + i, true);
            }
        }
    } else if (warp >= 8) {
        regs_dec<kMmaRegs>();
        if (warp == 8) {
        // ================= MMA issuer (the whole warp; one elected lane issues) =================
        const SmemDesc dq0 = sw128_desc_words(smem_u32(smem), 16, 1024);                  // Q, K-major
        const SmemDesc dk0 = sw128_desc_words(smem_u32(sKV), 16, 1024);                   // K tiles, K-major
        const SmemDesc dv0 = sw128_desc_words(smem_u32(sKV), T::BLK_BYTES, 1024);         // V tiles, MN-major
        int ring = 0;                // ring position of the segment's first K tile
        int pdone0 = 0, pdone1 = 0;  // P tiles of group g consumed in earlier segments
        int qdone0 = 0, qdone1 = 0;  // segments in which group g was live
        auto slot_desc = [&](SmemDesc base, int i) {
            return desc_add(base, static_cast<uint32_t>((i % T::KV_SLOTS) * T::TILE_BYTES));
        };
        auto wait_kv = [&](int i) {
            return wait_in_line(b_kv_full(i % T::KV_SLOTS), (i / T::KV_SLOTS) & 1, abort_flag, p.st, SITE_KV_FULL);
        };
        auto release = [&](int i) { mma_commit_warp(b_kv_empty(i % T::KV_SLOTS)); };
        auto issue_s = [&](int g, int ki) {  // S_g = Q_g K^T, K in ring position ki
            const SmemDesc qa = desc_add(dq0, static_cast<uint32_t>(g * T::TILE_BYTES));
            const SmemDesc kd = slot_desc(dk0, ki);
#pragma unroll
            for (int q = 0; q < D / 64; ++q)
                mma_ss_warp4<false, 0, 2, 4, 6, 0, 2, 4, 6>(tmem + (g ? T::COL_S1 : T::COL_S0),
                                                            desc_add(qa, q * T::BLK_BYTES), desc_add(kd, q * T::BLK_BYTES),
                                                            T::IDESC_S, q > 0 ? 1u : 0u);
            mma_commit_warp(b_s_full + 8u * g);
        };
        auto issue_pv = [&](int g, int vi, bool first) {  // O_g += P_g V, V in ring position vi
            const SmemDesc vd = slot_desc(dv0, vi);
            constexpr uint32_t VS = 16 * 8;  // V rows of one instruction (16), in 16-byte units
#pragma unroll
            for (int q = 0; q < 2; ++q)
                mma_ts_warp4<false, 0, 8, 16, 24, 0, VS, 2 * VS, 3 * VS>(
                    tmem + (g ? T::COL_O1 : T::COL_O0), tmem + (g ? T::COL_S1 : T::COL_S0) + 32 * q,
                    desc_add(vd, static_cast<uint32_t>(4 * q * 16 * 128)), T::IDESC_PV, (!first || q > 0) ? 1u : 0u);
        };
        auto wait_q = [&](int g) {
            const bool ok = wait_in_line(b_q + 8u * g, (g ? qdone1 : qdone0) & 1, abort_flag, p.st, SITE_Q);
            tc_fence_after();
            return ok;
        };
        auto wait_p = [&](int g, int j) {
            const bool ok = wait_in_line(b_p_full + 8u * g, ((g ? pdone1 : pdone0) + j) & 1, abort_flag, p.st, SITE_P_FULL);
            tc_fence_after();
            return ok;
        };
        // One copy of the products' code for both groups: it competes for the instruction cache with the
        // other roles' (2 x 2048 queries over 16384 keys 599 us for 611, 149 -> 131 with a window of 1023;
        // d = 64, whose code is shorter, 488 with two copies and 499 with one).
        constexpr int kRolled = D == 64 ? 2 : 1;
        // Every tile's full barrier is waited for, used or not: a phase that is skipped would
        // be taken for a later one.
        auto run_pair = [&](int a0, int a1, int steps) -> bool {
            if (!wait_kv(ring)) return false;
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if ((g ? a1 : a0) > 0) {
                    if (!wait_q(g)) return false;
                    issue_s(g, ring);
                }
            release(ring);
            for (int j = 0; j < steps; ++j) {
                const int vi = ring + 2 * j + 1;
                // both before P's, off the chain: a look at a barrier takes 250-350 cycles while
                // products run, and neither tile's slot waits for this step
                if (!wait_kv(vi) || (j + 1 < steps && !wait_kv(vi + 1))) return false;
#pragma unroll kRolled
                for (int g = 0; g < 2; ++g) {
                    const int a = g ? a1 : a0;
                    if (j >= a) continue;
                    if (!wait_p(g, j)) return false;
                    issue_pv(g, vi, j == 0);
                    if (j + 1 < a) {
                        issue_s(g, vi + 1);
                    } else {
                        mma_commit_warp(b_o_full + 8u * g);
                    }
                }
                release(vi);
                if (j + 1 < steps) release(vi + 1);
            }
            return true;
        };
        auto run_dual = [&](int a0, int a1) -> bool {  // group g: tiles g, g + 2, ... of the segment
            if (a0 == 0) {  // the tile that stands for none
                if (!wait_kv(ring) || !wait_kv(ring + 1)) return false;
                release(ring);
                release(ring + 1);
            }
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if ((g ? a1 : a0) > 0) {
                    if (!wait_kv(ring + 2 * g) || !wait_q(g)) return false;
                    issue_s(g, ring + 2 * g);
                    release(ring + 2 * g);
                }
            for (int j = 0; j < a0; ++j)
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {
                    const int a = g ? a1 : a0, vi = ring + 4 * j + 2 * g + 1;
                    if (j >= a) continue;
                    if (!wait_kv(vi) || (j + 1 < a && !wait_kv(vi + 3)) || !wait_p(g, j)) return false;
                    issue_pv(g, vi, j == 0);
                    release(vi);
                    if (j + 1 < a) {
                        issue_s(g, vi + 3);
                        release(vi + 3);
                    } else {
                        mma_commit_warp(b_o_full + 8u * g);
                    }
                }
            return true;
        };
        while (next_segment<PART>(p, walk)) {
            const int a0 = w.a0, a1 = w.a1;
            if (!(w.u.dual ? run_dual(a0, a1) : run_pair(a0, a1, w.v1 - w.v0))) break;
            ring += 2 * (w.v1 - w.v0);
            pdone0 += a0;
            pdone1 += a1;
            qdone0 += a0 > 0;
            qdone1 += a1 > 0;
        }
        mma_commit_warp(b_done);  // every product has finished before tensor memory is freed
        wait_drain_loop(b_done, 0, p.st.word, p.st.wait_limit_ns, SITE_DRAIN);
        } else if (PART == kPrefix && warp == 9) {  // where the merge finds the items that begin here
            while (next_segment<PART>(p, walk))
                if (w.v0 == 0 && lane == 0) {
                    const long long x = w.s.x - (w.v1 - w.v0);
                    p.items[static_cast<long long>(group_tile(p, w.b) + w.pair) * p.Hk + w.hk] =
                        make_int2(static_cast<int>(blockIdx.x), static_cast<int>(div_mostly32(x + w.u.n - 1, w.s.share)));
                }
        } else if (warp == 9) {  // what the joining kernel finds at the border before this share
            CacheBorder bd;
            bd.c_first = -1;
            bd.b = bd.item = bd.q_len = bd.c_last = 0;
            const long long x = w.s.x;
            if (next_segment<PART>(p, walk) && w.v0 > 0) {
                bd.b = w.b;
                bd.item = w.hk * ((w.u.rows + kPairRows - 1) / kPairRows) + w.pair;
                bd.q_len = w.u.q_len;
                bd.c_first = static_cast<int>(div_mostly32(x - w.v0, w.s.share)) + 1;
                bd.c_last = static_cast<int>(div_mostly32(x - w.v0 + w.u.n - 1, w.s.share));
            }
            if (lane == 0) p.border[blockIdx.x] = bd;
        }
    } else {
        regs_inc<kSoftmaxRegs>();
        // ================= softmax: one thread per row of query tile g =================
        const int g = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + (g ? T::COL_S1 : T::COL_S0) + lane_off;
        const uint32_t tO = tmem + (g ? T::COL_O1 : T::COL_O0) + lane_off;
        const uint32_t b_sf = b_s_full + 8u * g, b_pf = b_p_full + 8u * g, b_of = b_o_full + 8u * g;
        int s_seen = 0, o_seen = 0, tile_no = 0, merges = 0;
        bool ok = true;
        while (ok && next_segment<PART>(p, walk)) {
            const int n = g ? w.a1 : w.a0;
            const bool dual = w.u.dual;
            const int r = w.pair * kPairRows + (dual ? 0 : g * kTile) + row;  // row of the key/value head
            bool row_ok = r < w.u.rows;
            int t = row_ok ? r / G : 0, member = 0;  // member: sequence of a group's row
            const int h = w.hk * G + (row_ok ? r - t * G : 0);
            // rows behind the last query (zeros, never written) take its place: no mask of their own
            const int pos = w.u.first_pos + (PART == kPrefix ? 0 : row_ok ? t : w.u.q_len - 1);
            if constexpr (PART == kPrefix) {
                if (row_ok) {
                    const int m = t / p.T;
                    member = group_begin(p, w.b) + m;
                    t -= m * p.T;
                }
                row_ok = row_ok && t < query_count(p, member);
            }
            auto seq = [&] { return PART == kPrefix ? member : w.b; };
            const int key_min = p.left < 0 ? 0 : pos - p.left;
            float rq = 0.f;
            if (n > 0) {
                // Q rows to f16, times a power of two each.  The tile's place is free: the
                // previous segment's last S_g, read here, came after every product on it.
                // A row takes D / 8 lanes, the same for the copy and for the conversion in place: all of
                // the copies are out at once (Q comes after the first keys' loads: 1600 to 3000 cycles),
                // and the code is short (unrolled, what runs once a segment took longer).
                constexpr int LPR = D / 8, RPI = 32 / LPR;
                const unsigned there = __ballot_sync(0xffffffffu, row_ok);
                const unsigned long long src = reinterpret_cast<unsigned long long>(
                    static_cast<const uint16_t*>(p.q) + seq() * p.qs.b + h * p.qs.h + t * p.qs.n);
                const int sub = lane / LPR, c = lane % LPR;
                uint8_t* const q_at = smem + g * T::TILE_BYTES + (c >> 3) * T::BLK_BYTES + wq * 32 * 128;
                auto place = [&](int rr) { return q_at + rr * 128 + (((c & 7) ^ (rr & 7)) << 4); };
#pragma unroll 4
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int rr = i * RPI + sub;
                    const bool have = there >> rr & 1u;
                    const unsigned long long at = __shfl_sync(0xffffffffu, src, rr);
                    cp_async16(smem_u32(place(rr)), have ? reinterpret_cast<const uint4*>(at) + c : p.q, have);
                }
                cp_async_commit();
                cp_async_wait<0>();
                float f_row = 0.f;
#pragma unroll 1
                for (int i0 = 0; i0 < 32 / RPI; i0 += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const uint4*>(place((i0 + k) * RPI + sub));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // magnitudes of bf16 order as their bit patterns (a row with NaN is NaN whatever its power)
                        uint32_t top = 0u;
                        for (uint32_t u : {x[k].x, x[k].y, x[k].z, x[k].w}) top = __vmaxu2(top, u & 0x7FFF7FFFu);
                        top = max(top >> 16, top & 0xFFFFu);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float amax = __uint_as_float(top << 16);
                        const float f = f16_row_scale(amax);
                        auto cv = [&](uint32_t u) { return pack_f16x2(bf16lo(u) * f, bf16hi(u) * f); };
                        x[k] = make_uint4(cv(x[k].x), cv(x[k].y), cv(x[k].z), cv(x[k].w));
                        const float of_row = __shfl_sync(0xffffffffu, f, lane % RPI * LPR);
                        if (lane / RPI == i0 + k) f_row = of_row;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(place((i0 + k) * RPI + sub)) = x[k];
                }
                rq = p.cs * __uint_as_float((254u << 23) - __float_as_uint(f_row));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_q + 8u * g);
            }

            float m_used = -INFINITY;  // running maximum of score + log2 sv (log2 units), possibly stale
            float l_sum = 0.f;         // sum of 2^(score - m_used + kWeightShift) (value scales taken back out)
            float u = -INFINITY;       // apart (see kScaleReach): l_sum is of 2^(score - u)
            // Scales of key tile j.  Its entry is written again for the tile SCALES further
            // on, once that tile's K slot is free: the one of V(j + 1) (five slots, four
            // entries) or K(j + 4) (eight and eight), which products read that were issued
            // after this warp had arrived for tile j.
            auto wait_scales = [&](int j) {
                const int tn = tile_no + (dual ? 2 * j + g : j);
                return wait_in_line(b_scale + 8u * (tn % T::SCALES), (tn / T::SCALES) & 1, abort_flag, p.st, SITE_SCALE);
            };
            // apart_tag: a second copy of the code, so that the first has nothing more to hold
            auto step = [&](auto apart_tag, int j) -> bool {
                constexpr bool apart = decltype(apart_tag)::value;
                const int ti = dual ? 2 * j + g : j, tn = tile_no + ti;  // tile of the segment, and of all
                const int kv0 = w.u.tile(w.v0 + ti) * kTile;
                const int c_lo = key_min - kv0, c_hi = pos - kv0, c_sink = p.sinks - kv0;
                const bool masked = PART == kWhole && __any_sync(0xffffffffu, (c_lo > 0 && c_sink < c_lo) || c_hi < kTile - 1);
                const float4* sc = scales + (tn % T::SCALES) * 8;
                if (!wait_in_line(b_sf, (s_seen + j) & 1, abort_flag, p.st, SITE_S_FULL)) return false;
                tc_fence_after();
                // The 128 scores 32 at a time.  Only while a row has no maximum is there a pass for
                // the tile's; after it the weights are formed against m_used as it is, and 32
                // columns whose sum passes kWeightMax are done again with their own maximum, the
                // tile's weights before them scaled down (2 x 2048 queries over 16384 keys: 600 us,
                // with a pass for the maximum of each tile 700).  The loops stay rolled and the
                // mask is formed from bits: the roles' code does not fit the instruction caches
                // otherwise (with both passes unrolled 1033 us).
                auto take = [&](int c, uint32_t (&x)[32]) {  // columns 32 c .. 32 c + 31, hidden ones -inf
                    tmem_ld_wait(x);
                    if (masked) {  // bit i of `seen`: column 32 c + i
                        auto below = [&](int n) { n -= 32 * c; return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
                        const uint32_t seen = below(c_hi + 1) & (~below(c_lo) | below(c_sink));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen >> i & 1u)) x[i] = f2u(-INFINITY);
                    }
                };
                auto largest = [&](int c, const uint32_t (&x)[32]) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 e = sc[2 * c + h];
                        float a = fmax3(u2f(x[16 * h]), u2f(x[16 * h + 1]), u2f(x[16 * h + 2]));
                        float b = fmax3(u2f(x[16 * h + 3]), u2f(x[16 * h + 4]), u2f(x[16 * h + 5]));
#pragma unroll
                        for (int i = 6; i < 14; i += 4) {
                            a = fmax3(a, u2f(x[16 * h + i]), u2f(x[16 * h + i + 1]));
                            b = fmax3(b, u2f(x[16 * h + i + 2]), u2f(x[16 * h + i + 3]));
                        }
                        a = fmaxf(fmax3(a, u2f(x[16 * h + 14]), u2f(x[16 * h + 15])), b);
                        mx = fmaxf(mx, fmaf(a, score_factor(rq, e.x), e.y));
                    }
                    return mx;
                };
                float alpha = 1.f, tile_l = 0.f;
                bool rescale_o = false;
                // By whole powers of two, so that weights in f16 scaled down are not rounded twice.
                auto raise = [&](float mx) -> float {  // factor of what was summed against the old maximum
                    if (!(mx > m_used)) return 1.f;
                    if (m_used != -INFINITY) mx = m_used + ceilf(mx - m_used);
                    const float a = ex2_approx(m_used - mx);  // 0 while m_used is -inf
                    if (!apart) l_sum *= a;
                    tile_l *= a;
                    alpha *= a;
                    m_used = mx;
                    rescale_o = j > 0;
                    return a;
                };
                if constexpr (apart) {
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 8) {
                        uint32_t x[8];
                        tmem_ld8(tS + c, x);
                        const float f = score_factor(rq, sc[c >> 4].x);
                        float mx = u, sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const bool seen = PART == kPrefix || (c + i <= c_hi && (c + i >= c_lo || c + i < c_sink));
                            x[i] = f2u(seen ? u2f(x[i]) * f : -INFINITY);
                            mx = fmaxf(mx, u2f(x[i]));
                        }
                        const float sub = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum += ex2_approx(u2f(x[i]) - sub);
                        l_sum = fmaf(l_sum, u == mx ? 1.f : ex2_approx(u - mx), sum);
                        u = mx;
                    }
                }
                if (__any_sync(0xffffffffu, m_used == -INFINITY)) {
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        tmem_ld32(tS + 32 * c, x);
                        take(c, x);
                        mx = fmaxf(mx, largest(c, x));
                    }
                    raise(mx);
                }
                auto work = [&](int c, const uint32_t (&x)[32]) {
                    uint32_t pk[16];
                    float sum, l;
#pragma unroll 1
                    for (int pass = 0;; ++pass) {
                        const float sub = kWeightShift - (m_used == -INFINITY ? 0.f : m_used);
                        sum = l = 0.f;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 e = sc[2 * c + h];
                            const float f = score_factor(rq, e.x), add = e.y + sub;
                            float a0 = 0.f, a1 = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float x0, x1;
                                ffma2(x0, x1, u2f(x[16 * h + i]), u2f(x[16 * h + i + 1]), f, f, add, add);
                                x0 = ex2_approx(x0);
                                x1 = ex2_approx(x1);
                                // f16 (half a step, 2^-11 relative): finer than the bf16 output
                                pk[8 * h + i / 2] = pack_f16x2(x0, x1);
                                fadd2(a0, a1, a0, a1, x0, x1);
                            }
                            sum += a0 + a1;
                            l = fmaf(a0 + a1, e.z, l);
                        }
                        if (pass > 0 || !__any_sync(0xffffffffu, !(sum <= kWeightMax))) break;
                        const float a = raise(largest(c, x));
                        tmem_st_wait();  // the weights stored so far are read back
#pragma unroll 1
                        for (int b = 0; b < c; ++b) {
                            uint32_t w[32], o[16];
                            tmem_ld32(tS + 16 * b, w);
                            tmem_ld_wait(w);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float w0, w1;
                                unpack_f16x2(w[i], w0, w1);
                                o[i] = pack_f16x2(w0 * a, w1 * a);
                            }
                            tmem_st16(tS + 16 * b, o);
                        }
                    }
                    tile_l += l;
                    tmem_st16(tS + 16 * c, pk);  // over columns read before
                };
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32(tS + 32 * c, x);
                    take(c, x);
                    work(c, x);
                }
                if (!apart) l_sum += tile_l;
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
                return true;
            };
            int j = 0;
            for (; j < n; ++j) {
                if (!(ok = wait_scales(j))) break;
                const int tn = tile_no + (dual ? 2 * j + g : j);
                if (__any_sync(0xffffffffu, scales[(tn % T::SCALES) * 8 + (lane & 7)].w != 0.f)) break;
                if (!(ok = step(std::false_type{}, j))) break;
            }
            const bool apart = ok && j < n;
            if (apart) {
                if (l_sum != 0.f) u = m_used - kWeightShift;
                for (; j < n && ok; ++j) ok = wait_scales(j) && step(std::true_type{}, j);
            }
            s_seen += n;
            tile_no += w.v1 - w.v0;
            if (ok && n > 0) {
                ok = wait_in_line(b_of, o_seen & 1, abort_flag, p.st, SITE_O_FULL);
                ++o_seen;
                tc_fence_after();
            }
            if (!ok) break;
            if (apart) {
                float half;
                plain_units(m_used, l_sum, u, l_sum, half);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * half * half);
                    tmem_st32(tO + 32 * c, o);
                    tmem_st_wait();
                }
            }
            if (dual && w.a1 > 0) {
                if (g == 1) {
                    // This group's maximum and sum beside its O in tensor memory, whose lanes the
                    // other group's warp of the same number can read; the columns are its own P's,
                    // which the products have read.
                    uint32_t x[16] = {f2u(l_sum != 0.f ? m_used : -INFINITY), f2u(l_sum)};
                    tmem_st16(tS, x);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_merge);
                    // the next segment's Q lets products write there again
                    ok = wait_in_line(b_merged, merges & 1, abort_flag, p.st, SITE_MERGE);
                    ++merges;
                    continue;
                }
                ok = wait_in_line(b_merge, merges & 1, abort_flag, p.st, SITE_MERGE);
                ++merges;
                if (!ok) break;
                tc_fence_after();
            } else if (dual && g == 1) {
                continue;  // the only tile was group 0's
            }
            if (n > 0 && PART == kWhole) {
                // NaN values that the row sees in tiles that not every row sees (they stood as 0 in
                // the products); by now both groups' products are done, so every value of the
                // segment has been looked at.  Such tiles are seven a walk at most, however long
                // it is: 600 queries of 40 heads over 131072 keys, all values NaN, 1.90 ms for 1.57.
                // (lane 0's reading counts: the converters may be at the next segment, and all lanes
                // have to take the same side)
                const int lo = __shfl_sync(0xffffffffu, *static_cast<volatile int*>(nan_tiles), 0);
                const int hi = __shfl_sync(0xffffffffu, *static_cast<volatile int*>(nan_tiles + 1), 0);
                const TileSpan span = segment_span(lo, hi, tile_no - (w.v1 - w.v0), w.v0, w.v1);
                if (span.first < span.end) {
                    uint32_t nan[D / 32] = {};  // bit i of word c: column 32 c + i
#pragma unroll 1
                    for (int t = span.first; t < span.end; ++t) {
                        if (w.u.all_see(t, p.left, p.sinks)) continue;
                        const int tile0 = w.u.tile(t) * kTile;
#pragma unroll 1
                        for (int tok = tile0; tok < tile0 + kTile; ++tok) {
                            if (!row_ok || tok > pos || (tok < key_min && tok >= p.sinks)) continue;
                            const int pid = __ldg(p.c.table + w.b * p.c.table_stride + (tok >> p.c.page_shift));
                            if (static_cast<unsigned>(pid) >= static_cast<unsigned>(p.c.num_pages)) continue;
                            const uint4* codes = reinterpret_cast<const uint4*>(
                                p.c.v_pages + pid * p.c.vs.b + w.hk * p.c.vs.h + (tok & (p.c.page_size - 1)) * p.c.vs.n);
                            uint4 x[D / 16];
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) x[c] = __ldg(codes + c);
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t bits = 0u;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t u = e == 0 ? x[c].x : e == 1 ? x[c].y : e == 2 ? x[c].z : x[c].w;
                                    const uint32_t y = ((u & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                    bits |= (y >> 7 & 1u | y >> 14 & 2u | y >> 21 & 4u | y >> 28 & 8u) << (4 * e);
                                }
                                nan[c / 2] |= bits << (16 * (c & 1));
                            }
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        if (!__any_sync(0xffffffffu, nan[c] != 0u)) continue;
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (nan[c] >> i & 1u) o[i] = 0x7FC00000u;
                        tmem_st32(tO + 32 * c, o);
                        tmem_st_wait();
                    }
                }
            }
            const bool finished = w.v0 == 0 && w.v1 == w.u.n, merge = dual && w.a1 > 0;
            // group 0's O and sum times f0, and, merging, group 1's times f1
            float f0 = 1.f, f1 = 0.f;
            if (merge) {
                uint32_t x[32];
                tmem_ld32(tmem + T::COL_S1 + lane_off, x);
                tmem_ld_wait(x);
                const float m1 = u2f(x[0]), l1 = u2f(x[1]), m0 = l_sum != 0.f ? m_used : -INFINITY;
                m_used = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - m_used);
                f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m_used);
                l_sum = l_sum * f0 + l1 * f1;
            }
            // without a live key tile: O = 0 and LSE = +inf, or a segment that takes no part
            const float inv = n > 0 && l_sum != 0.f ? 1.f / l_sum : 0.f;  // NaN stays NaN
            const long long part_row =
                (2ll * blockIdx.x + (w.v0 == 0 ? 1 : 0)) * kPairRows + (dual ? 0 : g * kTile) + row;
            uint16_t* orow = static_cast<uint16_t*>(p.o) + w.b * p.os.b + h * p.os.h + t * p.os.n;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                if (merge) {
                    uint32_t o1[32];
                    tmem_ld32(tmem + T::COL_O1 + lane_off + 32 * c, o1);
                    tmem_ld_wait(o1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * f0 + u2f(o1[i]) * f1);
                }
                if (!row_ok) continue;
                if (finished && PART == kWhole) {
                    uint32_t pkd[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) pkd[i] = pack_bf16x2(u2f(o[2 * i]) * inv, u2f(o[2 * i + 1]) * inv);
                    st_global_row64<false>(reinterpret_cast<uint8_t*>(orow + 32 * c), pkd);
                } else {
                    float* dst = (PART == kPrefix && finished ? p.fin_o + fin_row(p, seq(), t, h) * D : p.part + part_row * D) + 32 * c;
                    if constexpr (PART == kWhole) {
#pragma unroll
                        for (int v = 0; v < 8; ++v) st_global_v4(dst + 4 * v, o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v) st_global_v8(dst + 8 * v, o + 8 * v);
                    }
                }
            }
            if (row_ok) {
                if (PART == kPrefix && finished)
                    p.fin_stat[fin_row(p, seq(), t, h)] = make_float2(l_sum != 0.f ? m_used : -INFINITY, l_sum);
                else if (finished)
                    p.lse[(static_cast<long long>(w.b) * p.H + h) * p.T + t] =
                        l_sum != 0.f ? (m_used - kWeightShift + log2f(l_sum)) * kLn2 : INFINITY;
                else
                    p.stat[part_row] = make_float2(l_sum != 0.f ? m_used : -INFINITY, l_sum);
            }
            if (merge) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_merged);
            }
            tc_fence_before();  // O_g may be overwritten once this warp arrives on q_full and p_full
        }
    }

    // ---- teardown: all tensor-memory traffic of this CTA is complete ----
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, CachePart PART>
cudaError_t launch_prompt_impl(CacheFwdParams& p, cudaStream_t stream) {
    using T = PromptTraits<D>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t attr = once_per_device(ready, [] {
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, cache_prompt_kernel<D, PART>);
        // the register split draws on what the launch has: with fewer it would wait for ever
        if (e == cudaSuccess && a.numRegs != kLaunchRegs) e = cudaErrorInvalidKernelImage;
        return e == cudaSuccess ? cudaFuncSetAttribute(cache_prompt_kernel<D, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       T::SMEM_BYTES)
                                : e;
    });
    if (attr != cudaSuccess) return attr;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    p.rows = kPairRows;
    p.grid = sms < kPromptGridMax ? sms : kPromptGridMax;
    const long long rows = static_cast<long long>(PART == kPrefix ? p.B : 1) * p.T * (p.H / p.Hk);  // at most
    const int pairs = static_cast<int>((rows + kPairRows - 1) / kPairRows);
    if ((e = dbg_set_word(p.st.word, stream)) != cudaSuccess) return e;
    e = launch_dependent(cache_prompt_kernel<D, PART>, dim3(static_cast<unsigned>(p.grid)), kPromptThreads, T::SMEM_BYTES,
                         stream, p, pairs);
    return e != cudaSuccess || PART == kPrefix ? e : launch_cache_join(p, 8, stream);
}

}  // namespace

cudaError_t launch_cache_prompt(CacheFwdParams* p, CachePart part, cudaStream_t stream) {
    if (p->D == 64) return part == kPrefix ? launch_prompt_impl<64, kPrefix>(*p, stream) : launch_prompt_impl<64, kWhole>(*p, stream);
    if (p->D == 128) return part == kPrefix ? launch_prompt_impl<128, kPrefix>(*p, stream) : launch_prompt_impl<128, kWhole>(*p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
