// A serving step's write into the paged 8-bit cache: new tokens' Q and K heads are normed and
// rotated at the tokens' positions in the cache, K and V are written as E4M3 codes and Q is
// given back, in one launch.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_append.cuh"
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rope_ops.cuh"

namespace attn {
namespace {

// Tokens of a page go by rounds of kAppendThreads / (D / 16), one a thread and round.  The first
// kHeld rounds' rotated elements stay in registers and their angles in shared memory (a place for each
// thread, 8 KB a round), for all of a block's up to kPageHeads heads.  (Room for the angles of eight
// rounds leaves an SM three blocks: pages of 128 tokens at d = 128, 133 us for 115.)
constexpr int kHeld = 4, kPageHeads = 8;
struct KeyShared {
    float4 weight[4][8];  // the head's, in the order of the pieces that its threads hold
    float4 at[kHeld][4][kAppendThreads];
    __device__ __forceinline__ void put_weight(const RopeView& r, int t, int row, int lo, int hi) {
        if (row != 0) return;
        float w[16];
        load_weight(r, r.k_weight, lo, hi, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) weight[i][t] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void put(int k, const RopeAngles& a) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at[k][i][threadIdx.x] = make_float4(a.c[4 * i], a.c[4 * i + 1], a.c[4 * i + 2], a.c[4 * i + 3]);
            at[k][2 + i][threadIdx.x] = make_float4(a.s[4 * i], a.s[4 * i + 1], a.s[4 * i + 2], a.s[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void get(int k, RopeAngles& a) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 c = at[k][i][threadIdx.x], s = at[k][2 + i][threadIdx.x];
            a.c[4 * i] = c.x, a.c[4 * i + 1] = c.y, a.c[4 * i + 2] = c.z, a.c[4 * i + 3] = c.w;
            a.s[4 * i] = s.x, a.s[4 * i + 1] = s.y, a.s[4 * i + 2] = s.z, a.s[4 * i + 3] = s.w;
        }
    }
};
// K of the page of AppendPage a, heads [hk, hk_end): rotated in fp32 and rounded once, to E4M3.  A
// thread holds 16 elements of its tokens as fp32 between the two looks at them; tokens beyond the ones
// held (pages of more than 64 tokens at d = 128, 128 at d = 64) are read and rotated again.
template <int D, bool INTER>
__device__ __forceinline__ void append_rotated(const CacheAppendRopeParams& p, const AppendPage& a, int b, int hk, int hk_end,
                                               KeyShared& sm) {
    constexpr int TPR = D / 16, RPP = kAppendThreads / TPR;
    const CacheAppendParams& c = p.c;
    const int t = threadIdx.x % TPR, rr = threadIdx.x / TPR, n = a.hi - a.lo, nrot = p.r.rot / 16;
    int lo, hi;
    rope_pieces<INTER>(t, nrot, lo, hi);
    const bool norm = p.r.k_weight != nullptr;
    for (int h = hk;;) {
        uint8_t* codes = c.c.k_pages + a.pid * c.c.ks.b + h * c.c.ks.h;
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.k) + b * c.ks.b + h * c.ks.h);
        float* scale = c.c.k_scale + static_cast<long long>(a.pid) * c.Hk + h;
        const float was = *scale;

        auto load = [&](int i, uint4& l, uint4& u) {  // the page's i-th new token
            l = u = make_uint4(0u, 0u, 0u, 0u);
            if (i < n) {
                const uint4* at = x + (a.lo + i - a.first) * (c.ks.n / 8);
                l = __ldcs(at + lo);
                u = __ldcs(at + hi);
            }
        };
        // norm and rotation of a token's elements, its angles as `angles` fills them in
        auto turn = [&](float (&v)[16], bool turns, auto angles) {
            if (norm) {
                const float r = head_rnorm<D>(v, p.r.eps);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 w = sm.weight[i / 4][t];
                    fmul2(v[i], v[i + 1], v[i], v[i + 1], r, r);
                    fmul2(v[i + 2], v[i + 3], v[i + 2], v[i + 3], r, r);
                    fmul2(v[i], v[i + 1], v[i], v[i + 1], w.x, w.y);
                    fmul2(v[i + 2], v[i + 3], v[i + 2], v[i + 3], w.z, w.w);
                }
            }
            if (turns) {
                RopeAngles ang;
                angles(ang);
                rotate16<INTER>(ang, v);
            }
        };
        float held[kHeld][16];
        {
            uint4 l[kHeld], u[kHeld];
#pragma unroll
            for (int k = 0; k < kHeld; ++k) load(rr + k * RPP, l[k], u[k]);
            if (h == hk) {  // while those are on their way
                if (norm) sm.put_weight(p.r, t, rr, lo, hi);
#pragma unroll 1
                for (int k = 0; k < kHeld && k * RPP < n; ++k) {
                    RopeAngles ang;
                    if (rr + k * RPP < n && t < nrot) {
                        ang.at(p.r, t, a.lo + rr + k * RPP, 1.f);
                        sm.put(k, ang);
                    }
                }
                if (norm) __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {  // (zeros stay zeros)
                unpack16(l[k], u[k], held[k]);
                if (k * RPP < n) turn(held[k], rr + k * RPP < n && t < nrot, [&](RopeAngles& ang) { sm.get(k, ang); });
            }
        }
        // Rounds of further tokens are the same for every thread: a norm's sum takes several.
        auto further = [&](auto each) {
            for (int i0 = kHeld * RPP; i0 < n; i0 += RPP) {
                uint4 l, u;
                float v[16];
                load(i0 + rr, l, u);
                unpack16(l, u, v);
                turn(v, i0 + rr < n && t < nrot, [&](RopeAngles& ang) { ang.at(p.r, t, a.lo + i0 + rr, 1.f); });
                each(i0 + rr, v);
            }
        };
        __shared__ uint32_t warp_max[kAppendThreads / 32];
        auto largest = [&](auto magnitude) -> float {  // of the block's new values (as bits, which order alike)
            uint32_t m = 0u;
            auto look = [&](const float (&v)[16]) {
#pragma unroll
                for (int e = 0; e < 16; ++e) m = max(m, magnitude(__float_as_uint(v[e]) & 0x7FFFFFFFu));
            };
#pragma unroll
            for (int k = 0; k < kHeld; ++k) look(held[k]);
            further([&](int, const float (&v)[16]) { look(v); });
            m = __reduce_max_sync(0xffffffffu, m);
            if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
            __syncthreads();  // and every thread has read the old scale
            return __uint_as_float(max(max(warp_max[0], warp_max[1]), max(warp_max[2], warp_max[3])));
        };
        float amax = largest([](uint32_t u) { return u; });
        if (!isfinite(amax)) {  // infinities or NaN: the largest finite magnitude counts
            __syncthreads();
            amax = largest([](uint32_t u) { return u < 0x7F800000u ? u : 0u; });
        }
        const bool keep = append_keeps(a.old, was, amax);
        const float s = keep ? was : append_scale(amax);
        if (a.old > 0 && !keep) {
            append_grow(codes + 8 * lo, c.c.ks.n, rr, RPP, a.old, was, s);
            append_grow(codes + 8 * hi, c.c.ks.n, rr, RPP, a.old, was, s);
        }
        const AppendQuotient quotient(s);
        auto put_all = [&](auto code) {
            auto put = [&](int i, const float (&v)[16]) {
                if (i >= n) return;
                uint8_t* at = codes + (a.old + i) * c.c.ks.n;
                uint32_t u[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    u[k] = pack_e4m3x4(code(v[4 * k]), code(v[4 * k + 1]), code(v[4 * k + 2]), code(v[4 * k + 3]));
                *reinterpret_cast<uint2*>(at + 8 * lo) = make_uint2(u[0], u[1]);
                *reinterpret_cast<uint2*>(at + 8 * hi) = make_uint2(u[2], u[3]);
            };
#pragma unroll
            for (int k = 0; k < kHeld; ++k) put(rr + k * RPP, held[k]);
            further(put);
        };
        if (quotient.exact()) put_all([&](float v) { return v * quotient.inv; });
        else put_all(quotient);
        if (threadIdx.x == 0 && !keep) *scale = s;
        if (++h == hk_end) return;
        __syncthreads();  // warp_max is written again
    }
}

// Q of p.token_slots tokens from t0 on and a chunk of heads, as in the kernel that rotates whole
// sequences.  Tokens that are not new, or lie before the sequence's start, are left alone.
template <int D, bool INTER>
__device__ __forceinline__ void rotate_queries(const CacheAppendRopeParams& p, int b, int t0, int chunk, RopeRing& ring) {
    constexpr int TPR = D / 16, SLOTS = kAppendThreads / TPR;
    const CacheAppendParams& c = p.c;
    const int slot = threadIdx.x / TPR, TT = p.token_slots, HT = SLOTS / TT;
    const int m = c.new_lens ? min(max(c.new_lens[b], 0), c.T) : c.T;
    if (t0 >= m) return;
    const int n = t0 + slot % TT, pos = max(c.c.seq_lens[b], 0) - m + n;
    const int first = chunk * HT * p.hp, heads = min(p.H - first, HT * p.hp);
    rotate_heads<D, INTER>(p.r, p.r.q_weight, 1.f, n < m && pos >= 0, pos,
                           static_cast<const uint4*>(p.q) + (b * p.qs.b + n * p.qs.n) / 8, p.qs.h / 8,
                           static_cast<uint4*>(p.q_out) + (b * p.qos.b + n * p.qos.n) / 8, p.qos.h / 8, first + slot / TT, HT,
                           first + heads, (heads + HT - 1) / HT, ring);
}

// Blocks [0, k_blocks): a touched page of a sequence and p.hk heads of K; [k_blocks, page_blocks): one
// and p.hk heads of V; the others: tokens and heads of Q.  Bound by the memory: 4 prompts of up to 8192
// tokens, 32/8 heads, d = 128, norms: 90 us, 5.5 TB/s, in pages of 16 126, of 128 115 (angles worked out for each head of K and Q's
// loads in registers: 109; Q in a launch of its own with six blocks an SM: 93; a head of K and of V a
// block, pages of 16: 154); one token for 32
// sequences 4.9 us in a row, the chain length, table, page, scale.
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_rope_kernel(const CacheAppendRopeParams p) {
    __shared__ union Shared {
        KeyShared keys;
        RopeRing ring;
        __device__ Shared() {}
    } sm;
    static_assert(kAppendThreads == kRopeThreads, "threads of a block");
    pdl_wait();
    const unsigned x = blockIdx.x;
    if (x < p.page_blocks) {
        const bool is_v = x >= p.k_blocks;
        const unsigned y = is_v ? x - p.k_blocks : x, of_page = y / p.pages, slot = y - of_page * p.pages;
        const unsigned b = of_page / p.parts, part = of_page - b * p.parts;
        if (slot == 0 && part == 0 && !is_v && threadIdx.x == 0) check_len(p.c.c, p.c.st, static_cast<int>(b));
        AppendPage a;
        if (!append_page(p.c, static_cast<int>(b), static_cast<int>(slot), a)) return;
        const int hk = static_cast<int>(part) * p.hk, hk_end = min(hk + p.hk, p.c.Hk);
        if (!is_v) {
            append_rotated<D, INTER>(p, a, static_cast<int>(b), hk, hk_end, sm.keys);
            return;
        }
        for (int h = hk;;) {
            append_plain<D>(p.c, a, static_cast<int>(b), h, true);
            if (++h == hk_end) return;
            __syncthreads();  // the head's largest magnitudes have been read
        }
    }
    const unsigned y = x - p.page_blocks, rest = y / p.token_tiles, tile = y - rest * p.token_tiles;
    const unsigned b = rest / p.chunks, chunk = rest - b * p.chunks;
    rotate_queries<D, INTER>(p, static_cast<int>(b), static_cast<int>(tile) * p.token_slots, static_cast<int>(chunk), sm.ring);
}

template <int D>
cudaError_t launch_append_rope_d(CacheAppendRopeParams p, cudaStream_t stream) {
    constexpr int SLOTS = kAppendThreads / (D / 16);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const CacheAppendParams& c = p.c;
    p.pages = static_cast<unsigned>((c.T + c.c.page_size - 2) / c.c.page_size + 1);  // pages that T tokens can touch
    p.token_slots = rope_token_slots(c.T, SLOTS);
    p.token_tiles = static_cast<unsigned>((c.T + p.token_slots - 1) / p.token_slots);
    const int HT = SLOTS / p.token_slots;
    for (p.hp = 8;; p.hp /= 2) {  // as many heads a thread as leave every SM some blocks
        p.chunks = static_cast<unsigned>((p.H + HT * p.hp - 1) / (HT * p.hp));
        if (p.hp == 1 || static_cast<long long>(p.token_tiles) * p.chunks * c.B >= 3ll * sms) break;
    }
    for (p.hk = c.Hk < kPageHeads ? c.Hk : kPageHeads;; p.hk = (p.hk + 1) / 2) {  // and as many heads of K and V a block
        p.parts = static_cast<unsigned>((c.Hk + p.hk - 1) / p.hk);
        if (p.hk == 1 || static_cast<long long>(p.pages) * p.parts * c.B >= 4ll * sms) break;
    }
    const long long k_blocks = static_cast<long long>(p.pages) * p.parts * c.B;
    const long long blocks = 2 * k_blocks + static_cast<long long>(p.token_tiles) * p.chunks * c.B;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    p.k_blocks = static_cast<unsigned>(k_blocks);
    p.page_blocks = 2 * p.k_blocks;
    const dim3 grid(static_cast<unsigned>(blocks));
    return p.r.interleaved ? launch_dependent(cache_append_rope_kernel<D, true>, grid, kAppendThreads, 0, stream, p)
                           : launch_dependent(cache_append_rope_kernel<D, false>, grid, kAppendThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_cache_append_rope(const CacheAppendRopeParams& p, cudaStream_t stream) {
    if (p.c.D == 64) return launch_append_rope_d<64>(p, stream);
    if (p.c.D == 128) return launch_append_rope_d<128>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
