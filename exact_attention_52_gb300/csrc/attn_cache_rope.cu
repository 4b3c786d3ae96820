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

// K of the page of AppendPage a, head hk: rotated in fp32 and rounded once, to E4M3.  A thread
// holds 16 elements of its tokens as fp32 between the two looks at them; tokens beyond the ones
// held (pages of more than 64 tokens at d = 128, 128 at d = 64) are read and rotated again.
template <int D, bool INTER>
__device__ __forceinline__ void append_rotated(const CacheAppendRopeParams& p, const AppendPage& a, int b, int hk) {
    constexpr int TPR = D / 16, RPP = kAppendThreads / TPR, kHeld = 4;
    const CacheAppendParams& c = p.c;
    const int t = threadIdx.x % TPR, rr = threadIdx.x / TPR, n = a.hi - a.lo, nrot = p.r.rot / 16;
    int lo, hi;
    rope_pieces<INTER>(t, nrot, lo, hi);
    uint8_t* codes = c.c.k_pages + a.pid * c.c.ks.b + hk * c.c.ks.h;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.k) + b * c.ks.b + hk * c.ks.h);
    float* scale = c.c.k_scale + static_cast<long long>(a.pid) * c.Hk + hk;
    const float was = *scale;
    const bool norm = p.r.k_weight != nullptr;
    float w[16] = {};
    if (norm) load_weight(p.r, p.r.k_weight, lo, hi, w);

    auto load = [&](int i, uint4& l, uint4& h) {  // the page's i-th new token
        l = h = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) {
            const uint4* at = x + (a.lo + i - a.first) * (c.ks.n / 8);
            l = __ldcs(at + lo);
            h = __ldcs(at + hi);
        }
    };
    auto turn = [&](int i, const uint4& l, const uint4& h, float (&v)[16]) {  // (zeros stay zeros)
        unpack16(l, h, v);
        RopeAngles ang;
        if (i < n && t < nrot) ang.at(p.r, t, a.lo + i, 1.f);
        norm_rotate<D, INTER>(v, norm, w, p.r.eps, i < n && t < nrot, ang);
    };
    float held[kHeld][16];
    {
        uint4 l[kHeld], h[kHeld];
#pragma unroll
        for (int k = 0; k < kHeld; ++k) load(rr + k * RPP, l[k], h[k]);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) turn(rr + k * RPP, l[k], h[k], held[k]);
    }
    // Rounds of further tokens are the same for every thread: a norm's sum takes several.
    auto further = [&](auto each) {
        for (int i0 = kHeld * RPP; i0 < n; i0 += RPP) {
            uint4 l, h;
            float v[16];
            load(i0 + rr, l, h);
            turn(i0 + rr, l, h, v);
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
}

// Q of p.token_slots tokens from t0 on and a chunk of heads, as in the kernel that rotates whole
// sequences.  Tokens that are not new, or lie before the sequence's start, are left alone.
template <int D, bool INTER>
__device__ __forceinline__ void rotate_queries(const CacheAppendRopeParams& p, int b, int t0, int chunk) {
    constexpr int TPR = D / 16, SLOTS = kAppendThreads / TPR, U = 4;
    const CacheAppendParams& c = p.c;
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR, TT = p.token_slots, HT = SLOTS / TT;
    const int m = c.new_lens ? min(max(c.new_lens[b], 0), c.T) : c.T;
    if (t0 >= m) return;
    const int n = t0 + slot % TT, pos = max(c.c.seq_lens[b], 0) - m + n, nrot = p.r.rot / 16;
    const bool there = n < m && pos >= 0;
    int lo, hi;
    rope_pieces<INTER>(t, nrot, lo, hi);
    const bool norm = p.r.q_weight != nullptr;
    float w[16] = {};
    if (norm) load_weight(p.r, p.r.q_weight, lo, hi, w);
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + b * p.qs.b + n * p.qs.n);
    uint4* y = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + b * p.qos.b + n * p.qos.n);
    const long long xh = p.qs.h / 8, yh = p.qos.h / 8;
    const int h0 = chunk * HT * p.hp + slot / TT, h1 = min(p.H, (chunk + 1) * HT * p.hp);
    RopeAngles a;
    if (there && t < nrot) a.at(p.r, t, pos, 1.f);
    for (int i = 0; i < p.hp; i += U) {
        uint4 vl[U], vh[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + (i + u) * HT;
            vl[u] = vh[u] = make_uint4(0u, 0u, 0u, 0u);
            if (there && h < h1) {
                vl[u] = x[h * xh + lo];
                vh[u] = x[h * xh + hi];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + (i + u) * HT;
            float v[16];
            unpack16(vl[u], vh[u], v);
            norm_rotate<D, INTER>(v, norm, w, p.r.eps, t < nrot, a);
            if (there && h < h1) {
                if (norm || t < nrot) pack16(v, vl[u], vh[u]);  // else the bits as they are
                y[h * yh + lo] = vl[u];
                y[h * yh + hi] = vh[u];
            }
        }
    }
}

// Blocks [0, page_blocks): a touched page of a sequence and head, of K or of V; the others:
// tokens and heads of Q.
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 4) cache_append_rope_kernel(const CacheAppendRopeParams p) {
    pdl_wait();
    const unsigned x = blockIdx.x;
    if (x < p.page_blocks) {
        const unsigned of_pages = x / p.pages, slot = x - of_pages * p.pages;
        const unsigned item = of_pages >> 1, is_v = of_pages & 1u;
        const int b = static_cast<int>(item / p.c.Hk), hk = static_cast<int>(item - b * p.c.Hk);
        if (slot == 0 && hk == 0 && !is_v && threadIdx.x == 0) check_len(p.c.c, p.c.st, b);
        AppendPage a;
        if (!append_page(p.c, b, static_cast<int>(slot), a)) return;
        if (is_v) append_plain<D>(p.c, a, b, hk, true);
        else append_rotated<D, INTER>(p, a, b, hk);
        return;
    }
    const unsigned y = x - p.page_blocks, rest = y / p.token_tiles, tile = y - rest * p.token_tiles;
    const unsigned b = rest / p.chunks, chunk = rest - b * p.chunks;
    rotate_queries<D, INTER>(p, static_cast<int>(b), static_cast<int>(tile) * p.token_slots, static_cast<int>(chunk));
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
        if (p.hp == 1 || static_cast<long long>(p.token_tiles) * p.chunks * c.B >= 8ll * sms) break;
    }
    const long long page_blocks = 2ll * p.pages * c.Hk * c.B;
    const long long blocks = page_blocks + static_cast<long long>(p.token_tiles) * p.chunks * c.B;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    p.page_blocks = static_cast<unsigned>(page_blocks);
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
