// Writing new tokens into the paged 8-bit cache: what the kernels that append share.
//
// One block per (touched page, head, K or V).  The page's scale is the power of
// two 2^e with the smallest e >= kMinScaleExp such that the largest finite new
// magnitude is at most 448 * 2^e, or the scale it has where older tokens are in
// it and that one is large enough; where it has to grow, the older codes are
// rounded again to the new scale (exact for a power of two, but for codes that
// fall below E4M3's normal range).  Dividing by a power of two is exact, so a
// new code carries one rounding, to nearest even, saturating at 448.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kAppendThreads = 128;
constexpr int kMinScaleExp = -100;

// Smallest power of two s >= 2^kMinScaleExp with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float append_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>(max(e, kMinScaleExp) + 127) << 23);
}

// The new tokens of sequence b that lie in the slot-th page that its new tokens touch.
struct AppendPage {
    int first;   // position of new token 0 (negative: it is not written)
    int lo, hi;  // new positions in this page
    int pid;     // the page
    int old;     // tokens that it holds already
};
// False (for the whole block) where there is nothing to write.
__device__ __forceinline__ bool append_page(const CacheAppendParams& p, int b, int slot, AppendPage& a) {
    const int page = p.c.page_size;
    const int len = p.c.seq_lens[b];
    const int m = p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
    if (m == 0 || len <= 0) return false;
    a.first = len - m;
    const int pg = max(a.first, 0) / page + slot;
    if (pg >= p.c.max_pages) return false;  // behind the table; below it positions stay far inside 32 bits
    a.lo = max(a.first, pg * page);
    a.hi = min(len, pg * page + page);
    if (a.lo >= a.hi) return false;
    a.pid = __ldg(p.c.table + b * p.c.table_stride + pg);
    if (static_cast<unsigned>(a.pid) >= static_cast<unsigned>(p.c.num_pages)) {
        if (threadIdx.x == 0) record_device_error(p.st, ATTN_DEVERR_PAGE, 0x303);
        return false;
    }
    a.old = a.lo - pg * page;
    return true;
}

// Whether the page keeps the scale that it has.
__device__ __forceinline__ bool append_keeps(int old, float was, float amax) {
    return old > 0 && was >= __uint_as_float((kMinScaleExp + 127) << 23) && amax <= 448.f * was;
}

// Tokens rr, rr + rows, ... of the page's older ones, of which the thread holds the 8 codes at
// `codes`, rounded again from scale was to s.
__device__ __forceinline__ void append_grow(uint8_t* codes, long long row, int rr, int rows, int old, float was, float s) {
    const float f = was > 0.f ? was / s : 0.f;
    for (int t = rr; t < old; t += rows) {
        uint2* at = reinterpret_cast<uint2*>(codes + t * row);
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

// Value / scale rounded once: a power of two's inverse is exact; for another scale (one that was
// there) the remainder of the product puts it right, as it would not change the former.  Beyond
// 448 the code saturates.
struct AppendQuotient {
    float s, inv;
    __device__ __forceinline__ explicit AppendQuotient(float scale) : s(scale), inv(1.f / scale) {}
    __device__ __forceinline__ bool exact() const { return (__float_as_uint(s) & 0x7FFFFFu) == 0u; }
    __device__ __forceinline__ float operator()(float v) const {
        const float q = v * inv;
        return fabsf(q) <= 448.f ? fmaf(fmaf(-q, s, v), inv, q) : q;
    }
};

// The page of AppendPage a, head hk, of K or V as they are.
// Bound by reading the new tokens, which stay in registers between the two looks at them
// (read twice they cost a quarter more), and by issue: magnitudes are compared two at a time
// as integers, and the quotient's correction is left out where the scale is a power of two
// (without both a quarter more again).  4 prompts of up to 8192 tokens, 8 heads, d = 128: 23
// us among other calls, 5.8 TB/s, 20 in a row; d = 64 16 in a row, 4.2 TB/s; one token for 32
// sequences 3 us in a row.
template <int D>
__device__ __forceinline__ void append_plain(const CacheAppendParams& p, const AppendPage& a, int b, int hk, bool is_v) {
    constexpr int TPR = D / 8;  // threads per token: 8 elements each
    constexpr int RPP = kAppendThreads / TPR;
    const int first = a.first, lo = a.lo, hi = a.hi, pid = a.pid, old = a.old;
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
    const bool keep = append_keeps(old, was, amax);
    const float s = keep ? was : append_scale(amax);
    if (old > 0 && !keep) append_grow(codes, cs.n, rr, RPP, old, was, s);
    const AppendQuotient quotient(s);
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
    if (quotient.exact()) put_all([&](float v) { return v * quotient.inv; });
    else put_all(quotient);
    if (threadIdx.x == 0 && !keep) *scale = s;
}

}  // namespace attn
