// Rotary positions and norms of single heads: the arithmetic shared by the kernels that
// rotate Q and K (attn_rope.cu) and by the cache's write of rotated keys (attn_cache_rope.cu).
//
// A pair (x1, x2) of a head at position p becomes
//   y1 = f (x1 cos a - x2 sin a),  y2 = f (x2 cos a + x1 sin a),  a = p theta_i,
// and, before that, with a weight w, x becomes x r w with r = (mean of the head's x^2 + eps)^-1/2.
// A thread holds 16 elements of a head, two pieces of 8 (16 bytes each), and a head takes
// D / 16 threads side by side, so that both elements of a pair are in one thread, in the half
// layout (pairs i, i + rot / 2) as in the interleaved one (2i, 2i + 1).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace attn {

// Pieces of 8 elements of thread t of a head, nrot = rot / 16 threads rotating.  Threads from
// nrot on hold elements that only pass.
template <bool INTER>
__device__ __forceinline__ void rope_pieces(int t, int nrot, int& lo, int& hi) {
    lo = INTER || t >= nrot ? 2 * t : t;
    hi = INTER || t >= nrot ? 2 * t + 1 : t + nrot;
}

// Cosines and sines (times f) of the 8 pairs of thread t at a position: pairs 8t .. 8t + 7 in
// either layout.  The table holds theta_i in units of 2^-64 turns, and a position times that,
// modulo 2^64, is the angle within its turn without any error but the table's (2^-65 turns a
// position): nothing is lost far out.  What it is off the nearest quarter turn, at most pi / 4, goes
// to fp32 (2^-25 of it).
struct RopeAngles {
    float c[8], s[8];
    __device__ __forceinline__ void at(const RopeView& r, int t, int pos, float sign) {
        const ulonglong2* turns = reinterpret_cast<const ulonglong2*>(r.turns + 8 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const ulonglong2 w = __ldg(turns + i);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(pos)) * (e ? w.y : w.x);
                const unsigned quarter = (static_cast<unsigned>(a >> 32) + (1u << 29)) >> 30;  // 0 .. 3; 4 of 4 is 0
                const int off = static_cast<int>(static_cast<long long>(a - (static_cast<unsigned long long>(quarter) << 62)) >> 30);
                float sn, cs;
                sincospif(static_cast<float>(off) * 0x1p-33f, &sn, &cs);  // off: 2^-34 turns
                const float x = quarter & 1u ? -sn : cs, y = quarter & 1u ? cs : sn;
                const float f = quarter & 2u ? -r.factor : r.factor;
                c[2 * i + e] = x * f;
                s[2 * i + e] = y * (f * sign);
            }
        }
    }
};

// The thread's elements: x[0 .. 7] of piece lo, x[8 .. 15] of piece hi.
__device__ __forceinline__ void unpack16(const uint4& lo, const uint4& hi, float (&x)[16]) {
    const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[2 * i] = bf16lo(u[i]), x[2 * i + 1] = bf16hi(u[i]);
}
__device__ __forceinline__ void pack16(const float (&x)[16], uint4& lo, uint4& hi) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    lo = make_uint4(u[0], u[1], u[2], u[3]);
    hi = make_uint4(u[4], u[5], u[6], u[7]);
}

template <bool INTER>
__device__ __forceinline__ void rotate16(const RopeAngles& a, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // two pairs at a time, in packed operations
        float &p1 = x[INTER ? 2 * i : i], &p2 = x[INTER ? 2 * i + 1 : i + 8];
        float &q1 = x[INTER ? 2 * i + 2 : i + 1], &q2 = x[INTER ? 2 * i + 3 : i + 9];
        float a0, a1, b0, b1, c0, c1;
        fmul2(a0, a1, p2, q2, a.s[i], a.s[i + 1]);
        fmul2(b0, b1, p1, q1, a.s[i], a.s[i + 1]);
        fmul2(c0, c1, p1, q1, a.c[i], a.c[i + 1]);
        fsub2(p1, q1, c0, c1, a0, a1);
        ffma2(p2, q2, p2, q2, a.c[i], a.c[i + 1], b0, b1);
    }
}

// Sum over the D / 16 threads of a head (neighbouring lanes).
template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = 1; o < D / 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// r of a head, of which x is the thread's part.
template <int D>
__device__ __forceinline__ float head_rnorm(const float (&x)[16], float eps) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) ffma2(a, b, x[i], x[i + 1], x[i], x[i + 1], a, b);
    return rsqrtf(fmaf(head_sum<D>(a + b), 1.f / D, eps));
}

// The thread's 16 weights.
__device__ __forceinline__ void load_weight(const RopeView& r, const void* w, int lo, int hi, float (&out)[16]) {
    if (r.weight_bf16) {
        const uint4* p = static_cast<const uint4*>(w);
        unpack16(__ldg(p + lo), __ldg(p + hi), out);
        return;
    }
    const float4* p = static_cast<const float4*>(w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 v = __ldg(p + 2 * (k < 2 ? lo : hi) + (k & 1));
        out[4 * k] = v.x, out[4 * k + 1] = v.y, out[4 * k + 2] = v.z, out[4 * k + 3] = v.w;
    }
}

// Norm (norm: every thread of a warp alike) and rotation (turns: this thread's pieces rotate) of
// a head, in fp32.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(float (&x)[16], bool norm, const float (&w)[16], float eps, bool turns,
                                            const RopeAngles& a) {
    if (norm) {
        const float r = head_rnorm<D>(x, eps);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            fmul2(x[i], x[i + 1], x[i], x[i + 1], r, r);
            fmul2(x[i], x[i + 1], x[i], x[i + 1], w[i], w[i + 1]);
        }
    }
    if (turns) rotate16<INTER>(a, x);
}

constexpr int kRopeThreads = 128;
// Heads that a thread copies ahead into its own places in shared memory, which takes no registers
// and no barrier: 32 bytes each.
constexpr int kRopeStages = 6;
struct RopeRing {
    uint4 at[kRopeStages][2][kRopeThreads];
};

// Norm (weight not null) and rotation of heads h, h + step, ... (count of them, the same for every
// thread of a block) below h_end of one token (there: it exists) at a position: x and y point to its
// head 0, whose heads are xh and yh pieces apart.
template <int D, bool INTER>
__device__ __forceinline__ void rotate_heads(const RopeView& r, const void* weight, float sign, bool there, int pos,
                                             const uint4* x, long long xh, uint4* y, long long yh, int h, int step, int h_end,
                                             int count, RopeRing& ring) {
    const int tid = threadIdx.x, t = tid % (D / 16), nrot = r.rot / 16;
    int lo, hi;
    rope_pieces<INTER>(t, nrot, lo, hi);
    x += h * xh;
    y += h * yh;
    int copied = 0, slot = 0, h_ahead = h;
    auto copy = [&] {
        if (copied < count) {
            if (there && h_ahead < h_end) {
                cp_async16(smem_u32(&ring.at[slot][0][tid]), x + lo);
                cp_async16(smem_u32(&ring.at[slot][1][tid]), x + hi);
            } else {  // zeros, which take part in a norm's shuffles
                ring.at[slot][0][tid] = ring.at[slot][1][tid] = make_uint4(0u, 0u, 0u, 0u);
            }
            x += step * xh;
            h_ahead += step;
            ++copied;
            slot = slot + 1 == kRopeStages ? 0 : slot + 1;
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kRopeStages - 1; ++i) copy();
    float w[16] = {};
    if (weight) load_weight(r, weight, lo, hi, w);
    RopeAngles a;
    if (there && t < nrot) a.at(r, t, pos, sign);
    int from = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        cp_async_wait<kRopeStages - 2>();
        uint4 vl = ring.at[from][0][tid], vh = ring.at[from][1][tid];
        from = from + 1 == kRopeStages ? 0 : from + 1;
        copy();  // over what was read a head ago
        float v[16];
        unpack16(vl, vh, v);
        norm_rotate<D, INTER>(v, weight != nullptr, w, r.eps, t < nrot, a);
        if (there && h < h_end) {
            if (weight || t < nrot) pack16(v, vl, vh);  // else the bits as they are
            y[lo] = vl;
            y[hi] = vh;
        }
        y += step * yh;
        h += step;
    }
}

// How many tokens a block of `slots` heads at a time takes side by side: all, or as few as
// there are, the rest of the slots taking further heads of the same token.
__host__ __device__ inline int rope_token_slots(long long tokens, int slots) {
    int t = 1;
    while (t < slots && t < tokens) t *= 2;
    return t;
}

}  // namespace attn
