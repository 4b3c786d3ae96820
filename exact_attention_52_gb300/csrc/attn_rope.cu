// Rotary positions on the heads of Q and K, with or without a norm of each head, forward and
// backward: one pass over the data, bound by reading and writing it.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"
#include "rope_ops.cuh"

namespace attn {
namespace {

// ---------------------------------------------------------------------------
// Rotation (forward; backward where there is no norm: the transpose, sign = -1)
// ---------------------------------------------------------------------------
// A block takes TT tokens and HT * hp heads of Q or of K: thread (slot, t) holds 16 elements of
// head slot / TT + HT * i of token slot % TT, i = 0 .. hp - 1, so that a token's angles (8 a
// thread, some 50 instructions each) serve hp heads.  Bound by the memory: 40 heads of 8192 tokens,
// d = 128, 26.7 us, 6.3 TB/s (with norms 29); 32 heads of 4 x 1024 tokens, d = 64, 9.2 us, a short wave
// of blocks.  (Four heads' loads at a time into registers: 29 us.)
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_kernel(const RopeParams p) {
    constexpr int TPR = D / 16, SLOTS = kRopeThreads / TPR;
    __shared__ RopeRing ring;
    pdl_wait();
    const int which = static_cast<int>(blockIdx.y) >= p.chunks[0] ? 1 : 0;
    const int chunk = static_cast<int>(blockIdx.y) - (which ? p.chunks[0] : 0);
    const int slot = threadIdx.x / TPR, TT = p.token_slots, HT = SLOTS / TT;
    const long long tok = static_cast<long long>(blockIdx.x) * TT + slot % TT;
    const bool there = tok < p.tokens;
    const long long b = there ? div_mostly32(tok, p.N) : 0;
    const int n = there ? static_cast<int>(tok - b * p.N) : 0;
    const Strides xs = p.xs[which], ys = p.ys[which];
    const int first = chunk * HT * p.hp, heads = min(p.heads[which] - first, HT * p.hp);
    rotate_heads<D, INTER>(p.r, which ? p.r.k_weight : p.r.q_weight, p.sign, there,
                           there && p.positions ? __ldg(p.positions + b * p.position_stride + n) : n,
                           static_cast<const uint4*>(p.x[which]) + (b * xs.b + n * xs.n) / 8, xs.h / 8,
                           static_cast<uint4*>(p.y[which]) + (b * ys.b + n * ys.n) / 8, ys.h / 8, first + slot / TT, HT,
                           first + heads, (heads + HT - 1) / HT, ring);
}

// ---------------------------------------------------------------------------
// Backward of norm and rotation
// ---------------------------------------------------------------------------
// With u = x r: dn = R^T dy, dw += dn u, g = dn w, dx = r (g - u mean(g u)).  Reads x and dy,
// writes dx; r is worked out again.  Block c of a tensor's share of the grid takes the c-th of
// equal ranges of (token tile, HT heads) units, works angles out when the tile changes and keeps dw
// in registers; a block's sums over its threads go to the workspace, one row a block, and a second
// kernel adds the rows in their order: no atomics, so the sums are the same every time.
// Bound by the memory, then by issue in 16 warps an SM: each thread copies its own elements
// kBwdStages - 1 units ahead into its own places in shared memory, which takes no registers and no
// barrier.  40 heads of 8192 tokens, d = 128: 45 us, 5.6 TB/s (one unit ahead in registers 55; five
// blocks an SM, whose registers spill, 64).
constexpr int kBwdStages = 4, kBwdBlocks = 4;  // stages; blocks an SM

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kBwdBlocks) rope_norm_bwd_kernel(const RopeBwdParams p) {
    constexpr int TPR = D / 16, SLOTS = kRopeThreads / TPR;
    __shared__ uint4 ring[kBwdStages][4][kRopeThreads];
    pdl_wait();
    pdl_launch_dependents();
    const int which = static_cast<int>(blockIdx.x) >= p.blocks[0] ? 1 : 0;
    const int c = static_cast<int>(blockIdx.x) - (which ? p.blocks[0] : 0);
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
    const int TT = p.token_slots, HT = SLOTS / TT, nrot = p.r.rot / 16;
    int lo, hi;
    rope_pieces<INTER>(t, nrot, lo, hi);
    // the head's weights, in the order of the pieces that its threads hold
    __shared__ float4 weights[4][TPR];
    if (slot == 0) {
        float w[16];
        load_weight(p.r, which ? p.r.k_weight : p.r.q_weight, lo, hi, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) weights[i][t] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __syncthreads();
    float dw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.f;
    const long long xh = p.xs[which].h / 8, gh = p.gs[which].h / 8, yh = p.ys[which].h / 8;
    const int heads = p.heads[which], per_tile = (heads + HT - 1) / HT;
    const long long units = p.tiles * per_tile;
    const long long u0 = units * c / p.blocks[which], u1 = units * (c + 1) / p.blocks[which];

    // A unit's token and head for this thread; walked twice, by the copies and behind them.
    struct Walk {
        long long tile;
        int b, n, h;
        bool there;  // the token
    };
    auto at_tile = [&](Walk& k, long long tile) {
        const long long tok = tile * TT + slot % TT;
        k.tile = tile;
        k.there = tok < p.tokens;
        k.b = k.there ? static_cast<int>(div_mostly32(tok, p.N)) : 0;
        k.n = k.there ? static_cast<int>(tok - static_cast<long long>(k.b) * p.N) : 0;
    };
    const int h_last = (per_tile - 1) * HT + slot / TT;  // this thread's head in a tile's last unit
    const uint4 *x = nullptr, *dy = nullptr;  // of the copies' token and head
    auto copy_tile = [&](Walk& k, long long tile, int group) {
        at_tile(k, tile);
        k.h = group * HT + slot / TT;
        x = static_cast<const uint4*>(p.x[which]) + (k.b * p.xs[which].b + k.n * p.xs[which].n) / 8 + k.h * xh;
        dy = static_cast<const uint4*>(p.dy[which]) + (k.b * p.gs[which].b + k.n * p.gs[which].n) / 8 + k.h * gh;
    };
    Walk ahead = {}, k;
    long long copied = u0;
    int to_slot = 0;
    auto copy = [&] {
        if (copied < u1) {
            uint4(*to)[kRopeThreads] = ring[to_slot];
            to_slot = to_slot + 1 == kBwdStages ? 0 : to_slot + 1;
            if (ahead.there && ahead.h < heads) {
                cp_async16(smem_u32(&to[0][threadIdx.x]), x + lo);
                cp_async16(smem_u32(&to[1][threadIdx.x]), x + hi);
                cp_async16(smem_u32(&to[2][threadIdx.x]), dy + lo);
                cp_async16(smem_u32(&to[3][threadIdx.x]), dy + hi);
            } else {
                to[0][threadIdx.x] = to[1][threadIdx.x] = to[2][threadIdx.x] = to[3][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (ahead.h == h_last) {
                copy_tile(ahead, ahead.tile + 1, 0);
            } else {
                ahead.h += HT;
                x += HT * xh;
                dy += HT * gh;
            }
        }
        ++copied;
        cp_async_commit();
    };
    copy_tile(ahead, u0 / per_tile, static_cast<int>(u0 % per_tile));
    k = ahead;
#pragma unroll 1
    for (int i = 0; i < kBwdStages - 1; ++i) copy();
    RopeAngles a;
    uint4* dx = nullptr;
    bool turned = false;  // angles and dx are this tile's
    int from_slot = 0;
    for (long long u = u0; u < u1; ++u) {
        cp_async_wait<kBwdStages - 2>();
        const uint4(*from)[kRopeThreads] = ring[from_slot];
        from_slot = from_slot + 1 == kBwdStages ? 0 : from_slot + 1;
        float v[16], g[16];
        unpack16(from[0][threadIdx.x], from[1][threadIdx.x], v);
        unpack16(from[2][threadIdx.x], from[3][threadIdx.x], g);
        copy();  // over what was read a unit ago
        if (!turned) {
            turned = true;
            dx = static_cast<uint4*>(p.dx[which]) + (k.b * p.ys[which].b + k.n * p.ys[which].n) / 8 + k.h * yh;
            if (t < nrot) a.at(p.r, t, p.positions ? __ldg(p.positions + k.b * p.position_stride + k.n) : k.n, -1.f);
        }
        const float r = head_rnorm<D>(v, p.r.eps);
        if (t < nrot) rotate16<INTER>(a, g);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 w = weights[i / 4][t];
            fmul2(v[i], v[i + 1], v[i], v[i + 1], r, r);
            fmul2(v[i + 2], v[i + 3], v[i + 2], v[i + 3], r, r);
            ffma2(dw[i], dw[i + 1], g[i], g[i + 1], v[i], v[i + 1], dw[i], dw[i + 1]);  // (rows that are not there are zeros)
            ffma2(dw[i + 2], dw[i + 3], g[i + 2], g[i + 3], v[i + 2], v[i + 3], dw[i + 2], dw[i + 3]);
            fmul2(g[i], g[i + 1], g[i], g[i + 1], w.x, w.y);
            fmul2(g[i + 2], g[i + 3], g[i + 2], g[i + 3], w.z, w.w);
            ffma2(s0, s1, g[i], g[i + 1], v[i], v[i + 1], s0, s1);
            ffma2(s0, s1, g[i + 2], g[i + 3], v[i + 2], v[i + 3], s0, s1);
        }
        const float mean = head_sum<D>(s0 + s1) * (1.f / D);
        if (k.there && k.h < heads) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                fmul2(g[i], g[i + 1], g[i], g[i + 1], r, r);
                ffma2(v[i], v[i + 1], v[i], v[i + 1], -r * mean, -r * mean, g[i], g[i + 1]);
            }
            uint4 ol, ou;
            pack16(v, ol, ou);
            dx[lo] = ol;
            dx[hi] = ou;
        }
        if (k.h == h_last) {
            at_tile(k, k.tile + 1);
            k.h = slot / TT;
            turned = false;
        } else {
            k.h += HT;
            dx += HT * yh;
        }
    }

    __shared__ float sums[kRopeThreads / 32][D];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
        if ((threadIdx.x & 31) < TPR) sums[threadIdx.x >> 5][8 * (i < 8 ? lo : hi) + (i & 7)] = dw[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kRopeThreads) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kRopeThreads / 32; ++i) v += sums[i][e];
        p.part[static_cast<long long>(blockIdx.x) * D + e] = v;
    }
}

// dw of one tensor (blockIdx.y) and 8 elements: its blocks' rows added up, thread group i taking rows
// i, i + 64, ..., all of whose loads are out at once (3 us by itself, most of it behind the kernel
// before it; ten rows one after the other took 6.5).
__global__ void __launch_bounds__(512) rope_dw_kernel(const RopeBwdParams p) {
    __shared__ float sums[8][65];
    const int e = threadIdx.x & 7, from = threadIdx.x >> 3, which = blockIdx.y;
    pdl_wait();
    const float* part = p.part + static_cast<long long>(which ? p.blocks[0] : 0) * p.D + blockIdx.x * 8 + e;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < (kRopeBwdGridMax + 63) / 64; ++i)
        if (from + 64 * i < p.blocks[which]) v += part[(from + 64ll * i) * p.D];
    sums[e][from] = v;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= 8) return;
    v = sums[warp][lane] + sums[warp][lane + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && p.dw[which]) p.dw[which][blockIdx.x * 8 + warp] = v;
}

int sm_count(cudaError_t* e) {
    int dev = 0, sms = 0;
    *e = cudaGetDevice(&dev);
    if (*e == cudaSuccess) *e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int D>
cudaError_t launch_rope_d(RopeParams p, cudaStream_t stream) {
    constexpr int SLOTS = kRopeThreads / (D / 16);
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess) return e;
    p.token_slots = rope_token_slots(p.tokens, SLOTS);
    const long long tiles = (p.tokens + p.token_slots - 1) / p.token_slots;
    const int HT = SLOTS / p.token_slots;
    // As many heads a thread as leave every SM three blocks (20 heads of 2 x 1999 tokens, forward and
    // backward: 15.8 us; eight blocks, with fewer heads for a thread's angles, 17.3).
    for (p.hp = 8;; p.hp /= 2) {
        for (int i = 0; i < 2; ++i) p.chunks[i] = (p.heads[i] + HT * p.hp - 1) / (HT * p.hp);
        if (p.hp == 1 || tiles * (p.chunks[0] + p.chunks[1]) >= 3ll * sms) break;
    }
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.chunks[0] + p.chunks[1]));
    return p.r.interleaved ? launch_dependent(rope_kernel<D, true>, grid, kRopeThreads, 0, stream, p)
                           : launch_dependent(rope_kernel<D, false>, grid, kRopeThreads, 0, stream, p);
}

template <int D>
cudaError_t launch_rope_norm_bwd_d(RopeBwdParams p, cudaStream_t stream) {
    constexpr int SLOTS = kRopeThreads / (D / 16);
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess) return e;
    p.token_slots = rope_token_slots(p.tokens, SLOTS);
    p.tiles = (p.tokens + p.token_slots - 1) / p.token_slots;
    const int HT = SLOTS / p.token_slots;
    const int grid = sms * kBwdBlocks < kRopeBwdGridMax ? sms * kBwdBlocks : kRopeBwdGridMax;
    const int all = p.heads[0] + p.heads[1];
    for (int i = 0; i < 2; ++i) {
        const long long units = p.tiles * ((p.heads[i] + HT - 1) / HT);
        long long n = i == 0 ? (static_cast<long long>(grid) * p.heads[0] + all / 2) / all : grid - p.blocks[0];
        n = n < units ? n : units;
        p.blocks[i] = p.heads[i] > 0 ? static_cast<int>(n > 1 ? n : 1) : 0;
        if (i == 0 && p.blocks[0] == grid && p.heads[1] > 0) --p.blocks[0];
    }
    const dim3 blocks(static_cast<unsigned>(p.blocks[0] + p.blocks[1]));
    e = p.r.interleaved ? launch_dependent(rope_norm_bwd_kernel<D, true>, blocks, kRopeThreads, 0, stream, p)
                        : launch_dependent(rope_norm_bwd_kernel<D, false>, blocks, kRopeThreads, 0, stream, p);
    return e != cudaSuccess ? e : launch_dependent(rope_dw_kernel, dim3(D / 8, 2), 512, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    if (p.D == 64) return launch_rope_d<64>(p, stream);
    if (p.D == 128) return launch_rope_d<128>(p, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_rope_norm_bwd(const RopeBwdParams& p, cudaStream_t stream) {
    if (p.D == 64) return launch_rope_norm_bwd_d<64>(p, stream);
    if (p.D == 128) return launch_rope_norm_bwd_d<128>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
