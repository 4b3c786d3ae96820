// Building blocks of the kernels over the paged 8-bit key/value cache: which
// keys a sequence's new queries see, how a page's address is formed, the E4M3
// conversions and per-thread asynchronous copies.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {

// Softmax weights of the cache attention are 2^(score - m + kWeightShift), rounded to
// f16; m may be up to kWeightSlack below the largest score, so a weight is at most 2^15,
// and one is lost to underflow below 2^-31 of the largest.
constexpr float kWeightShift = 7.f, kWeightSlack = 8.f;

// The weights hold the value scales sv, as 2^(score + log2 sv - m + kWeightShift), and the sum
// of a row's probabilities takes them back by 1 / sv.  While every page of a walk has |log2 sv|
// <= kScaleReach, a weight that fp32 flushes (2^-126) is below 2^(-126 + 48) of a sum that is at
// least 2^(kWeightShift - 48), 2^-37 of it, and nothing overflows.  From the first page beyond
// (an append gives a page of zeros 2^-100) the rest of the walk sums 2^(score - u) apart, with
// a maximum u of the plain scores and an exponential more for each of them.  All pages at
// 2^-100: 64 x 4600 tokens 97 us for 95, 40 rows over 16 x 3000 tokens 45 for 34, 2 x 2048
// queries over 16384 keys 1.68 ms for 0.81 (all in a row).  The check and the second copy of
// the step's code cost a call without such pages 0 to 3 %.
constexpr float kScaleReach = 48.f;

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Quotient of numbers that hardly ever pass 32 bits (a 64-bit division takes some
// hundred instructions).
__device__ __forceinline__ long long div_mostly32(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

constexpr float kLn2 = 0.69314718055994530942f;

// The new queries of one sequence and the keys they see.  Query t of q_len sits
// at position len - q_len + t; key j is visible to position p iff j <= p and
// (left < 0, or j >= p - left, or j < sinks).  Keys are walked in blocks of TB
// tokens: the n_sink first blocks (sinks), then n - n_sink blocks from block lo
// on (everything between is seen by no query and is not read).
struct CacheSeq {
    int len, q_len, n, n_sink, lo;
    int key_lo;  // first key of the window of the first query
};

template <int TB>
__device__ __forceinline__ CacheSeq cache_seq(const CacheView& c, const int* q_lens, int T, int left, int sinks,
                                              int b) {
    CacheSeq s;
    const int cap = c.max_pages * c.page_size;
    s.len = min(max(c.seq_lens[b], 0), cap);
    s.q_len = q_lens ? min(max(q_lens[b], 0), T) : T;
    const int first = max(0, s.len - s.q_len);
    s.key_lo = left < 0 ? 0 : max(0, first - left);
    s.lo = s.key_lo / TB;
    s.n_sink = min((min(sinks, s.key_lo) + TB - 1) / TB, s.lo);
    s.n = s.len > 0 ? s.n_sink + (s.len - 1) / TB - s.lo + 1 : 1;
    return s;
}

// Records a length that leaves the table (the kernels read as if it ended with it).
__device__ __forceinline__ void check_len(const CacheView& c, const DevStatus& st, int b) {
    if (static_cast<unsigned>(c.seq_lens[b]) > static_cast<unsigned>(c.max_pages * c.page_size))
        record_device_error(st, ATTN_DEVERR_PAGE, 0x304);
}

// Block v of the walk -> block of the sequence.
__device__ __forceinline__ int cache_block(const CacheSeq& s, int v) { return v < s.n_sink ? v : s.lo + v - s.n_sink; }

// Page of token `tok` of sequence b.  An entry outside the pool is recorded in
// the error word and read as page 0, so that no access leaves the pool.
__device__ __forceinline__ int cache_page(const CacheView& c, const DevStatus& st, int b, int tok) {
    const int pid = __ldg(c.table + static_cast<long long>(b) * c.table_stride + (tok >> c.page_shift));
    if (static_cast<unsigned>(pid) >= static_cast<unsigned>(c.num_pages)) {
        record_device_error(st, ATTN_DEVERR_PAGE, 0x301);
        return 0;
    }
    return pid;
}

// Asynchronous copy of 16 bytes; with `there` false the destination is filled with
// zeros and nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four E4M3 codes (bytes 0-1, bytes 2-3 of w) as two f16 pairs; exact (every
// E4M3 number is an f16 number).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Two floats -> packed f16x2 (round to nearest even); `lo` in bits 15..0.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack_f16x2(uint32_t w, float& lo, float& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
}

// D (16x8, fp32) += A (16x16, f16) B (16x8, f16).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit elements held by a warp: in, lane l has row l/4,
// columns 2(l%4) and + 1; out, the same of the transposed matrix.
__device__ __forceinline__ uint32_t transpose_b16(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A walk whose sum was taken apart (2^u times s, s >= 1; 0: no key) as one like the others: its
// maximum and sum become those of plain scores, and its output sum is to be multiplied twice
// by `half` (the square leaves fp32's range sooner than the product does).
__device__ __forceinline__ void plain_units(float& m, float& l, float u, float s, float& half) {
    const float k = s != 0.f ? floorf(lg2_approx(s)) : 0.f;
    half = s != 0.f ? ex2_approx(0.5f * (m - kWeightShift - u - k)) : 1.f;
    m = s != 0.f ? u + k + kWeightShift : -INFINITY;
    l = s * ex2_approx(-k);
}

// Power of two that brings a row whose largest finite magnitude is `amax` to
// [2^7, 2^8): bf16 values of the row are then exact in f16 down to 2^-24 of that
// largest one, and what lies below is off by at most 2^-32 of it.  Its inverse is
// the power of two with biased exponent 254 minus its own.
__device__ __forceinline__ float f16_row_scale(float amax) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23);  // biased exponent (0: zero or subnormal)
    return __uint_as_float(static_cast<uint32_t>(min(max(261 - e, 1), 254)) << 23);
}

// Row factor times key scale, which turns a product into a score.  Never zero, so
// that a hidden score of -inf stays one (a row of zeros has a row factor of zero); a
// product is below 2^24, so the least normal number in place of less moves no score.
__device__ __forceinline__ float score_factor(float row, float key_scale) { return fmaxf(row * key_scale, 0x1p-126f); }

}  // namespace attn
