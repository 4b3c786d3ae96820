// C ABI of libattn_sm103a.so: argument validation, TMA tensor maps, launch
// sequencing and the device error word.  The declarations and their contract
// are in include/attn_sm103a.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_sm103a.h"
#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

// Device error word: [0] error bits, [1] id of the first wait that gave up.
__device__ unsigned int g_err_word[2];

constexpr unsigned long long kDefaultWaitLimitNs = 1000000000ull;
unsigned long long g_wait_limit_ns = kDefaultWaitLimitNs;
int g_exp2_offload = 0;  // attn_set_exp2_offload

constexpr int kMaxDevices = 64;

// Architecture check, cached per device (a device's compute capability never
// changes).
struct DeviceArch {
    bool probed = false;
    bool supported = false;
};
DeviceArch g_dev[kMaxDevices];
std::mutex g_dev_mutex;

// Current device: check the architecture and look up the device address of the
// error word.  The address is looked up on every call, not cached: it belongs
// to the module loaded into the device's current context, and a context made
// after cudaDeviceReset (or another context made current on the same device)
// loads the module again, possibly at another address.  The lookup allocates
// nothing.
struct DeviceState {
    unsigned int* err = nullptr;  // device address of g_err_word in the current context
};

attn_status device_state(DeviceState* out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(g_dev_mutex);
        DeviceArch& a = g_dev[dev];
        if (!a.probed) {
            int major = 0, minor = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
                return ATTN_ERR_CUDA;
            a.supported = (major == 10 && minor == 3);
            a.probed = true;
        }
        if (!a.supported) return ATTN_ERR_UNSUPPORTED;
    }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_err_word) != cudaSuccess || p == nullptr) return ATTN_ERR_CUDA;
    out->err = static_cast<unsigned int*>(p);
    return ATTN_OK;
}

DevStatus dev_status(const DeviceState& s) {
    DevStatus st;
    st.word = s.err;
    st.wait_limit_ns = g_wait_limit_ns;
    return st;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point, so that the
// library has no link-time dependency on libcuda.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// 4-D view {d, N, heads, B} of a [B, heads, N, d] tensor with element strides
// s (d contiguous); box {128 bytes of d, 128 rows, 1, 1}, 128-byte swizzle,
// rows >= N read as zero.
bool make_map(CUtensorMap* m, const void* base, bool fp8, int d, int N, int heads, int B,
              const Strides& st) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t eb = fp8 ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                                static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.n) * eb, static_cast<cuuint64_t>(st.h) * eb,
                                   static_cast<cuuint64_t>(st.b) * eb};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / eb), 128u, 1u, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D view {d, Npad, B*H} of the fp32 dQ accumulator; box {32, box_rows, 1}
// (128 bytes x box_rows rows), 128-byte swizzle, used for TMA reductions.
bool make_map_acc(CUtensorMap* m, const float* base, int d, int Npad, int BH, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Npad),
                                static_cast<cuuint64_t>(BH)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4,
                                   static_cast<cuuint64_t>(Npad) * d * 4};
    const cuuint32_t box[3] = {32u, static_cast<cuuint32_t>(box_rows), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every row of a bf16 tensor (base + element strides s) starts on a 32-byte
// boundary: the epilogues then write rows with 32-byte stores.
int rows_v8(const void* base, const Strides& s) {
    return (reinterpret_cast<uintptr_t>(base) & 31u) == 0 && (s.b * 2) % 32 == 0 && (s.h * 2) % 32 == 0 &&
                   (s.n * 2) % 32 == 0
               ? 1
               : 0;
}

Strides dense(int heads, int N, int d) {
    Strides s;
    s.n = d;
    s.h = static_cast<long long>(N) * d;
    s.b = static_cast<long long>(heads) * N * d;
    return s;
}

// Strides usable by TMA and by the 16-byte vector stores: non-negative,
// multiples of 16 bytes, below 2^40 bytes.
bool strides_ok(const Strides& s, int elem_bytes) {
    for (long long x : {s.b, s.h, s.n}) {
        if (x < 0 || (x * elem_bytes) % 16 != 0 || x * elem_bytes >= (1ll << 40)) return false;
    }
    return true;
}

// No two elements of an output share a place: no zero stride over more than one.
bool distinct(const Strides& s, long long nb, long long nh, long long nn) {
    return (nb == 1 || s.b != 0) && (nh == 1 || s.h != 0) && (nn == 1 || s.n != 0);
}

constexpr long long kMaxElems = (1ll << 40);  // keeps every byte offset well inside 64 bits

attn_status check_sizes(int B, int H, int N, int d, float scale, int causal) {
    if (B < 1 || H < 1 || N < 1) return ATTN_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (d <= 0) return ATTN_ERR_INVALID;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    const long long bh = static_cast<long long>(B) * H;
    if (bh > (1ll << 31) - 1) return ATTN_ERR_INVALID;
    if (bh * N * d > kMaxElems) return ATTN_ERR_INVALID;
    const long long ctas = bh * ((N + 2 * kTile - 1) / (2 * kTile));
    const long long ctas_bwd = bh * ((N + kTile - 1) / kTile);
    if (ctas > 0x7fffffffll / 16 || ctas_bwd > 0x7fffffffll) return ATTN_ERR_INVALID;
    return ATTN_OK;
}

attn_status check_group(int H, int Hk) {
    return (Hk >= 1 && Hk <= H && H % Hk == 0) ? ATTN_OK : ATTN_ERR_INVALID;
}

attn_status check_window(int wl, int wr) { return (wl >= -1 && wr >= -1) ? ATTN_OK : ATTN_ERR_INVALID; }

// A bound past the sequence's length is that length: the kernels add it to a position.
void within_length(int N, int* left, int* right) {
    if (*left > N) *left = N;
    if (*right > N) *right = N;
}

long long npad(int N) { return (static_cast<long long>(N) + kTile - 1) / kTile * kTile; }

int sink_tiles_of(int sinks) { return (sinks + kTile - 1) / kTile; }
long long sink_items_of(int B, int Hk, int sinks) { return static_cast<long long>(B) * Hk * sink_tiles_of(sinks); }

// Window and sinks of a sequence of N tokens, as the kernels take them: sinks within
// the sequence, none where the window has no left bound or covers the sequence (which
// is then the plain causal or unmasked launch).
attn_status sink_mask(int N, int* left, int* right, int* sinks) {
    if (*sinks < 0 || check_window(*left, *right) != ATTN_OK) return ATTN_ERR_INVALID;
    if (*left >= N - 1) *left = -1;
    if (*right >= N - 1) *right = -1;
    if (*sinks > N) *sinks = N;
    if (*left < 0) *sinks = 0;
    return ATTN_OK;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BwdLayout {
    size_t dq_acc, lse2, dsum, split_cnt, split_part, total;
    int split_cap;  // parts of split items the workspace holds (0: none)
    int split_cnt_words;
};

// fp32 dQ accumulator, -LSE log2 e, D; for d = 128 (split) also the counters and
// partials of split items: at most min(kBwdSplitCap, items * min(10, ceil(N / 128)))
// parts, items <= B * H * ceil(N / 128) (an item is split at most ten ways, and
// never into more parts than its steps); with sinks (sink_items: key tiles of all
// key/value heads that hold one) at most min(kBwdSinkCap, sink_items * kBwdSinkParts).
BwdLayout bwd_layout(int B, int H, int N, int d, bool split, long long sink_items) {
    const size_t rows = static_cast<size_t>(B) * H * npad(N);
    BwdLayout L;
    L.dq_acc = 0;
    L.lse2 = round256(rows * d * sizeof(float));
    L.dsum = L.lse2 + round256(rows * sizeof(float));
    L.split_cnt = L.split_part = L.dsum + round256(rows * sizeof(float));
    L.total = L.split_cnt;
    L.split_cap = L.split_cnt_words = 0;
    if (split && (d == 128 || sink_items > 0)) {
        const long long tiles = npad(N) / kTile;
        const long long room = sink_items > 0 ? sink_items * kBwdSinkParts
                                              : static_cast<long long>(B) * H * tiles * (tiles < 10 ? tiles : 10);
        const long long most = sink_items > 0 ? kBwdSinkCap : kBwdSplitCap;
        L.split_cap = static_cast<int>(room < most ? room : most);
        if (L.split_cap > 0) {
            L.split_cnt_words = sink_items > 0 ? 0 : kBwdSplitCntWords;
            L.split_part = L.split_cnt + round256(L.split_cnt_words * sizeof(unsigned));
            L.total = L.split_part + round256(static_cast<size_t>(L.split_cap) * 2 * kTile * d * sizeof(float));
        }
    }
    return L;
}

__global__ void wait_selftest_kernel(DevStatus st) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);  // nothing ever arrives on it
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x < 32) {
        wait_warp(b, 0, &abort_flag, st, 0x901);
    } else if (threadIdx.x == 32) {
        wait_one(b, 0, &abort_flag, st, 0x902);
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Launch paths shared by the entry points (all arguments validated here)
// ---------------------------------------------------------------------------

// Split-KV partial buffers (null: single pass).
struct SplitArgs {
    int n_splits = 1;
    int split_len = 0;
    float* o_part = nullptr;
    float* lse_part = nullptr;
};

attn_status fwd_run(const void* q, const Strides& qs, const void* k, const Strides& ks, const void* v,
                    const Strides& vs, void* o, const Strides& os, float* lse, int B, int H, int Hk,
                    int N, int d, float scale, int win_left, int win_right, attn_stream_t stream,
                    const SplitArgs& split = SplitArgs(), int sinks = 0) {
    const int causal = (win_left == -1 && win_right == 0) ? 1 : 0;
    attn_status rc = check_sizes(B, H, N, d, scale, causal);
    if (rc != ATTN_OK) return rc;
    if ((rc = check_group(H, Hk)) != ATTN_OK || (rc = check_window(win_left, win_right)) != ATTN_OK)
        return rc;
    within_length(N, &win_left, &win_right);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return ATTN_ERR_INVALID;
    if (!strides_ok(qs, 2) || !strides_ok(ks, 2) || !strides_ok(vs, 2) || !strides_ok(os, 2))
        return ATTN_ERR_INVALID;
    DeviceState ds;
    if ((rc = device_state(&ds)) != ATTN_OK) return rc;
    CUtensorMap tq, tk, tv;
    if (!make_map(&tq, q, false, d, N, H, B, qs) || !make_map(&tk, k, false, d, N, Hk, B, ks) ||
        !make_map(&tv, v, false, d, N, Hk, B, vs))
        return ATTN_ERR_CUDA;
    FwdParams p;
    p.o = o;
    p.os = os;
    p.lse = lse;
    p.N = N;
    p.BH = B * H;
    p.H = H;
    p.Hk = Hk;
    p.n_pairs = (N + 2 * kTile - 1) / (2 * kTile);
    p.causal = causal;
    p.win_left = win_left;
    p.win_right = win_right;
    p.sinks = sinks;
    p.cs = scale * 1.44269504088896340736f;
    p.out_scale = 1.f;
    p.n_splits = split.n_splits;
    p.split_len = split.n_splits > 1 ? split.split_len : (N + kTile - 1) / kTile;
    p.o_part = split.o_part;
    p.lse_part = split.lse_part;
    p.exp2_offload = 0;
    p.single = 0;
    p.o_v8 = rows_v8(o, os);
    p.st = dev_status(ds);
    return launch_fwd_bf16(d, tq, tk, tv, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

// Number of key-tile splits: none while the CTAs already cover most SMs
// (the partials and the combine then cost more than they give back), else
// the smallest power of two that covers them, at most one split per key tile
// and at most kMaxSplits.
constexpr int kMaxSplits = 16;
int auto_splits(int BH, int N, int num_sms) {
    const long long ctas = static_cast<long long>(BH) * ((N + 2 * kTile - 1) / (2 * kTile));
    const int n_kv = (N + kTile - 1) / kTile;
    int s = 1;
    while (s < kMaxSplits && s < n_kv && ctas * s * 4 < 3ll * num_sms) s *= 2;
    return s < n_kv ? s : n_kv;
}

size_t splitkv_bytes(int B, int H, int N, int d, int S) {
    const size_t rows = static_cast<size_t>(B) * H * N;
    return round256(static_cast<size_t>(S) * rows * d * sizeof(float)) +
           round256(static_cast<size_t>(S) * rows * sizeof(float));
}

// Validated view of the backward workspace.
struct BwdCall {
    DeviceState ds;
    float* dq_acc = nullptr;
    float* lse2 = nullptr;
    float* dsum = nullptr;
    unsigned* split_cnt = nullptr;
    float* split_part = nullptr;
    int split_cap = 0, split_cnt_words = 0;
    int BH = 0, Np = 0;
};

attn_status bwd_prepare(void* workspace, int B, int H, int N, int d, float scale, int causal, bool split,
                        long long sink_items, BwdCall* c) {
    attn_status rc = check_sizes(B, H, N, d, scale, causal);
    if (rc != ATTN_OK) return rc;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return ATTN_ERR_INVALID;
    if ((rc = device_state(&c->ds)) != ATTN_OK) return rc;
    const BwdLayout L = bwd_layout(B, H, N, d, split, sink_items);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    c->dq_acc = reinterpret_cast<float*>(ws + L.dq_acc);
    c->lse2 = reinterpret_cast<float*>(ws + L.lse2);
    c->dsum = reinterpret_cast<float*>(ws + L.dsum);
    c->split_cap = L.split_cap;
    c->split_cnt_words = L.split_cnt_words;
    if (L.split_cap > 0) {
        c->split_cnt = reinterpret_cast<unsigned*>(ws + L.split_cnt);
        c->split_part = reinterpret_cast<float*>(ws + L.split_part);
    }
    c->BH = B * H;
    c->Np = static_cast<int>(npad(N));
    return ATTN_OK;
}

attn_status bwd_pre_run(const void* o, const Strides& os, const void* dout, const Strides& dos,
                        const float* lse, void* workspace, int B, int H, int N, int d, bool split,
                        long long sink_items, attn_stream_t stream) {
    for (const void* p : {o, dout, static_cast<const void*>(lse)})
        if (!aligned16(p)) return ATTN_ERR_INVALID;
    if (!strides_ok(os, 2) || !strides_ok(dos, 2)) return ATTN_ERR_INVALID;
    BwdCall c;
    attn_status rc = bwd_prepare(workspace, B, H, N, d, 1.f, 0, split, sink_items, &c);
    if (rc != ATTN_OK) return rc;
    BwdPreParams pp;
    pp.split_cnt = c.split_cnt;
    pp.split_cnt_words = c.split_cnt_words;
    pp.o = o;
    pp.dout = dout;
    pp.os = os;
    pp.dos = dos;
    pp.lse = lse;
    pp.dq_acc = c.dq_acc;
    pp.lse2 = c.lse2;
    pp.dsum = c.dsum;
    pp.N = N;
    pp.Npad = c.Np;
    pp.BH = c.BH;
    pp.H = H;
    pp.D = d;
    return launch_bwd_pre(pp, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                     : ATTN_ERR_CUDA;
}

attn_status bwd_main_run(const void* q, const Strides& qs, const void* k, const Strides& ks,
                         const void* v, const Strides& vs, const void* dout, const Strides& dos,
                         void* dk, const Strides& dks, void* dv, const Strides& dvs, void* workspace,
                         int B, int H, int Hk, int N, int d, float scale, int win_left, int win_right,
                         int sinks, bool split, attn_stream_t stream, DqConvertParams* sink = nullptr) {
    for (const void* p : {q, k, v, dout, static_cast<const void*>(dk), static_cast<const void*>(dv)})
        if (!aligned16(p)) return ATTN_ERR_INVALID;
    for (const Strides* st : {&qs, &ks, &vs, &dos, &dks, &dvs})
        if (!strides_ok(*st, 2)) return ATTN_ERR_INVALID;
    attn_status rc;
    if ((rc = check_group(H, Hk)) != ATTN_OK || (rc = check_window(win_left, win_right)) != ATTN_OK)
        return rc;
    within_length(N, &win_left, &win_right);
    const int causal = (win_left == -1 && win_right == 0) ? 1 : 0;
    BwdCall c;
    if ((rc = bwd_prepare(workspace, B, H, N, d, scale, causal, split, sink_items_of(B, Hk, sinks), &c)) != ATTN_OK)
        return rc;
    CUtensorMap tq, tk, tv, tdo, tdq;
    if (!make_map(&tq, q, false, d, N, H, B, qs) || !make_map(&tk, k, false, d, N, Hk, B, ks) ||
        !make_map(&tv, v, false, d, N, Hk, B, vs) || !make_map(&tdo, dout, false, d, N, H, B, dos) ||
        !make_map_acc(&tdq, c.dq_acc, d, c.Np, c.BH, d == 128 ? 64 : 128))
        return ATTN_ERR_CUDA;
    BwdParams bp;
    bp.lse2 = c.lse2;
    bp.dsum = c.dsum;
    bp.dq_acc = c.dq_acc;
    bp.dk = dk;
    bp.dv = dv;
    bp.dks = dks;
    bp.dvs = dvs;
    bp.N = N;
    bp.Npad = c.Np;
    bp.BHk = B * Hk;
    bp.H = H;
    bp.Hk = Hk;
    bp.n_kv = (N + kTile - 1) / kTile;
    bp.causal = causal;
    bp.win_left = win_left;
    bp.win_right = win_right;
    bp.sinks = sinks;
    bp.sink_tiles = sink_tiles_of(sinks);
    bp.cs = scale * 1.44269504088896340736f;
    bp.scale = scale;
    bp.split_cap = c.split_cap;
    if (bwd_sink_parts(d, &bp) != cudaSuccess) return ATTN_ERR_CUDA;  // without sinks the launcher decides on a split
    if (sink != nullptr && bp.split_parts > 1) {  // for the conversion
        sink->sink_part = c.split_part;
        sink->parts = bp.split_parts;
        sink->sink_items = static_cast<int>(sink_items_of(B, Hk, sinks));
        sink->BHk = bp.BHk;
        sink->Hk = Hk;
        sink->dk = dk;
        sink->dv = dv;
        sink->dks = dks;
        sink->dvs = dvs;
    }
    bp.split_part = c.split_part;
    bp.split_cnt = c.split_cnt;
    bp.dkv_v8 = rows_v8(dk, dks) && rows_v8(dv, dvs);
    bp.st = dev_status(c.ds);
    return launch_bwd_main(d, tq, tk, tv, tdo, tdq, bp, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

attn_status dq_convert_run(void* dq, const Strides& dqs, void* workspace, int B, int H, int N, int d,
                           float scale, attn_stream_t stream, const DqConvertParams* sink = nullptr) {
    if (!aligned16(dq) || !strides_ok(dqs, 2)) return ATTN_ERR_INVALID;
    BwdCall c;
    attn_status rc = bwd_prepare(workspace, B, H, N, d, scale, 0, false, 0, &c);
    if (rc != ATTN_OK) return rc;
    DqConvertParams cp = {};
    if (sink != nullptr) cp = *sink;
    cp.dq_acc = c.dq_acc;
    cp.dq = dq;
    cp.dqs = dqs;
    cp.N = N;
    cp.Npad = c.Np;
    cp.BH = c.BH;
    cp.H = H;
    cp.D = d;
    cp.scale = scale;
    return launch_dq_convert(cp, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

// The whole backward: everything is validated before the first launch, so a
// bad argument leaves the stream untouched.
attn_status bwd_run(const void* q, const Strides& qs, const void* k, const Strides& ks, const void* v,
                    const Strides& vs, const void* o, const Strides& os, const void* dout,
                    const Strides& dos, const float* lse, void* dq, const Strides& dqs, void* dk,
                    const Strides& dks, void* dv, const Strides& dvs, void* workspace, int B, int H,
                    int Hk, int N, int d, float scale, int win_left, int win_right,
                    attn_stream_t stream, bool split = true, int sinks = 0) {
    const int causal = (win_left == -1 && win_right == 0) ? 1 : 0;
    attn_status rc = check_sizes(B, H, N, d, scale, causal);
    if (rc != ATTN_OK) return rc;
    if ((rc = check_group(H, Hk)) != ATTN_OK || (rc = check_window(win_left, win_right)) != ATTN_OK)
        return rc;
    for (const void* p : {q, k, v, o, dout, static_cast<const void*>(lse), static_cast<const void*>(dq),
                          static_cast<const void*>(dk), static_cast<const void*>(dv)})
        if (!aligned16(p)) return ATTN_ERR_INVALID;
    for (const Strides* st : {&qs, &ks, &vs, &os, &dos, &dqs, &dks, &dvs})
        if (!strides_ok(*st, 2)) return ATTN_ERR_INVALID;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return ATTN_ERR_INVALID;
    DqConvertParams sink = {};
    if ((rc = bwd_pre_run(o, os, dout, dos, lse, workspace, B, H, N, d, split, sink_items_of(B, Hk, sinks),
                          stream)) != ATTN_OK)
        return rc;
    if ((rc = bwd_main_run(q, qs, k, ks, v, vs, dout, dos, dk, dks, dv, dvs, workspace, B, H, Hk, N, d,
                           scale, win_left, win_right, sinks, split, stream, &sink)) != ATTN_OK)
        return rc;
    return dq_convert_run(dq, dqs, workspace, B, H, N, d, scale, stream, &sink);
}

// Strides of a [nb, nh, nn, d] view.  A stride over one element is only ever multiplied by 0,
// and PyTorch may hold any number there: a row's length takes its place, which no check of
// alignment turns down.
Strides from_abi(const attn_strides_t& s, int nb, int nh, int nn, int d) {
    Strides r;
    r.b = nb == 1 ? d : s.b;
    r.h = nh == 1 ? d : s.h;
    r.n = nn == 1 ? d : s.n;
    return r;
}

attn_status cache_view(const attn_cache_t* c, int B, int Hk, int d, CacheView* out) {
    if (c == nullptr || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return ATTN_ERR_INVALID;
    for (const void* p : {static_cast<const void*>(c->k_scale), static_cast<const void*>(c->v_scale),
                          static_cast<const void*>(c->page_table), static_cast<const void*>(c->seq_lens)})
        if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return ATTN_ERR_INVALID;
    if (c->num_pages < 1 || c->max_pages < 1 || (B > 1 && c->table_stride < c->max_pages) ||
        c->table_stride < 0 || c->table_stride > kMaxElems)
        return ATTN_ERR_INVALID;
    const int ps = c->page_size;
    if (ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0 || c->max_pages > (1 << 30) / ps) return ATTN_ERR_INVALID;
    out->ks = from_abi(c->ks, c->num_pages, Hk, ps, d);
    out->vs = from_abi(c->vs, c->num_pages, Hk, ps, d);
    if (!strides_ok(out->ks, 1) || !strides_ok(out->vs, 1)) return ATTN_ERR_INVALID;
    out->k_pages = static_cast<uint8_t*>(c->k_pages);
    out->v_pages = static_cast<uint8_t*>(c->v_pages);
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->table = c->page_table;
    out->table_stride = c->table_stride;
    out->seq_lens = c->seq_lens;
    out->num_pages = c->num_pages;
    out->page_size = ps;
    out->max_pages = c->max_pages;
    out->page_shift = 0;
    while ((1 << out->page_shift) < ps) ++out->page_shift;
    return ATTN_OK;
}

// The workspace is laid out for the largest launch, so that its size needs no device.
struct CacheLayout {
    size_t stat, border, total;
};
CacheLayout cache_layout(bool prompt, int d) {
    const size_t rows = prompt ? static_cast<size_t>(2) * kPromptGridMax * kPromptRows
                               : static_cast<size_t>(2) * kCacheGridMax * kCacheRowsMax;
    CacheLayout L;
    L.stat = round256(rows * d * sizeof(float));
    L.border = L.stat + round256(rows * sizeof(float2));
    L.total = L.border + round256((prompt ? kPromptGridMax : kCacheGridMax) * sizeof(CacheBorder));
    return L;
}
bool cache_prompt(int H, int Hk, int T) { return static_cast<long long>(T) * (H / Hk) > kPromptMinRows; }


}  // namespace

int check_problem(int B, int H, int N, int d, float scale, int causal) {
    return static_cast<int>(check_sizes(B, H, N, d, scale, causal));
}

size_t bwd_workspace_bytes_for(int B, int H, int N, int d, bool split) {
    if (check_sizes(B, H, N, d, 1.f, 0) != ATTN_OK) return 0;
    return bwd_layout(B, H, N, d, split, 0).total;
}

int bwd_dense(const void* q, const void* k, const void* v, const void* o, const void* dout,
              const float* lse, void* dq, void* dk, void* dv, void* workspace, int B, int H, int N,
              int d, float scale, int causal, bool split, cudaStream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    const Strides ds = dense(H, N, d);
    return static_cast<int>(bwd_run(q, ds, k, ds, v, ds, o, ds, dout, ds, lse, dq, ds, dk, ds, dv, ds,
                                    workspace, B, H, H, N, d, scale, -1, causal ? 0 : -1, stream, split));
}

cudaError_t launch_wait_selftest(DevStatus st, cudaStream_t stream) {
    wait_selftest_kernel<<<1, 64, 0, stream>>>(st);
    return cudaGetLastError();
}

}  // namespace attn

using namespace attn;

extern "C" {

attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                     int N, int d, float scale, int causal, attn_stream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    const Strides ds = dense(H, N, d);
    return fwd_run(q, ds, k, ds, v, ds, o, ds, lse, B, H, H, N, d, scale, -1, causal ? 0 : -1, stream);
}

attn_status attn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int Hk, int N, int d, float scale, int causal, attn_stream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (check_group(H, Hk) != ATTN_OK) return ATTN_ERR_INVALID;
    const Strides qs = dense(H, N, d), ks = dense(Hk, N, d);
    return fwd_run(q, qs, k, ks, v, ks, o, qs, lse, B, H, Hk, N, d, scale, -1, causal ? 0 : -1, stream);
}

attn_status attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                            int H, int Hk, int N, int d, float scale, int window_left,
                            int window_right, attn_stream_t stream) {
    if (check_group(H, Hk) != ATTN_OK) return ATTN_ERR_INVALID;
    const Strides qs = dense(H, N, d), ks = dense(Hk, N, d);
    return fwd_run(q, qs, k, ks, v, ks, o, qs, lse, B, H, Hk, N, d, scale, window_left, window_right,
                   stream);
}

attn_status attn_fwd_strided(const void* q, attn_strides_t qs, const void* k, attn_strides_t ks,
                             const void* v, attn_strides_t vs, void* o, attn_strides_t os, float* lse,
                             int B, int H, int Hk, int N, int d, float scale, int window_left,
                             int window_right, attn_stream_t stream) {
    const auto of_q = [&](const attn_strides_t& s) { return from_abi(s, B, H, N, d); };
    const auto of_k = [&](const attn_strides_t& s) { return from_abi(s, B, Hk, N, d); };
    return fwd_run(q, of_q(qs), k, of_k(ks), v, of_k(vs), o, of_q(os), lse, B, H, Hk, N, d, scale,
                   window_left, window_right, stream);
}

size_t attn_fwd_splitkv_workspace_bytes(int B, int H, int N, int d, int num_splits) {
    if (check_sizes(B, H, N, d, 1.f, 0) != ATTN_OK) return 0;
    if (num_splits < 0 || num_splits > kMaxSplits) return 0;
    if (num_splits == 0) num_splits = kMaxSplits;  // enough for any automatic choice
    return splitkv_bytes(B, H, N, d, num_splits);
}

attn_status attn_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                             void* workspace, int B, int H, int N, int d, float scale, int causal,
                             int num_splits, attn_stream_t stream) {
    attn_status rc = check_sizes(B, H, N, d, scale, causal);
    if (rc != ATTN_OK) return rc;
    if (num_splits < 0 || num_splits > kMaxSplits) return ATTN_ERR_INVALID;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return ATTN_ERR_INVALID;
    const int BH = B * H;
    const int n_kv = (N + kTile - 1) / kTile;
    int S = num_splits;
    if (S == 0) {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return ATTN_ERR_CUDA;
        S = auto_splits(BH, N, sms);
    }
    if (S > n_kv) S = n_kv;
    const Strides ds = dense(H, N, d);
    const int wr = causal ? 0 : -1;
    if (S <= 1) return fwd_run(q, ds, k, ds, v, ds, o, ds, lse, B, H, H, N, d, scale, -1, wr, stream);
    SplitArgs sp;
    sp.split_len = (n_kv + S - 1) / S;
    sp.n_splits = (n_kv + sp.split_len - 1) / sp.split_len;  // no empty trailing split
    const size_t rows = static_cast<size_t>(BH) * N;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    sp.o_part = reinterpret_cast<float*>(ws);
    sp.lse_part = reinterpret_cast<float*>(
        ws + round256(static_cast<size_t>(sp.n_splits) * rows * d * sizeof(float)));
    if ((rc = fwd_run(q, ds, k, ds, v, ds, o, ds, lse, B, H, H, N, d, scale, -1, wr, stream, sp)) !=
        ATTN_OK)
        return rc;
    CombineParams c;
    c.o_part = sp.o_part;
    c.lse_part = sp.lse_part;
    c.o = o;
    c.os = ds;
    c.lse = lse;
    c.S = sp.n_splits;
    c.BH = BH;
    c.H = H;
    c.N = N;
    c.D = d;
    return launch_splitkv_combine(c, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

attn_status attn_fwd_fp8(const void* q8, const void* k8, const void* v8, float sq, float sk, float sv,
                         void* o, float* lse, int B, int H, int N, int d, float scale, int causal,
                         attn_stream_t stream) {
    attn_status rc = check_sizes(B, H, N, d, scale, causal);
    if (rc != ATTN_OK) return rc;
    if (d != 128) return ATTN_ERR_UNSUPPORTED;
    for (float s : {sq, sk, sv})
        if (!(s > 0.f) || !std::isfinite(s)) return ATTN_ERR_INVALID;
    if (!aligned16(q8) || !aligned16(k8) || !aligned16(v8) || !aligned16(o) || !aligned16(lse))
        return ATTN_ERR_INVALID;
    DeviceState ds;
    if ((rc = device_state(&ds)) != ATTN_OK) return rc;
    const Strides st = dense(H, N, d);
    CUtensorMap tq, tk, tv;
    if (!make_map(&tq, q8, true, d, N, H, B, st) || !make_map(&tk, k8, true, d, N, H, B, st) ||
        !make_map(&tv, v8, true, d, N, H, B, st))
        return ATTN_ERR_CUDA;
    FwdParams p;
    p.o = o;
    p.os = st;
    p.lse = lse;
    p.N = N;
    p.BH = B * H;
    p.H = H;
    p.Hk = H;
    p.n_pairs = (N + 2 * kTile - 1) / (2 * kTile);
    p.causal = causal;
    p.win_left = -1;
    p.win_right = causal ? 0 : -1;
    p.sinks = 0;
    p.cs = scale * sq * sk * 1.44269504088896340736f;
    p.out_scale = sv;
    p.n_splits = 1;
    p.split_len = (N + kTile - 1) / kTile;
    p.o_part = nullptr;
    p.lse_part = nullptr;
    p.exp2_offload = g_exp2_offload;
    p.single = 0;
    p.o_v8 = rows_v8(o, st);
    p.st = dev_status(ds);
    return launch_fwd_fp8(d, tq, tk, tv, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

size_t attn_bwd_workspace_bytes(int B, int H, int N, int d) {
    return bwd_workspace_bytes_for(B, H, N, d, true);
}

attn_status attn_bwd_preprocess(const void* o, const void* dout, const float* lse, void* workspace,
                                int B, int H, int N, int d, attn_stream_t stream) {
    if (check_sizes(B, H, N, d, 1.f, 0) != ATTN_OK) return check_sizes(B, H, N, d, 1.f, 0);
    const Strides ds = dense(H, N, d);
    return bwd_pre_run(o, ds, dout, ds, lse, workspace, B, H, N, d, true, 0, stream);
}

attn_status attn_bwd_main(const void* q, const void* k, const void* v, const void* dout, void* dk,
                          void* dv, void* workspace, int B, int H, int N, int d, float scale,
                          int causal, attn_stream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (check_sizes(B, H, N, d, scale, causal) != ATTN_OK) return check_sizes(B, H, N, d, scale, causal);
    const Strides ds = dense(H, N, d);
    return bwd_main_run(q, ds, k, ds, v, ds, dout, ds, dk, ds, dv, ds, workspace, B, H, H, N, d, scale,
                        -1, causal ? 0 : -1, 0, true, stream);
}

attn_status attn_bwd_dq_convert(void* dq, void* workspace, int B, int H, int N, int d, float scale,
                                attn_stream_t stream) {
    if (check_sizes(B, H, N, d, scale, 0) != ATTN_OK) return check_sizes(B, H, N, d, scale, 0);
    return dq_convert_run(dq, dense(H, N, d), workspace, B, H, N, d, scale, stream);
}

attn_status attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, void* workspace, int B, int H,
                     int N, int d, float scale, int causal, attn_stream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (check_sizes(B, H, N, d, scale, causal) != ATTN_OK) return check_sizes(B, H, N, d, scale, causal);
    const Strides ds = dense(H, N, d);
    return bwd_run(q, ds, k, ds, v, ds, o, ds, dout, ds, lse, dq, ds, dk, ds, dv, ds, workspace, B, H,
                   H, N, d, scale, -1, causal ? 0 : -1, stream);
}

attn_status attn_bwd_gqa(const void* q, const void* k, const void* v, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv,
                         void* workspace, int B, int H, int Hk, int N, int d, float scale, int causal,
                         attn_stream_t stream) {
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (check_group(H, Hk) != ATTN_OK) return ATTN_ERR_INVALID;
    if (check_sizes(B, H, N, d, scale, causal) != ATTN_OK) return check_sizes(B, H, N, d, scale, causal);
    const Strides qs = dense(H, N, d), ks = dense(Hk, N, d);
    return bwd_run(q, qs, k, ks, v, ks, o, qs, dout, qs, lse, dq, qs, dk, ks, dv, ks, workspace, B, H,
                   Hk, N, d, scale, -1, causal ? 0 : -1, stream);
}

attn_status attn_bwd_window(const void* q, const void* k, const void* v, const void* o,
                            const void* dout, const float* lse, void* dq, void* dk, void* dv,
                            void* workspace, int B, int H, int Hk, int N, int d, float scale,
                            int window_left, int window_right, attn_stream_t stream) {
    if (check_group(H, Hk) != ATTN_OK) return ATTN_ERR_INVALID;
    if (check_sizes(B, H, N, d, scale, 0) != ATTN_OK) return check_sizes(B, H, N, d, scale, 0);
    const Strides qs = dense(H, N, d), ks = dense(Hk, N, d);
    return bwd_run(q, qs, k, ks, v, ks, o, qs, dout, qs, lse, dq, qs, dk, ks, dv, ks, workspace, B, H,
                   Hk, N, d, scale, window_left, window_right, stream);
}

attn_status attn_bwd_strided(const void* q, attn_strides_t qs, const void* k, attn_strides_t ks,
                             const void* v, attn_strides_t vs, const void* o, attn_strides_t os,
                             const void* dout, attn_strides_t dos, const float* lse, void* dq,
                             attn_strides_t dqs, void* dk, attn_strides_t dks, void* dv,
                             attn_strides_t dvs, void* workspace, int B, int H, int Hk, int N, int d,
                             float scale, int window_left, int window_right, attn_stream_t stream) {
    const auto of_q = [&](const attn_strides_t& s) { return from_abi(s, B, H, N, d); };
    const auto of_k = [&](const attn_strides_t& s) { return from_abi(s, B, Hk, N, d); };
    return bwd_run(q, of_q(qs), k, of_k(ks), v, of_k(vs), o, of_q(os), dout,
                   of_q(dos), lse, dq, of_q(dqs), dk, of_k(dks), dv, of_k(dvs),
                   workspace, B, H, Hk, N, d, scale, window_left, window_right, stream);
}

attn_status attn_fwd_sinks(const void* q, attn_strides_t qs, const void* k, attn_strides_t ks, const void* v,
                           attn_strides_t vs, void* o, attn_strides_t os, float* lse, int B, int H, int Hk, int N,
                           int d, float scale, int window_left, int window_right, int sinks, attn_stream_t stream) {
    const auto of_q = [&](const attn_strides_t& s) { return from_abi(s, B, H, N, d); };
    const auto of_k = [&](const attn_strides_t& s) { return from_abi(s, B, Hk, N, d); };
    if (sink_mask(N, &window_left, &window_right, &sinks) != ATTN_OK || !distinct(of_q(os), B, H, N))
        return ATTN_ERR_INVALID;
    return fwd_run(q, of_q(qs), k, of_k(ks), v, of_k(vs), o, of_q(os), lse, B, H, Hk, N, d, scale,
                   window_left, window_right, stream, SplitArgs(), sinks);
}

size_t attn_bwd_sinks_workspace_bytes(int B, int H, int Hk, int N, int d, int sinks) {
    if (check_sizes(B, H, N, d, 1.f, 0) != ATTN_OK || check_group(H, Hk) != ATTN_OK || sinks < 0) return 0;
    // room for either launch: whether there are sinks to split for depends on the window
    const size_t plain = bwd_layout(B, H, N, d, true, 0).total;
    const size_t split = bwd_layout(B, H, N, d, true, sink_items_of(B, Hk, sinks < N ? sinks : N)).total;
    return plain > split ? plain : split;
}

attn_status attn_bwd_sinks(const void* q, attn_strides_t qs, const void* k, attn_strides_t ks, const void* v,
                           attn_strides_t vs, const void* o, attn_strides_t os, const void* dout, attn_strides_t dos,
                           const float* lse, void* dq, attn_strides_t dqs, void* dk, attn_strides_t dks, void* dv,
                           attn_strides_t dvs, void* workspace, int B, int H, int Hk, int N, int d, float scale,
                           int window_left, int window_right, int sinks, attn_stream_t stream) {
    const auto of_q = [&](const attn_strides_t& s) { return from_abi(s, B, H, N, d); };
    const auto of_k = [&](const attn_strides_t& s) { return from_abi(s, B, Hk, N, d); };
    if (sink_mask(N, &window_left, &window_right, &sinks) != ATTN_OK || !distinct(of_q(dqs), B, H, N) ||
        !distinct(of_k(dks), B, Hk, N) || !distinct(of_k(dvs), B, Hk, N))
        return ATTN_ERR_INVALID;
    return bwd_run(q, of_q(qs), k, of_k(ks), v, of_k(vs), o, of_q(os), dout, of_q(dos), lse, dq,
                   of_q(dqs), dk, of_k(dks), dv, of_k(dvs), workspace, B, H, Hk, N, d, scale, window_left,
                   window_right, stream, true, sinks);
}

attn_status attn_cache_append(const attn_cache_t* cache, const void* k, attn_strides_t ks, const void* v,
                              attn_strides_t vs, const int32_t* new_lens, int B, int Hk, int T, int d,
                              attn_stream_t stream) {
    attn_status rc = check_sizes(B, Hk, T, d, 1.f, 0);
    if (rc != ATTN_OK) return rc;
    CacheAppendParams p;
    if ((rc = cache_view(cache, B, Hk, d, &p.c)) != ATTN_OK) return rc;
    if (B > 32767 || Hk > 65535) return ATTN_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(new_lens) & 3u) != 0) return ATTN_ERR_INVALID;
    p.k = k;
    p.v = v;
    p.ks = from_abi(ks, B, Hk, T, d);
    p.vs = from_abi(vs, B, Hk, T, d);
    if (!strides_ok(p.ks, 2) || !strides_ok(p.vs, 2)) return ATTN_ERR_INVALID;
    if (!distinct(p.c.ks, p.c.num_pages, Hk, p.c.page_size) || !distinct(p.c.vs, p.c.num_pages, Hk, p.c.page_size))
        return ATTN_ERR_INVALID;
    p.new_lens = new_lens;
    p.B = B;
    p.Hk = Hk;
    p.T = T;
    p.D = d;
    DeviceState ds;
    if ((rc = device_state(&ds)) != ATTN_OK) return rc;
    p.st = dev_status(ds);
    return launch_cache_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_cache_workspace_bytes(int B, int H, int Hk, int T, int d) {
    if (check_sizes(B, H, T, d, 1.f, 0) != ATTN_OK || check_group(H, Hk) != ATTN_OK) return 0;
    return cache_layout(cache_prompt(H, Hk, T), d).total;
}

attn_status attn_fwd_cache(const attn_cache_t* cache, const void* q, attn_strides_t qs, void* o, attn_strides_t os,
                           float* lse, void* workspace, const int32_t* q_lens, int B, int H, int Hk, int T, int d,
                           float scale, int window_left, int sinks, attn_stream_t stream) {
    attn_status rc = check_sizes(B, H, T, d, scale, 0);
    if (rc != ATTN_OK) return rc;
    if ((rc = check_group(H, Hk)) != ATTN_OK || (rc = check_window(window_left, 0)) != ATTN_OK) return rc;
    if (sinks < 0) return ATTN_ERR_INVALID;
    CacheFwdParams p;
    if ((rc = cache_view(cache, B, Hk, d, &p.c)) != ATTN_OK) return rc;
    if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || (reinterpret_cast<uintptr_t>(q_lens) & 3u) != 0)
        return ATTN_ERR_INVALID;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return ATTN_ERR_INVALID;
    // rows of a key/value head, and pairs of query tiles of all sequences, count in 32 bits
    const long long rows = static_cast<long long>(T) * (H / Hk);
    if (rows > (1 << 30) || B * ((rows + kPromptRows - 1) / kPromptRows) > (1 << 30)) return ATTN_ERR_INVALID;
    p.q = q;
    p.o = o;
    p.qs = from_abi(qs, B, H, T, d);
    p.os = from_abi(os, B, H, T, d);
    if (!strides_ok(p.qs, 2) || !strides_ok(p.os, 2) || !distinct(p.os, B, H, T)) return ATTN_ERR_INVALID;
    p.lse = lse;
    p.q_lens = q_lens;
    p.B = B;
    p.H = H;
    p.Hk = Hk;
    p.T = T;
    p.D = d;
    p.cs = scale * 1.44269504088896340736f;
    // A window that covers the longest sequence the table can hold is none, and positions
    // stay far inside 32 bits.
    const int cap = cache->max_pages * cache->page_size;
    p.left = window_left >= cap ? -1 : window_left;
    p.sinks = p.left < 0 ? 0 : (sinks < cap ? sinks : cap);
    p.part = static_cast<float*>(workspace);
    const bool prompt = cache_prompt(H, Hk, T);
    const CacheLayout L = cache_layout(prompt, d);
    p.stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + L.stat);
    p.border = reinterpret_cast<CacheBorder*>(static_cast<uint8_t*>(workspace) + L.border);
    DeviceState ds;
    if ((rc = device_state(&ds)) != ATTN_OK) return rc;
    p.st = dev_status(ds);
    p.rows = p.grid = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return (prompt ? launch_cache_prompt(p, s) : launch_cache_decode(p, s)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_check_device_error(attn_stream_t stream, unsigned int* site) {
    if (site) *site = 0;
    DeviceState ds;
    attn_status rc = device_state(&ds);
    if (rc != ATTN_OK) return rc;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return ATTN_ERR_CUDA;
    unsigned int host[2] = {0, 0};
    const unsigned int zero[2] = {0, 0};
    if (cudaMemcpy(host, ds.err, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemcpy(ds.err, zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (site) *site = host[1];
    if (host[0] == ATTN_DEVERR_PAGE) return ATTN_ERR_PAGE;
    return host[0] ? ATTN_ERR_TIMEOUT : ATTN_OK;
}

void attn_set_exp2_offload(int on) { g_exp2_offload = on ? 1 : 0; }

void attn_set_wait_limit_ns(unsigned long long ns) {
    g_wait_limit_ns = ns ? ns : kDefaultWaitLimitNs;
}

attn_status attn_selftest_wait_timeout(attn_stream_t stream) {
    DeviceState ds;
    attn_status rc = device_state(&ds);
    if (rc != ATTN_OK) return rc;
    return launch_wait_selftest(dev_status(ds), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

const char* attn_status_string(attn_status s) {
    switch (s) {
        case ATTN_OK: return "ATTN_OK";
        case ATTN_ERR_INVALID: return "ATTN_ERR_INVALID";
        case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
        case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
        case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT";
        case ATTN_ERR_PAGE: return "ATTN_ERR_PAGE";
    }
    return "ATTN_ERR_UNKNOWN";
}

int attn_build_flags(void) { return kDebugChecks ? 1 : 0; }

int attn_kernel_smem_bytes(int which, int d) {
    if (which == 0) return fwd_smem_bytes(d, false);
    if (which == 1) return fwd_smem_bytes(d, true);
    if (which == 2) return bwd_smem_bytes(d);
    return 0;
}

}  // extern "C"
