// kv_cache.cuh -- device view of a paged key-value cache (qg_kv_cache in
// include/qgemv.h) and what its kernels share: finding a slot, the element
// types, programmatic launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"

namespace qg {

int *device_error_word();
int num_sms();

constexpr int kErrPage = -10;

// Element types (QG_F32 ... in include/qgemv.h).
enum { kF32 = 0, kBf16 = 1, kF16 = 2, kE4m3 = 3 };

// x / d for 0 <= x < 2^31 by one multiplication: mul = ceil(2^(31+L) / d) with
// 2^(L-1) < d <= 2^L errs by less than 2^L / 2^(31+L) per unit of x, under 1/d
// in all.
struct FastDiv { unsigned d, mul, shift; };
inline FastDiv fast_div(int d) {
    unsigned l = 0;
    while ((1ull << l) < (unsigned long long)d) ++l;
    return FastDiv{(unsigned)d, (unsigned)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}
__host__ __device__ __forceinline__ int quotient(int x, FastDiv f) {
    return (int)(((unsigned long long)(unsigned)x * f.mul) >> f.shift);
}

struct KvView {
    char *k, *v;
    const float *k_scale, *v_scale;   // e4m3 only
    float *weight;                    // [n_pages][n_heads][page], or NULL
    long long page_b, head_b, token_b;   // strides of k and v in bytes
    int n_pages, page;
    FastDiv page_div;
    int n_heads, dim, type;
};

struct SlotRef { int page, off; };    // page of the pool (-1: none) and slot inside it

// Page index of slot t in a sequence's table, and t's place in that page.
__device__ __forceinline__ void split_slot(const KvView &c, int t, int *index, int *off) {
    *index = quotient(t, c.page_div);
    *off = t - *index * c.page;
}

// Slot t of the sequence whose table row is `row`; page -1 when the table
// names no page of the pool.
__device__ __forceinline__ SlotRef find_slot(const KvView &c, const int *row, int t) {
    SlotRef r;
    int index;
    split_slot(c, t, &index, &r.off);
    const int p = row[index];
    r.page = (unsigned)p < (unsigned)c.n_pages ? p : -1;
    return r;
}

__device__ __forceinline__ long long slot_bytes(const KvView &c, SlotRef r, int head) {
    return r.page * c.page_b + head * c.head_b + r.off * c.token_b;
}
__device__ __forceinline__ size_t slot_weight(const KvView &c, SlotRef r, int head) {
    return ((size_t)r.page * c.n_heads + head) * c.page + r.off;
}

// Length of sequence b, held to [0, max_len]; a length outside raises the
// error word (by the thread that asks with err != NULL).
__device__ __forceinline__ int seq_len(const int *lens, int b, int max_len, int *err) {
    const int n = lens[b];
    if ((unsigned)n <= (unsigned)max_len) return n;
    raise_device_error(err, kErrPage);
    return n < 0 ? 0 : max_len;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes, the nearest finite ones of lo and hi (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t w;
    asm("cvt.u32.u16 %0, %1;" : "=r"(w) : "h"(r));
    return w;
}
__device__ __forceinline__ uint32_t pack_16(int type, float lo, float hi) {
    return type == kF16 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}
// Four e4m3 codes as two exact f16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t *lo, uint32_t *hi) {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(*lo), "=r"(*hi)
        : "r"(w));
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
    float2 r;
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(r.x), "=f"(r.y) : "r"(w));
    return r;
}

// Launch with programmatic stream serialization: the kernel may start while
// its predecessor runs, and waits for it with griddep_wait().  `cluster`
// consecutive blocks of x form a thread-block cluster.
template <class... P, class... A>
inline int launch_clusters(const char *what, void (*kernel)(P...), dim3 grid, dim3 block, int cluster, size_t smem,
                           cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    count_launch();
    return check_launch(what);
}
template <class... P, class... A>
inline int launch_pdl(const char *what, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                      A... args) {
    return launch_clusters(what, kernel, grid, block, 1, smem, st, args...);
}

// Arguments of the attention over the cache (qattn_paged).
struct AttnArgs {
    KvView c;
    const int *table;
    int table_stride;
    const int *lens;
    int n_seq, max_len;
    void *o;
    int o_type;
    float *lse;                       // or NULL
    const void *q;
    int q_type;
    size_t q_stride;
    int S, n_q_heads, group;          // group = n_q_heads / c.n_heads
    float scale;
    int accumulate;
    int *err;
};

// Arguments of the cache write with rotary positions (qg_rope_append).
constexpr int kMaxPairs = 128;
struct RopeArgs {
    KvView c;
    const int *table;
    int table_stride, n_seq;
    const int *seq, *slot;
    int T;
    void *q;
    int q_type;
    const void *qkv;
    size_t qkv_stride;
    int n_q_heads;
    const int *pos;
    int n_axes;
    const float *inv_freq;
    int rotary, interleaved;
    int *err;
    unsigned char axis[kMaxPairs];
};

// Arguments of the eviction (qg_kv_evict).
struct EvictArgs {
    KvView c;
    const int *table;
    int table_stride;
    const int *dst_table;
    int dst_stride;
    const int *lens;
    int n_seq, max_len, budget, sinks, recent;
    int *kept, *new_lens;
    int *err;
};

int run_rope_append(const RopeArgs &a, int qkv_type, cudaStream_t st);
// Cost units (steps and segments' own) of a sequence of max_len slots; a launch counts up to kAttnMaxUnits.
constexpr double kAttnMaxUnits = 1 << 30;
double attn_units(const KvView &c, int max_len, int S, int n_q_heads);
// Workspace of one call, and of every call of at most these sizes.
size_t ws_attn_paged(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate);
size_t ws_attn_paged_most(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate);
int run_attn_paged(const AttnArgs &a, void *ws, cudaStream_t st);
int run_kv_evict(const EvictArgs &a, cudaStream_t st);

}  // namespace qg
