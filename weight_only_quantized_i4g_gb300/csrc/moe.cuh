// moe.cuh -- internal interface of the expert layer's operators (declared in
// include/qgemv.h): slots sorted by expert, rows dispatched and combined, the
// combination's gradient, e4m3 x e4m3 products.  Arguments reaching these
// functions have been validated by abi_moe.cu.
#pragma once

#include "kv_cache.cuh"   // element types, packing, programmatic launches

namespace qg {

constexpr int kErrExpert = -8;
constexpr int kMaxSortExperts = 8192;
constexpr int kTogether = 8;        // slots of a token in flight at once; their count goes past k by less

struct SortArgs {
    int *offsets, *order, *place;   // order may be NULL
    const int *ids;
    int slots, experts;
    int bits;                       // of the number `experts` (set by the launch)
};
size_t ws_moe_sort(int slots, int experts);
int run_moe_sort(SortArgs a, void *ws, cudaStream_t st);

struct DispatchArgs {
    void *rows;
    float *scales;                  // e4m3 rows only
    const void *x;
    size_t x_stride;                // elements
    const int *place;               // NULL: slot s is row s
    int tokens, k, width, n_rows;
};
int run_moe_dispatch(const DispatchArgs &a, int x_type, bool codes, cudaStream_t st);

struct CombineArgs {
    void *out;
    const void *y;
    const float *weights;           // NULL: ones
    const int *place;               // NULL: slot s is row s
    int tokens, k, width, n_rows;
};
int run_moe_combine(const CombineArgs &a, int out_type, int y_type, cudaStream_t st);

struct CombineGradArgs {
    void *dy;                       // NULL: not wanted
    float *dweights;                // NULL: not wanted
    const void *dout, *y;
    const float *weights;
    const int *place;
    int tokens, k, width, n_rows;
};
int run_moe_combine_grad(const CombineGradArgs &a, int dout_type, int y_type, cudaStream_t st);

// Y rows of expert e: offsets[e] to offsets[e+1] (device), or all M rows of
// one matrix where offsets is NULL.
struct E4m3Args {
    void *Y;
    int y_type;
    const uint8_t *X;
    const float *x_scale;           // [M, ceil(I/128)]
    const uint8_t *w;               // [experts, O, I]
    const void *w_scale;            // [experts, ceil(O/128), ceil(I/128)], f32 or UE8M0
    bool w_power;                   // UE8M0
    const int *offsets;
    int experts, M, I, O;
    int *err;
};
int run_gemm_e4m3(const E4m3Args &a, cudaStream_t st);
// Where the first expert's rows begin and, from there, expert by expert, rows
// [*from, *most) of expert g: row bounds are held to [0, M] and to their order,
// so a table that leaves the rows or decreases gives no row twice, and the
// thread that asks with err != NULL raises the error word.
__device__ __forceinline__ int held_row(int row, int M) { return min(max(row, 0), M); }
__device__ __forceinline__ void check_offsets(int from, int to, int M, int *err) {
    if (from < 0 || to < from || to > M) raise_device_error(err, kErrExpert);
}
__device__ __forceinline__ void next_rows(const int *offsets, int g, int M, int *from, int *most, int *err) {
    const int lo = offsets[g], hi = offsets[g + 1];
    check_offsets(lo, hi, M, err);
    *from = *most;
    *most = max(*most, held_row(hi, M));
}

// Row of slot s (NULL table: s), -1 for none.
__device__ __forceinline__ int row_of(const int *place, long long s, int n_rows) {
    const long long p = place ? place[s] : s;
    return p >= 0 && p < n_rows ? (int)p : -1;
}

// Elements of the three wide types as f32.
template <int T> struct Elem;
template <> struct Elem<kF32> {
    typedef float Word;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<kBf16> {
    typedef uint16_t Word;
    static __device__ __forceinline__ float get(uint16_t v) { return bf16_bits_to_f32(v); }
    static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)pack_bf16(v, 0.f); }
};
template <> struct Elem<kF16> {
    typedef uint16_t Word;
    static __device__ __forceinline__ float get(uint16_t v) { return f16_bits_to_f32(v); }
    static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)pack_f16(v, 0.f); }
};

}  // namespace qg
