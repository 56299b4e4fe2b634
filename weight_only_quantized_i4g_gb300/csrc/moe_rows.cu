// moe_rows.cu -- token rows to their experts and back (qg_moe_dispatch,
// qg_moe_combine, qg_moe_combine_grad).
//
//   dispatch  rows[place[t,j]] = x[t], or e4m3(x[t] / s) with s = 2^e for each
//             128 elements, e the least integer >= -126 for which the block's
//             largest finite |x| is at most 448 * 2^e
//   combine   out[t] = sum_j w[t,j] y[place[t,j]], f32, j ascending
//   gradient  dy[place[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[place[t,j]]>
// All three move rows once and are bound by HBM.  Rows of whole 16-byte lines
// at 16-byte addresses go in units of 16 (codes) or 8 elements a thread, a
// token's k rows in flight at once; other rows element by element, eight of a
// thread's 32 apart, so that a warp's loads stay together.
#include "moe.cuh"

namespace qg {
namespace {

constexpr int kRowThreads = 256;
constexpr int kBlock = 128;      // elements of one scale

// Blocks of (ux, ty) threads: ty tokens, ux units of one, `chunks` blocks along a row.
struct RowGrid {
    int units, chunks, ux, ty;
    unsigned blocks;
    RowGrid(int tokens, int n, int threads, int align) : units(n) {
        chunks = (n + threads - 1) / threads;
        ux = ((n + chunks - 1) / chunks + align - 1) / align * align;
        ty = threads / ux > 1 ? threads / ux : 1;
        blocks = (unsigned)(((long long)tokens + ty - 1) / ty * chunks);
    }
    dim3 block() const { return dim3(ux, ty); }
};
// Small calls in small blocks: their time is one block's, and more SMs share the loads.
inline int threads_for(long long units) { return units >= 64LL * kRowThreads * 4 ? kRowThreads : 64; }

struct Place2 {
    unsigned t;                  // token and unit of this thread, which may lie past the last ones
    int u;
};
__device__ __forceinline__ Place2 unit_of(int chunks) {
    const unsigned b = blockIdx.x / chunks, c = blockIdx.x - b * chunks;
    return Place2{b * blockDim.y + threadIdx.y, (int)(c * blockDim.x + threadIdx.x)};
}

// 16 bytes, or zeros, without a branch: a branch a row would have the rows of
// a token wait for one another (combine_prompt: 254 us).
__device__ __forceinline__ uint4 load16_if(bool there, const void *p) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%5];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "r"((int)there), "l"(p));     // volatile: stays behind the wait for the previous kernel
    return v;
}
__device__ __forceinline__ uint16_t load_if(bool there, const uint16_t *p) {
    uint16_t v = 0;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q ld.global.b16 %0, [%2];\n\t}" : "+h"(v) : "r"((int)there), "l"(p));
    return v;
}
__device__ __forceinline__ float load_if(bool there, const float *p) {
    float v = 0.f;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q ld.global.f32 %0, [%2];\n\t}" : "+f"(v) : "r"((int)there), "l"(p));
    return v;
}
// Eight elements, as loaded from a 16-byte address and as f32.
template <int T> struct Raw8 {
    uint4 w[T == kF32 ? 2 : 1];
    __device__ __forceinline__ void load(bool there, const void *p) {
        w[0] = load16_if(there, p);
        if constexpr (T == kF32) w[1] = load16_if(there, static_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (T == kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[4 * i] = __uint_as_float(w[i].x), v[4 * i + 1] = __uint_as_float(w[i].y),
                      v[4 * i + 2] = __uint_as_float(w[i].z), v[4 * i + 3] = __uint_as_float(w[i].w);
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = T == kBf16 ? unpack_bf16(u[i]) : unpack_f16(u[i]);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
    }
};
template <int T>
__device__ __forceinline__ void load8(const void *p, float (&v)[8]) {
    Raw8<T> r;
    r.load(true, p);
    r.get(v);
}
template <int T>
__device__ __forceinline__ void store8(void *p, const float (&v)[8]) {
    if constexpr (T == kF32) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_16(T, v[0], v[1]), pack_16(T, v[2], v[3]), pack_16(T, v[4], v[5]),
                                                   pack_16(T, v[6], v[7]));
    }
}
template <int T> constexpr int kSize = T == kF32 ? 4 : 2;
template <int T>
__device__ __forceinline__ const void *element(const void *p, size_t i) { return static_cast<const char *>(p) + i * kSize<T>; }
template <int T>
__device__ __forceinline__ void *element(void *p, size_t i) { return static_cast<char *>(p) + i * kSize<T>; }

// Rows of slots j0 .. j0 + 7 of token t, -1 for none.
template <class A>
__device__ __forceinline__ void rows_of(const A &a, unsigned t, int j0, int (&p)[kTogether]) {
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
        p[j] = j0 + j < a.k ? row_of(a.place, (long long)t * a.k + j0 + j, a.n_rows) : -1;
}

// 2^e as described above.  448 = 1.75 * 2^8, so with |x| = 1.f * 2^p the
// exponent is p - 8 where 1.f <= 1.75 and p - 7 otherwise; powers of two make
// x / s exact, so a code is rounded once.
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t b = __float_as_uint(top);       // finite, not negative
    const int p = (int)(b >> 23) - 127;            // subnormals: below the least e all the same
    const int e = p - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, -126);
}
__device__ __forceinline__ float larger_finite(float top, float v) {
    const float m = fabsf(v);
    return m <= 3.402823466e38f ? fmaxf(top, m) : top;
}
// Of x / 2^e, times up = 2^-e; an infinity or NaN makes NaN (x * 0).
__device__ __forceinline__ uint32_t codes2(float x, float y, float up) {
    return pack_e4m3(fmaf(x, 0.f, x * up), fmaf(y, 0.f, y * up));
}

// Copies: 16 bytes a thread.
__global__ void __launch_bounds__(kRowThreads) dispatch_lines_kernel(const __grid_constant__ DispatchArgs a, int chunks,
                                                                     int lines, size_t stride_b) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    if (at.t >= (unsigned)a.tokens || at.u >= lines) return;
    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) + at.t * stride_b + at.u * 16ll);
    for (int j0 = 0; j0 < a.k; j0 += kTogether) {
        int p[kTogether];
        rows_of(a, at.t, j0, p);
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
            if (p[j] >= 0) reinterpret_cast<uint4 *>(a.rows)[(size_t)p[j] * lines + at.u] = v;
    }
}

// Copies of other rows: a thread's elements are 32 apart.
template <class Word>
__global__ void __launch_bounds__(kRowThreads) dispatch_words_kernel(const __grid_constant__ DispatchArgs a, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    const int c0 = (at.u & ~31) * 8 + (at.u & 31);
    if (at.t >= (unsigned)a.tokens || c0 >= a.width) return;
    const Word *x = static_cast<const Word *>(a.x) + at.t * a.x_stride;
    Word v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c0 + 32 * i < a.width) v[i] = x[c0 + 32 * i];
    for (int j = 0; j < a.k; ++j) {
        const int p = row_of(a.place, (long long)at.t * a.k + j, a.n_rows);
        if (p < 0) continue;
        Word *r = static_cast<Word *>(a.rows) + (size_t)p * a.width;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i < a.width) r[c0 + 32 * i] = v[i];
    }
}

// Codes: a thread takes 16 elements, eight threads a block of 128.
template <int T>
__global__ void __launch_bounds__(kRowThreads) dispatch_codes_kernel(const __grid_constant__ DispatchArgs a, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    const int nb = (a.width + kBlock - 1) / kBlock, c = at.u * 16;
    const bool here = at.t < (unsigned)a.tokens && c < a.width;
    float v[2][8] = {};
    int p[kTogether];
    if (here) {
        rows_of(a, at.t, 0, p);
        const size_t x0 = at.t * a.x_stride + c;
        load8<T>(element<T>(a.x, x0), v[0]);
        load8<T>(element<T>(a.x, x0 + 8), v[1]);
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = larger_finite(top, v[i >> 3][i & 7]);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (!here) return;
    const int ex = scale_exponent(top);            // -126 .. 120, so 2^ex and 2^-ex are normal
    const float s = __uint_as_float((uint32_t)(127 + ex) << 23), up = __uint_as_float((uint32_t)(127 - ex) << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *q = &v[i >> 1][4 * (i & 1)];
        w[i] = codes2(q[0], q[1], up) | codes2(q[2], q[3], up) << 16;
    }
    for (int j0 = 0;;) {
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            if (p[j] < 0) continue;
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.rows) + (size_t)p[j] * a.width + c) =
                make_uint4(w[0], w[1], w[2], w[3]);
            if ((at.u & 7) == 0) a.scales[(size_t)p[j] * nb + at.u / 8] = s;
        }
        if ((j0 += kTogether) >= a.k) break;
        rows_of(a, at.t, j0, p);
    }
}

// Codes of other rows: a warp takes a block of 128, a lane's four elements 32 apart.
template <int T>
__global__ void __launch_bounds__(kRowThreads) dispatch_codes_words_kernel(const __grid_constant__ DispatchArgs a, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    const int nb = (a.width + kBlock - 1) / kBlock, block = at.u >> 5, lane = at.u & 31, c = block * kBlock + lane;
    if (at.t >= (unsigned)a.tokens || block >= nb) return;         // the same for a warp
    const typename Elem<T>::Word *x = static_cast<const typename Elem<T>::Word *>(a.x) + at.t * a.x_stride;
    float v[4], top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = c + 32 * i < a.width ? Elem<T>::get(x[c + 32 * i]) : 0.f;
        top = larger_finite(top, v[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int ex = scale_exponent(top);
    const float s = __uint_as_float((uint32_t)(127 + ex) << 23), up = __uint_as_float((uint32_t)(127 - ex) << 23);
    const uint32_t w[2] = {codes2(v[0], v[1], up), codes2(v[2], v[3], up)};
    for (int j = 0; j < a.k; ++j) {
        const int p = row_of(a.place, (long long)at.t * a.k + j, a.n_rows);
        if (p < 0) continue;
        uint8_t *dst = static_cast<uint8_t *>(a.rows) + (size_t)p * a.width + c;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < a.width) dst[32 * i] = (uint8_t)(w[i >> 1] >> (8 * (i & 1)));
        if (lane == 0) a.scales[(size_t)p * nb + block] = s;
    }
}

template <int TO, int TY>
__global__ void __launch_bounds__(kRowThreads) combine_lines_kernel(const __grid_constant__ CombineArgs a, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    const int c = at.u * 8;
    if (at.t >= (unsigned)a.tokens || c >= a.width) return;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += kTogether) {
        int p[kTogether];
        float w[kTogether];
        Raw8<TY> y[kTogether];
        rows_of(a, at.t, j0, p);
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
            y[j].load(p[j] >= 0, element<TY>(a.y, (size_t)max(p[j], 0) * a.width + c));
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
            w[j] = p[j] < 0 ? 0.f : a.weights ? a.weights[(long long)at.t * a.k + j0 + j] : 1.f;
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {      // 0 * 0 for a slot without a row
            float v[8];
            y[j].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], v[i], sum[i]);
        }
    }
    store8<TO>(element<TO>(a.out, (size_t)at.t * a.width + c), sum);
}

template <int TO, int TY>
__global__ void __launch_bounds__(kRowThreads) combine_words_kernel(const __grid_constant__ CombineArgs a, int chunks) {
    griddep_wait();
    griddep_launch_dependents();
    const Place2 at = unit_of(chunks);
    const int c0 = (at.u & ~31) * 8 + (at.u & 31);
    if (at.t >= (unsigned)a.tokens || c0 >= a.width) return;
    float sum[8] = {};
    for (int j = 0; j < a.k; ++j) {
        const long long s = (long long)at.t * a.k + j;
        const int p = row_of(a.place, s, a.n_rows);
        if (p < 0) continue;
        const float w = a.weights ? a.weights[s] : 1.f;
        const typename Elem<TY>::Word *y = static_cast<const typename Elem<TY>::Word *>(a.y) + (size_t)p * a.width;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i < a.width) sum[i] = fmaf(w, Elem<TY>::get(y[c0 + 32 * i]), sum[i]);
    }
    typename Elem<TO>::Word *out = static_cast<typename Elem<TO>::Word *>(a.out) + (size_t)at.t * a.width;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c0 + 32 * i < a.width) out[c0 + 32 * i] = Elem<TO>::put(sum[i]);
}

// A token a block (threadIdx.y = 0) or a warp of it; the dot products of eight
// slots at a time are added up over the lanes, then over the warps in order.
template <int TD, int TY, bool VEC>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const __grid_constant__ CombineGradArgs a) {
    __shared__ float s_sum[kRowThreads / 32][kTogether];
    typedef typename Elem<TD>::Word WordD;
    typedef typename Elem<TY>::Word WordY;
    griddep_wait();
    griddep_launch_dependents();
    const long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.tokens) return;                     // whole warps: a warp's lanes share a token
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < a.k; j0 += kTogether) {
        int p[kTogether];
        float w[kTogether], sum[kTogether] = {};
        rows_of(a, (unsigned)t, j0, p);
#pragma unroll
        for (int j = 0; j < kTogether; ++j) w[j] = a.weights && p[j] >= 0 ? a.weights[t * a.k + j0 + j] : 1.f;
        for (int u = threadIdx.x;; u += blockDim.x) {
            const int c = VEC ? u * 8 : (u & ~31) * 8 + (u & 31);
            if (c >= a.width) break;
            float d[8] = {};
            if constexpr (VEC) {
                load8<TD>(element<TD>(a.dout, (size_t)t * a.width + c), d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + 32 * i < a.width) d[i] = Elem<TD>::get(static_cast<const WordD *>(a.dout)[(size_t)t * a.width + c + 32 * i]);
            }
            if constexpr (VEC) {
                Raw8<TY> y[kTogether];
#pragma unroll
                for (int j = 0; j < kTogether; ++j)
                    y[j].load(p[j] >= 0 && a.dweights, element<TY>(a.y, (size_t)max(p[j], 0) * a.width + c));
#pragma unroll
                for (int j = 0; j < kTogether; ++j) {
                    if (p[j] < 0) continue;
                    float v[8], g[8];
                    y[j].get(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sum[j] = fmaf(d[i], v[i], sum[j]);
                        g[i] = w[j] * d[i];
                    }
                    if (a.dy) store8<TY>(element<TY>(a.dy, (size_t)p[j] * a.width + c), g);
                }
            } else {
                WordY y[kTogether][8];
#pragma unroll
                for (int j = 0; j < kTogether; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool in = p[j] >= 0 && a.dweights && c + 32 * i < a.width;
                        y[j][i] = load_if(in, static_cast<const WordY *>(a.y) + (size_t)max(p[j], 0) * a.width + c + 32 * i);
                    }
#pragma unroll
                for (int j = 0; j < kTogether; ++j) {
                    if (p[j] < 0) continue;
                    WordY *dy = static_cast<WordY *>(a.dy) + (size_t)p[j] * a.width + c;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sum[j] = fmaf(d[i], Elem<TY>::get(y[j][i]), sum[j]);       // zeros past the row's end
                        if (a.dy && c + 32 * i < a.width) dy[32 * i] = Elem<TY>::put(w[j] * d[i]);
                    }
                }
            }
        }
        if (!a.dweights) continue;
        const float all = warp_reduce_scatter<kTogether>(sum, lane);
        const int j = reduce_scatter_index<kTogether>(lane);
        if (blockDim.y > 1) {                      // a warp a token
            if ((lane & 3) == 0 && j0 + j < a.k) a.dweights[t * a.k + j0 + j] = all;
            continue;
        }
        if ((lane & 3) == 0) s_sum[threadIdx.x >> 5][j] = all;
        __syncthreads();
        if (threadIdx.x < kTogether && j0 + (int)threadIdx.x < a.k) {
            float v = 0.f;
            for (int i = 0; i < warps; ++i) v += s_sum[i][threadIdx.x];
            a.dweights[t * a.k + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

template <int A, class F>
int by_type2(int b, F f) {
    switch (b) {
        case kF32: return f(std::integral_constant<int, A>(), std::integral_constant<int, kF32>());
        case kBf16: return f(std::integral_constant<int, A>(), std::integral_constant<int, kBf16>());
        default: return f(std::integral_constant<int, A>(), std::integral_constant<int, kF16>());
    }
}
template <class F>
int by_types(int a, int b, F f) {
    switch (a) {
        case kF32: return by_type2<kF32>(b, f);
        case kBf16: return by_type2<kBf16>(b, f);
        default: return by_type2<kF16>(b, f);
    }
}

inline bool lines16(const void *p) { return (uintptr_t)p % 16 == 0; }
inline int size_of(int type) { return type == kF32 ? 4 : 2; }

template <int T>
int launch_codes(const DispatchArgs &a, cudaStream_t st) {
    const bool vec = a.width % 16 == 0 && a.x_stride * kSize<T> % 16 == 0 && lines16(a.x) && lines16(a.rows);
    const int units = (a.width + kBlock - 1) / kBlock * (vec ? 8 : 32);   // whole blocks: their threads meet
    const RowGrid g(a.tokens, units, threads_for((long long)a.tokens * units), vec ? 8 : 32);
    return vec ? launch_pdl("qg_moe_dispatch", dispatch_codes_kernel<T>, g.blocks, g.block(), 0, st, a, g.chunks)
               : launch_pdl("qg_moe_dispatch", dispatch_codes_words_kernel<T>, g.blocks, g.block(), 0, st, a, g.chunks);
}

}  // namespace

int run_moe_dispatch(const DispatchArgs &a, int x_type, bool codes, cudaStream_t st) {
    const char *what = "qg_moe_dispatch";
    if (codes) return x_type == kF32 ? launch_codes<kF32>(a, st) : x_type == kBf16 ? launch_codes<kBf16>(a, st) : launch_codes<kF16>(a, st);
    const size_t esz = size_of(x_type), row = (size_t)a.width * esz;
    if (row % 16 == 0 && a.x_stride * esz % 16 == 0 && lines16(a.x) && lines16(a.rows)) {
        const RowGrid g(a.tokens, (int)(row / 16), threads_for((long long)a.tokens * (row / 16)), 8);
        return launch_pdl(what, dispatch_lines_kernel, g.blocks, g.block(), 0, st, a, g.chunks, g.units, a.x_stride * esz);
    }
    const int units = (a.width + 255) / 256 * 32;              // 32 threads take 256 elements
    const RowGrid g(a.tokens, units, threads_for((long long)a.tokens * units), 32);
    return esz == 4 ? launch_pdl(what, dispatch_words_kernel<uint32_t>, g.blocks, g.block(), 0, st, a, g.chunks)
                    : launch_pdl(what, dispatch_words_kernel<uint16_t>, g.blocks, g.block(), 0, st, a, g.chunks);
}

int run_moe_combine(const CombineArgs &a, int out_type, int y_type, cudaStream_t st) {
    const char *what = "qg_moe_combine";
    const bool vec = a.width % 8 == 0 && lines16(a.out) && lines16(a.y);
    const int units = vec ? a.width / 8 : (a.width + 255) / 256 * 32;
    const RowGrid g(a.tokens, units, threads_for((long long)a.tokens * units), vec ? 8 : 32);
    return by_types(out_type, y_type, [&](auto to, auto ty) {
        constexpr int TO = decltype(to)::value, TY = decltype(ty)::value;
        return vec ? launch_pdl(what, combine_lines_kernel<TO, TY>, g.blocks, g.block(), 0, st, a, g.chunks)
                   : launch_pdl(what, combine_words_kernel<TO, TY>, g.blocks, g.block(), 0, st, a, g.chunks);
    });
}

int run_moe_combine_grad(const CombineGradArgs &a, int dout_type, int y_type, cudaStream_t st) {
    const char *what = "qg_moe_combine_grad";
    const bool vec = a.width % 8 == 0 && lines16(a.dout) && lines16(a.y) && lines16(a.dy);
    const int units = vec ? a.width / 8 : (a.width + 255) / 256 * 32;
    // a warp a token where a row is little more than a warp's units, else a block
    const bool warp = units <= 64;
    const int threads = units >= 256 ? 256 : (units + 31) / 32 * 32;
    const dim3 block = warp ? dim3(32, 4) : dim3(threads, 1);
    const unsigned blocks = warp ? ((unsigned)a.tokens + 3) / 4 : (unsigned)a.tokens;
    return by_types(dout_type, y_type, [&](auto td, auto ty) {
        constexpr int TD = decltype(td)::value, TY = decltype(ty)::value;
        return vec ? launch_pdl(what, combine_grad_kernel<TD, TY, true>, blocks, block, 0, st, a)
                   : launch_pdl(what, combine_grad_kernel<TD, TY, false>, blocks, block, 0, st, a);
    });
}

}  // namespace qg
