// moe_rows.cu -- token rows to their experts and back (qg_moe_dispatch,
// qg_moe_combine, qg_moe_combine_grad).
//
//   dispatch  rows[place[t,j]] = x[t], or e4m3(x[t] / s) with s = 2^e for each
//             128 elements, e the least integer >= -126 for which the block's
//             largest finite |x| is at most 448 * 2^e
//   combine   out[t] = sum_j w[t,j] y[place[t,j]], f32, j ascending
//   gradient  dy[place[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[place[t,j]]>
#include "moe.cuh"

namespace qg {
namespace {

constexpr int kRowThreads = 256;
constexpr int kBlock = 128;      // elements of one scale

// 2^e as described above.  448 = 1.75 * 2^8, so with |x| = 1.f * 2^p the
// exponent is p - 8 where 1.f <= 1.75 and p - 7 otherwise; powers of two make
// x / s exact, so a code is rounded once.
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t b = __float_as_uint(top);       // finite, not negative
    const int p = (int)(b >> 23) - 127;            // subnormals: below the least e all the same
    const int e = p - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, -126);
}

template <int T>
__global__ void __launch_bounds__(kRowThreads) dispatch_copy_kernel(const DispatchArgs a) {
    typedef typename Elem<T>::Word Word;
    griddep_wait();
    griddep_launch_dependents();
    const long long n = (long long)a.tokens * a.width;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const long long t = i / a.width;
    const int c = (int)(i - t * a.width);
    const Word v = static_cast<const Word *>(a.x)[t * a.x_stride + c];
    for (int j = 0; j < a.k; ++j) {
        const int p = row_of(a.place, t * a.k + j, a.n_rows);
        if (p >= 0) static_cast<Word *>(a.rows)[(size_t)p * a.width + c] = v;
    }
}

// A warp takes one block of 128 elements of one token.
template <int T>
__global__ void __launch_bounds__(kRowThreads) dispatch_codes_kernel(const DispatchArgs a) {
    typedef typename Elem<T>::Word Word;
    griddep_wait();
    griddep_launch_dependents();
    const int nb = (a.width + kBlock - 1) / kBlock, lane = threadIdx.x & 31;
    const long long g = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (g >= (long long)a.tokens * nb) return;
    const long long t = g / nb;
    const int b = (int)(g - t * nb), c = b * kBlock + lane * 4;
    float v[4], top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = c + e < a.width ? Elem<T>::get(static_cast<const Word *>(a.x)[t * a.x_stride + c + e]) : 0.f;
        const float m = fabsf(v[e]);
        top = m <= 3.402823466e38f ? fmaxf(top, m) : top;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int ex = scale_exponent(top);
    // 2^-ex in two factors, as 2^126 * 448 and its like are no f32
    const float up = __uint_as_float((uint32_t)(127 - ex / 2) << 23), up2 = __uint_as_float((uint32_t)(127 - (ex - ex / 2)) << 23);
    const float nan = __uint_as_float(0x7FC00000u);
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float y = fabsf(v[e]) <= 3.402823466e38f ? v[e] * up * up2 : nan;
        code[e] = pack_e4m3(y, 0.f) & 0xFFu;
    }
    const float s = __uint_as_float((uint32_t)(ex + 127) << 23);
    for (int j = 0; j < a.k; ++j) {
        const int p = row_of(a.place, t * a.k + j, a.n_rows);
        if (p < 0) continue;
        uint8_t *dst = static_cast<uint8_t *>(a.rows) + (size_t)p * a.width + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < a.width) dst[e] = (uint8_t)code[e];
        if (lane == 0) a.scales[(size_t)p * nb + b] = s;
    }
}

template <int TO, int TY>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const CombineArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const long long n = (long long)a.tokens * a.width;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const long long t = i / a.width;
    const int c = (int)(i - t * a.width);
    float sum = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const long long s = t * a.k + j;
        const int p = row_of(a.place, s, a.n_rows);
        if (p < 0) continue;
        const float y = Elem<TY>::get(static_cast<const typename Elem<TY>::Word *>(a.y)[(size_t)p * a.width + c]);
        sum = a.weights ? fmaf(a.weights[s], y, sum) : sum + y;
    }
    static_cast<typename Elem<TO>::Word *>(a.out)[i] = Elem<TO>::put(sum);
}

template <int TD, int TY>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const CombineGradArgs a) {
    __shared__ float s_sum[kRowThreads / 32];
    typedef typename Elem<TY>::Word Word;
    griddep_wait();
    griddep_launch_dependents();
    const long long t = blockIdx.x;
    const typename Elem<TD>::Word *d = static_cast<const typename Elem<TD>::Word *>(a.dout) + (size_t)t * a.width;
    for (int j = 0; j < a.k; ++j) {
        const long long s = t * a.k + j;
        const int p = row_of(a.place, s, a.n_rows);
        const float w = a.weights ? a.weights[s] : 1.f;
        float sum = 0.f;
        if (p >= 0)
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                const float g = Elem<TD>::get(d[c]);
                if (a.dweights) sum = fmaf(g, Elem<TY>::get(static_cast<const Word *>(a.y)[(size_t)p * a.width + c]), sum);
                if (a.dy) static_cast<Word *>(a.dy)[(size_t)p * a.width + c] = Elem<TY>::put(w * g);
            }
        if (!a.dweights) continue;
        sum = warp_sum(sum);
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            float all = 0.f;
            for (int i = 0; i < kRowThreads / 32; ++i) all += s_sum[i];
            a.dweights[s] = all;
        }
        __syncthreads();
    }
}

inline unsigned blocks_for(long long items) { return (unsigned)((items + kRowThreads - 1) / kRowThreads); }

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

}  // namespace

int run_moe_dispatch(const DispatchArgs &a, int x_type, bool codes, cudaStream_t st) {
    const char *what = "qg_moe_dispatch";
    if (codes) {
        const unsigned n = blocks_for((long long)a.tokens * ((a.width + kBlock - 1) / kBlock) * 32);
        switch (x_type) {
            case kF32: return launch_pdl(what, dispatch_codes_kernel<kF32>, n, kRowThreads, 0, st, a);
            case kBf16: return launch_pdl(what, dispatch_codes_kernel<kBf16>, n, kRowThreads, 0, st, a);
            default: return launch_pdl(what, dispatch_codes_kernel<kF16>, n, kRowThreads, 0, st, a);
        }
    }
    const unsigned n = blocks_for((long long)a.tokens * a.width);
    return x_type == kF32 ? launch_pdl(what, dispatch_copy_kernel<kF32>, n, kRowThreads, 0, st, a)
                          : launch_pdl(what, dispatch_copy_kernel<kBf16>, n, kRowThreads, 0, st, a);
}

int run_moe_combine(const CombineArgs &a, int out_type, int y_type, cudaStream_t st) {
    const unsigned n = blocks_for((long long)a.tokens * a.width);
    return by_types(out_type, y_type, [&](auto to, auto ty) {
        return launch_pdl("qg_moe_combine", combine_kernel<decltype(to)::value, decltype(ty)::value>, n, kRowThreads, 0,
                          st, a);
    });
}

int run_moe_combine_grad(const CombineGradArgs &a, int dout_type, int y_type, cudaStream_t st) {
    return by_types(dout_type, y_type, [&](auto td, auto ty) {
        return launch_pdl("qg_moe_combine_grad", combine_grad_kernel<decltype(td)::value, decltype(ty)::value>,
                          (unsigned)a.tokens, kRowThreads, 0, st, a);
    });
}

}  // namespace qg
