// gemm_e4m3.cu -- products of e4m3 activations with e4m3 weights (qgemm_e4m3,
// qgemm_e4m3_moe):
//
//   Y[m, o] = sum_b xs[m, b] ws[o/128, b] sum_{i in block b} X[m, i] W[o, i]
//
// with a scale for each token and 128 elements and one for each 128 x 128
// weights; rows [offsets[e], offsets[e+1]) use expert e's weights.
//
// Rows of whole 16-byte lines run on the tensor cores (gemm_e4m3_tc.cuh);
// this file has the choice between their kernels, and the general kernel, for
// every shape and alignment: 64 x 64 outputs a block, K in steps of 32, codes
// widened to f32 in shared memory, f32 sums of a 128-block scaled when it
// ends.  A block of rows that several experts share goes over each of them.
#include <algorithm>

#include "gemm_e4m3_tc.cuh"

namespace qg {
namespace {

constexpr int kGT = 64, kGK = 32;

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)c));
    return f16_bits_to_f32((uint16_t)h2);
}

__device__ __forceinline__ void store_y(void *Y, int type, size_t at, float v) {
    if (type == kF32) static_cast<float *>(Y)[at] = v;
    else if (type == kBf16) static_cast<uint16_t *>(Y)[at] = Elem<kBf16>::put(v);
    else static_cast<uint16_t *>(Y)[at] = Elem<kF16>::put(v);
}

template <class SC>
__global__ void __launch_bounds__(256) gemm_e4m3_general_kernel(const E4m3Args a) {
    __shared__ float Ws[kGK][kGT + 1];   // [k][o]
    __shared__ float Xs[kGK][kGT + 1];   // [k][m]
    griddep_wait();
    griddep_launch_dependents();
    const int o0 = blockIdx.x * kGT, m0 = blockIdx.y * kGT;
    const int nb = (a.I + 127) / 128, nbo = (a.O + 127) / 128;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;   // 16 x 16 threads, 4 x 4 each
    int to = a.offsets ? held_row(a.offsets[0], a.M) : a.M;
    for (int g = 0; g < a.experts; ++g) {
        int from = 0;
        if (a.offsets) next_rows(a.offsets, g, a.M, &from, &to, threadIdx.x == 0 ? a.err : nullptr);
        if (to <= m0 || from >= m0 + kGT || to <= from) continue;      // the same for the whole block
        const uint8_t *w = a.w + (size_t)g * a.O * a.I;
        const typename SC::T *ws = static_cast<const typename SC::T *>(a.w_scale) + (size_t)g * nbo * nb;
        float sum[4][4] = {}, acc[4][4] = {};
        for (int k0 = 0; k0 < a.I; k0 += kGK) {
            for (int e = threadIdx.x; e < kGK * kGT; e += blockDim.x) {
                const int kk = e % kGK, r = e / kGK, i = k0 + kk, o = o0 + r, m = m0 + r;
                Ws[kk][r] = o < a.O && i < a.I ? e4m3_to_f32(w[(size_t)o * a.I + i]) : 0.f;
                Xs[kk][r] = m >= from && m < to && i < a.I ? e4m3_to_f32(a.X[(size_t)m * a.I + i]) : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int kk = 0; kk < kGK; ++kk) {
                float x[4], v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    x[t] = Xs[kk][ty * 4 + t];
                    v[t] = Ws[kk][tx * 4 + t];
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(x[r], v[c], acc[r][c]);
            }
            __syncthreads();
            if ((k0 + kGK) % 128 && k0 + kGK < a.I) continue;
            const int b = k0 / 128;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = m0 + ty * 4 + r;
                const float xs = m >= from && m < to ? a.x_scale[(size_t)m * nb + b] : 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int o = o0 + tx * 4 + c;
                    if (o < a.O) sum[r][c] = fmaf(acc[r][c], xs * SC::get(ws, (size_t)(o / 128) * nb + b), sum[r][c]);
                    acc[r][c] = 0.f;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + ty * 4 + r;
            if (m < from || m >= to) continue;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int o = o0 + tx * 4 + c;
                if (o < a.O) store_y(a.Y, a.y_type, (size_t)m * a.O + o, sum[r][c]);
            }
        }
    }
}

// A launch for each kMaxExperts experts, planned with their share of the rows.
int run_tc(const char *what, const E4m3Args &all, cudaStream_t st) {
    if (!tc::encode_fn()) QG_REFUSE(kECuda, "%s: cuTensorMapEncodeTiled is not available from the driver", what);
    const int KB = (all.I + 127) / 128, NB = (all.O + 127) / 128;
    for (int e0 = 0; e0 < all.experts; e0 += e8::kMaxExperts) {
        E4m3Args g = all;
        g.experts = std::min(all.experts - e0, e8::kMaxExperts);
        g.w = all.w + (size_t)e0 * all.O * all.I;
        g.w_scale = static_cast<const char *>(all.w_scale) + (size_t)e0 * NB * KB * (all.w_power ? 1 : 4);
        if (all.offsets) g.offsets = all.offsets + e0;
        const int rows = (int)(((long long)all.M * g.experts + all.experts - 1) / all.experts);
        const e8::Args8 a{g.Y, g.y_type, g.x_scale, g.w_scale, g.offsets, e0, g.experts, g.M, g.O, KB, NB, 0, g.err};
        const e8::FewPlan few = e8::plan_few(rows, g.I, g.O, g.experts);
        const e8::ManyPlan many = e8::plan_many(rows, g.I, g.O, g.experts);
        const int rc = many.cost < few.cost ? e8::launch_many(what, many, g, a, st) : e8::launch_few(what, few, g, a, st);
        if (rc != kOk) return rc;
    }
    return kOk;
}

// TMA's rules for the rows, and 32-bit rows and tiles of a launch.
bool tc_takes(const E4m3Args &a) {
    const long long experts = std::min(a.experts, e8::kMaxExperts), wrows = experts * a.O;
    const long long tiles = ((long long)a.M / 32 + experts) * ((a.O + 127) / 128);
    return a.I % 16 == 0 && (uintptr_t)a.X % 16 == 0 && (uintptr_t)a.w % 16 == 0 && wrows < (1ll << 31) - 256 &&
           tiles < (1ll << 31) - 65536;
}

}  // namespace

int run_gemm_e4m3(const E4m3Args &a, cudaStream_t st) {
    const char *what = a.offsets ? "qgemm_e4m3_moe" : "qgemm_e4m3";
    if (tc_takes(a)) return run_tc(what, a, st);
    const dim3 grid((a.O + kGT - 1) / kGT, (a.M + kGT - 1) / kGT);
    return a.w_power ? launch_pdl(what, gemm_e4m3_general_kernel<ScaleE8M0>, grid, 256, 0, st, a)
                     : launch_pdl(what, gemm_e4m3_general_kernel<ScaleF32>, grid, 256, 0, st, a);
}

}  // namespace qg
