// attn_paged.cu -- attention of a few new tokens over a paged key-value cache
// (qattn_paged).
//
// Row (b, s, h) sees the slots t < len_b - S + 1 + s:
//   z_t = scale q . k_t,   o = sum_t exp(z_t - lse) v_t,   lse = log sum_t exp(z_t).
// One block a row; its warps take every fourth slot, keep a running maximum
// and sum (online softmax) and are joined at the end.
#include "kv_cache.cuh"

namespace qg {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPerLane = 8;    // head elements a lane holds (dim <= 256)

__device__ __forceinline__ float cache_value(const char *p, int type, int d) {
    if (type == kBf16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[d]);
    if (type == kF16) return f16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[d]);
    return unpack_f16(e4m3x2_to_f16x2((uint32_t)reinterpret_cast<const uint8_t *>(p)[d])).x;
}

__global__ void __launch_bounds__(32 * kWarps) attn_row_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][256];
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x % a.n_q_heads, bs = blockIdx.x / a.n_q_heads;
    const int s = bs % a.S, b = bs / a.S, kh = h / a.group;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.c.dim;
    const int len = seq_len(a.lens, b, a.max_len, threadIdx.x == 0 ? a.err : nullptr);
    const int limit = len - a.S + 1 + s;
    const int *row = a.table + (size_t)b * a.table_stride;
    const char *q = static_cast<const char *>(a.q) + 2 * ((size_t)bs * a.q_stride + (size_t)h * D);
    const float ks = a.c.type == kE4m3 ? __ldg(a.c.k_scale + kh) : 1.f;
    const float vs = a.c.type == kE4m3 ? __ldg(a.c.v_scale + kh) : 1.f;
    float qv[kMaxPerLane], o[kMaxPerLane], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
        qv[i] = 32 * i + lane < D ? cache_value(q, a.q_type, 32 * i + lane) : 0.f;
        o[i] = 0.f;
    }
    for (int t = warp; t < limit; t += kWarps) {
        const SlotRef r = find_slot(a.c, row, t);
        float z = NAN;
        long long at = 0;
        if (r.page >= 0) {
            at = slot_bytes(a.c, r, kh);
            z = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxPerLane; ++i)
                if (32 * i + lane < D) z = fmaf(qv[i], cache_value(a.c.k + at, a.c.type, 32 * i + lane), z);
            z = warp_sum(z) * ks * a.scale;
        } else if (lane == 0) {
            raise_device_error(a.err, kErrPage);
        }
        const float mn = fmaxf(m, z), ref = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - ref), p = expf(z - ref);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < kMaxPerLane; ++i)
            if (32 * i + lane < D)
                o[i] = o[i] * f + p * (r.page >= 0 ? cache_value(a.c.v + at, a.c.type, 32 * i + lane) : 0.f);
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) s_o[warp][32 * i + lane] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < kWarps; ++w) ll += s_l[w] * expf(s_m[w] - ref);
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += s_o[w][d] * expf(s_m[w] - ref);
        x = ll == 0.f ? 0.f : x * vs / ll;
        const size_t at = ((size_t)bs * a.n_q_heads + h) * D + d;
        if (a.o_type == kF32) static_cast<float *>(a.o)[at] = x;
        else static_cast<uint16_t *>(a.o)[at] = (uint16_t)(pack_16(a.o_type, x, 0.f) & 0xFFFFu);
    }
    if (threadIdx.x == 0) a.lse[(size_t)bs * a.n_q_heads + h] = ll == 0.f ? -INFINITY : ref + logf(ll);
}

// weight[t] += sum over the head group's rows of exp(z_t - lse); one warp a slot.
__global__ void __launch_bounds__(32 * kWarps) attn_weight_kernel(const __grid_constant__ AttnArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int kh = blockIdx.x % a.c.n_heads, b = blockIdx.x / a.c.n_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.c.dim;
    const int len = seq_len(a.lens, b, a.max_len, nullptr);
    const int *row = a.table + (size_t)b * a.table_stride;
    const float ks = a.c.type == kE4m3 ? __ldg(a.c.k_scale + kh) : 1.f;
    for (int t = blockIdx.y * kWarps + warp; t < len; t += gridDim.y * kWarps) {
        const SlotRef r = find_slot(a.c, row, t);
        if (r.page < 0) continue;
        const char *k = a.c.k + slot_bytes(a.c, r, kh);
        float sum = 0.f;
        for (int s = 0; s < a.S; ++s) {
            if (t >= len - a.S + 1 + s) continue;
            for (int g = 0; g < a.group; ++g) {
                const size_t bs = (size_t)b * a.S + s;
                const int h = kh * a.group + g;
                const char *q = static_cast<const char *>(a.q) + 2 * (bs * a.q_stride + (size_t)h * D);
                float z = 0.f;
                for (int d = lane; d < D; d += 32) z = fmaf(cache_value(q, a.q_type, d), cache_value(k, a.c.type, d), z);
                z = warp_sum(z) * ks * a.scale;
                const float lse = a.lse[bs * a.n_q_heads + h];
                sum += lse == -INFINITY ? 0.f : expf(z - lse);
            }
        }
        if (lane == 0) a.c.weight[slot_weight(a.c, r, kh)] += sum;
    }
}

size_t lse_bytes(int n_seq, int S, int n_q_heads) {
    return (((size_t)n_seq * S * n_q_heads * 4) + 255) & ~(size_t)255;
}

}  // namespace

size_t ws_attn_paged(const KvView &, int n_seq, int, int S, int n_q_heads, int) {
    return lse_bytes(n_seq, S, n_q_heads);   // the row statistics, where the caller wants none
}

int run_attn_paged(const AttnArgs &args, void *ws, cudaStream_t st) {
    AttnArgs a = args;
    if (!a.lse) a.lse = static_cast<float *>(ws);
    int rc = launch_pdl("qattn_paged", attn_row_kernel, dim3(a.n_seq * a.S * a.n_q_heads), 32 * kWarps, 0, st, a);
    if (rc != kOk || !a.accumulate || a.max_len == 0) return rc;
    int y = (a.max_len + 63) / 64;
    if (y > 1024) y = 1024;
    return launch_pdl("qattn_paged", attn_weight_kernel, dim3(a.n_seq * a.c.n_heads, y), 32 * kWarps, 0, st, a);
}

}  // namespace qg
