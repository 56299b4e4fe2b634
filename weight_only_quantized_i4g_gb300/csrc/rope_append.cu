// rope_append.cu -- rotary positions on q and k and the write of k and v into
// the paged cache (qg_rope_append).
//
// Pair j of a q or k head, (x_j, x_{j+r/2}) or (x_{2j}, x_{2j+1}), turns by
// a_j = pos[axis_j] * inv_freq_j:
//   x' = x cos a - y sin a,   y' = y cos a + x sin a.
// Every element is read once and written once, so the call is bound by bytes
// (by the launch and two dependent loads, positions then table, for a few
// tokens).  One block takes one token and a group of heads: its cosines and
// sines are computed once into shared memory and serve all heads of the group.
#include "kv_cache.cuh"

namespace qg {

namespace {

constexpr int kRopeThreads = 256;

// Four consecutive elements of a row as f32.
template <int IN>
__device__ __forceinline__ void load4(const void *p, size_t i, float *x) {
    if (IN == kF32) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
        const float2 a = IN == kBf16 ? unpack_bf16(v.x) : unpack_f16(v.x);
        const float2 b = IN == kBf16 ? unpack_bf16(v.y) : unpack_f16(v.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
}
template <int IN>
__device__ __forceinline__ float load1(const void *p, size_t i) {
    if (IN == kF32) return static_cast<const float *>(p)[i];
    const uint16_t b = static_cast<const uint16_t *>(p)[i];
    return IN == kBf16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Stores elements of a head at `base` (its element 0): 16-bit values, or e4m3
// codes of x / scale (one IEEE division, then round to nearest even).
__device__ __forceinline__ void store4(char *base, int type, int d, const float *x, float scale) {
    if (type == kE4m3) {
        const uint32_t lo = pack_e4m3(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale));
        const uint32_t hi = pack_e4m3(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale));
        *reinterpret_cast<uint32_t *>(base + d) = lo | (hi << 16);
    } else {
        *reinterpret_cast<uint2 *>(base + 2 * d) = make_uint2(pack_16(type, x[0], x[1]), pack_16(type, x[2], x[3]));
    }
}
__device__ __forceinline__ void store1(char *base, int type, int d, float x, float scale) {
    if (type == kE4m3) {
        // the code travels in a 32-bit register: see pack_e4m3
        *reinterpret_cast<uint8_t *>(base + d) = (uint8_t)(pack_e4m3(__fdiv_rn(x, scale), 0.f) & 0xFFu);
    } else {
        *reinterpret_cast<uint16_t *>(base + 2 * d) = (uint16_t)(pack_16(type, x, 0.f) & 0xFFFFu);
    }
}

// VEC: rows, sizes and pointers allow four elements per access; a thread then
// takes units of 8 elements of a head (two such groups), otherwise of a pair.
// Eight blocks an SM: a block is a chain of waits, and only other blocks fill
// them (6001 tokens, 56 heads: 40.7 us, 93% of the measured copy rate; 43.6 with
// six blocks, 50 with four, where a thread kept its pairs' cosines in registers).
template <int IN, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_append_kernel(const __grid_constant__ RopeArgs a,
                                                                   int heads_per_block, FastDiv units_div) {
    __shared__ float s_cos[kMaxPairs], s_sin[kMaxPairs];
    griddep_launch_dependents();
    griddep_wait();
    const int t = blockIdx.x;
    const int D = a.c.dim, half = a.rotary >> 1;
    const int heads = a.n_q_heads + 2 * a.c.n_heads;
    const int h0 = blockIdx.y * heads_per_block;
    const int h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;

    // units of work: kUnit elements of a head, two halves of kHalf
    constexpr int kUnit = VEC ? 8 : 2, kHalf = kUnit / 2;
    const size_t row = (size_t)t * a.qkv_stride;
    const int units = D / kUnit, work = (h1 - h0) * units;
    struct Unit { float x[kHalf], y[kHalf]; };
    // where unit u's halves start, and the first pair it holds (-1: none)
    auto halves = [&](int u, int *d0, int *d1) {
        *d0 = kUnit * u, *d1 = *d0 + kHalf;
        if (*d0 >= a.rotary) return -1;
        const int j = kHalf * u;
        if (!a.interleaved) *d0 = j, *d1 = j + half;
        return j;
    };
    auto load = [&](int i) {
        Unit v;
        const int hh = quotient(i, units_div), u = i - hh * units;
        const size_t at = row + (size_t)(h0 + hh) * D;
        int d0, d1;
        halves(u, &d0, &d1);
        if constexpr (VEC) {
            load4<IN>(a.qkv, at + d0, v.x);
            load4<IN>(a.qkv, at + d1, v.y);
        } else {
            v.x[0] = load1<IN>(a.qkv, at + d0), v.y[0] = load1<IN>(a.qkv, at + d1);
        }
        return v;
    };
    // the first unit is on its way while the angles and the slot are found
    Unit next = {};
    if ((int)threadIdx.x < work) next = load(threadIdx.x);

    // The angle is formed and reduced to one turn in 64 bits: in binary32 it
    // would be off by pos * 2^-24 radians, 0.06 at position 2^20.
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        const double x = (double)a.pos[(size_t)t * a.n_axes + a.axis[j]] * (double)a.inv_freq[j] *
                         0.15915494309189533577;   // 1 / (2 pi): turns
        sincospif(2.0f * (float)(x - rint(x)), &s_sin[j], &s_cos[j]);
    }

    // where this token's k and v go
    SlotRef ref{-1, 0};
    if (h1 > a.n_q_heads) {
        const int b = a.seq[t], slot = a.slot[t];
        if (slot >= 0) {
            if ((unsigned)b < (unsigned)a.n_seq && slot < (long long)a.table_stride * a.c.page)
                ref = find_slot(a.c, a.table + (size_t)b * a.table_stride, slot);
            if (ref.page < 0 && threadIdx.x == 0) raise_device_error(a.err, kErrPage);
        }
    }
    __syncthreads();

    for (int i = threadIdx.x; i < work; i += kRopeThreads) {
        Unit v = next;
        if (i + kRopeThreads < work) next = load(i + kRopeThreads);
        const int hh = quotient(i, units_div), u = i - hh * units, h = h0 + hh;
        const bool is_q = h < a.n_q_heads, is_v = h >= a.n_q_heads + a.c.n_heads;
        int d0, d1;
        const int j = halves(u, &d0, &d1);
        if (j >= 0 && !is_v) {
#pragma unroll
            for (int e = 0; e < kHalf; ++e) {
                // pair e is (x[e], y[e]), or elements 2e, 2e + 1 of the unit
                const int at = 2 * e % kHalf;
                const bool split = !VEC || !a.interleaved, low = 2 * e < kHalf;
                float &p = split ? v.x[e] : low ? v.x[at] : v.y[at];
                float &q = split ? v.y[e] : low ? v.x[(at + 1) % kHalf] : v.y[(at + 1) % kHalf];
                const float p0 = p, cs = s_cos[j + e], sn = s_sin[j + e];
                p = p0 * cs - q * sn;
                q = q * cs + p0 * sn;
            }
        }
        char *base;
        float scale = 1.f;
        int type = a.c.type;
        if (is_q) {
            base = static_cast<char *>(a.q) + ((size_t)t * a.n_q_heads + h) * D * 2;
            type = a.q_type;
        } else {
            if (ref.page < 0) continue;
            const int kh = h - a.n_q_heads - (is_v ? a.c.n_heads : 0);
            base = (is_v ? a.c.v : a.c.k) + slot_bytes(a.c, ref, kh);
            if (type == kE4m3) scale = *((is_v ? a.c.v_scale : a.c.k_scale) + kh);
            if (!is_v && u == 0 && a.c.weight) a.c.weight[slot_weight(a.c, ref, kh)] = 0.f;
        }
        if constexpr (VEC) {
            store4(base, type, d0, v.x, scale);
            store4(base, type, d1, v.y, scale);
        } else {
            store1(base, type, d0, v.x[0], scale);
            store1(base, type, d1, v.y[0], scale);
        }
    }
}

template <int IN>
int launch(const RopeArgs &a, bool vec, cudaStream_t st) {
    const int heads = a.n_q_heads + 2 * a.c.n_heads;
    // a block per token and as many heads as leave two blocks for every SM
    long long groups = (2LL * num_sms() + a.T - 1) / a.T;
    if (groups > heads) groups = heads;
    const int per = (int)((heads + groups - 1) / groups);
    const dim3 grid(a.T, (heads + per - 1) / per);
    const FastDiv units = fast_div(a.c.dim / (vec ? 8 : 2));
    return vec ? launch_pdl("qg_rope_append", rope_append_kernel<IN, true>, grid, kRopeThreads, 0, st, a, per, units)
               : launch_pdl("qg_rope_append", rope_append_kernel<IN, false>, grid, kRopeThreads, 0, st, a, per, units);
}

}  // namespace

int run_rope_append(const RopeArgs &a, int qkv_type, cudaStream_t st) {
    const size_t esz = qkv_type == kF32 ? 4 : 2;
    const bool vec = a.rotary % 8 == 0 && a.qkv_stride % 4 == 0 && (uintptr_t)a.qkv % (4 * esz) == 0 &&
                     (uintptr_t)a.q % 8 == 0;
    switch (qkv_type) {
        case kF32: return launch<kF32>(a, vec, st);
        case kBf16: return launch<kBf16>(a, vec, st);
        default: return launch<kF16>(a, vec, st);
    }
}

}  // namespace qg
