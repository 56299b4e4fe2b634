// kv_evict.cu -- eviction by accumulated attention weight (qg_kv_evict).
//
// Per sequence and head, of L slots N = min(L, budget) are kept: the first
// `sinks`, the last `recent` and, of the slots between them, those of largest
// weight (equal weights: the lower slot).  A select kernel finds them with a
// radix select over order-preserving 32-bit keys and writes their slots in
// order; a move kernel copies K, V and weight of the kept slots to the new
// pages.  Selection reads 4 bytes a slot; the copies, 4 D bytes a kept slot
// and 16-bit element each way, are the bulk and bound by HBM.
#include "kv_cache.cuh"

namespace qg {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// Order of weights: every NaN above +inf, -0 equal to +0; larger key = larger weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ int s_hist[2048];
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    __shared__ int s_digit, s_need;
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x % a.c.n_heads, b = blockIdx.x / a.c.n_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = seq_len(a.lens, b, a.max_len, tid == 0 ? a.err : nullptr);
    const int N = L < a.budget ? L : a.budget;
    int *kept = a.kept + (size_t)blockIdx.x * a.budget;
    if (h == 0 && tid == 0) a.new_lens[b] = N;
    for (int i = N + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
    if (L <= a.budget) {
        for (int i = tid; i < N; i += kSelThreads) kept[i] = i;
        return;
    }
    // sinks + recent <= budget < L: the protected ends do not meet
    const int *row = a.table + (size_t)b * a.table_stride;
    const int lo = a.sinks, hi = L - a.recent;
    int need = N - a.sinks - a.recent;             // to take from [lo, hi)
    auto key_at = [&](int t) -> uint32_t {
        const SlotRef r = find_slot(a.c, row, t);
        return r.page < 0 ? 0u : weight_key(__ldg(a.c.weight + slot_weight(a.c, r, h)));
    };
    // radix select: the key of the need-th largest weight, digit by digit (11, 11, 10 bits)
    uint32_t prefix = 0;
    if (need > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bins = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            const uint32_t above = pass == 0 ? 0u : prefix >> (pass == 1 ? 21 : 10);
            for (int t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t k = key_at(t);
                if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == above)
                    atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
            }
            __syncthreads();
            if (warp == 0) {   // from the top bin down: where the count passes `need`
                int left = need;
                for (int top = bins; top > 0; top -= 32) {
                    const int bin = top - 1 - lane, c = s_hist[bin];
                    int sum = c;
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(~0u, sum, o);
                        if (lane >= o) sum += v;
                    }
                    const unsigned hit = __ballot_sync(~0u, sum >= left);
                    if (hit) {
                        const int first = __ffs(hit) - 1;
                        if (lane == first) s_digit = bin, s_need = left - (sum - c);
                        break;
                    }
                    left -= __shfl_sync(~0u, sum, 31);
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            need = s_need;                        // slots of this digit still to take
            __syncthreads();
        }
    }
    // Emit in slot order.  Every warp takes one stretch of slots: it counts
    // (protected or above the threshold) and (equal to it), the counts are
    // summed over the warps before it, then it writes.
    const bool any = N > a.sinks + a.recent;
    const int per = ((L + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int t0 = warp * per, t1 = t0 + per < L ? t0 + per : L;
    int gt = 0, eq = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int base_gt = 0, base_eq = 0;
        if (pass) {
            for (int w = 0; w < warp; ++w) base_gt += s_gt[w], base_eq += s_eq[w];
        }
        for (int t = t0 + lane; t - lane < t1; t += 32) {
            const bool safe = t < t1 && (t < lo || t >= hi);
            const uint32_t k = t < t1 && !safe && any ? key_at(t) : 0u;
            const bool mid = t < t1 && !safe && any;
            const unsigned g = __ballot_sync(~0u, safe || (mid && k > prefix));
            const unsigned e = __ballot_sync(~0u, mid && k == prefix);
            if (!pass) {
                gt += __popc(g), eq += __popc(e);
            } else {
                const unsigned below = (1u << lane) - 1u;
                const int rank_e = base_eq + __popc(e & below);     // equal ones before this slot
                const int taken = rank_e < need ? rank_e : need;
                const bool take = (g >> lane & 1u) || ((e >> lane & 1u) && rank_e < need);
                if (take) kept[base_gt + __popc(g & below) + taken] = t;
                base_gt += __popc(g), base_eq += __popc(e);
            }
        }
        if (!pass) {
            if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
            __syncthreads();
        }
    }
}

// Copies kept slots: `lanes` threads a slot and side (K or V), 16 bytes a thread and step.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, int row_b,
                                                                  int slots_per_block) {
    griddep_launch_dependents();
    griddep_wait();
    const int bh = blockIdx.x, h = bh % a.c.n_heads, b = bh / a.c.n_heads;
    const int n = __ldg(a.new_lens + b);
    const int i0 = blockIdx.y * slots_per_block;
    const int i1 = i0 + slots_per_block < n ? i0 + slots_per_block : n;
    const int *src_row = a.table + (size_t)b * a.table_stride;
    const int *dst_row = a.dst_table + (size_t)b * a.dst_stride;
    const int *kept = a.kept + (size_t)bh * a.budget;
    const int chunks = row_b / 16;
    for (int w = threadIdx.x; w < (i1 - i0) * chunks; w += kMoveThreads) {
        const int i = i0 + w / chunks, c = w % chunks;
        const SlotRef s = find_slot(a.c, src_row, __ldg(kept + i)), d = find_slot(a.c, dst_row, i);
        if (s.page < 0 || d.page < 0) {
            if (c == 0) raise_device_error(a.err, kErrPage);
            continue;
        }
        const long long so = slot_bytes(a.c, s, h) + 16 * c, to = slot_bytes(a.c, d, h) + 16 * c;
        const uint4 k = *reinterpret_cast<const uint4 *>(a.c.k + so), v = *reinterpret_cast<const uint4 *>(a.c.v + so);
        *reinterpret_cast<uint4 *>(a.c.k + to) = k;
        *reinterpret_cast<uint4 *>(a.c.v + to) = v;
        if (c == 0) a.c.weight[slot_weight(a.c, d, h)] = a.c.weight[slot_weight(a.c, s, h)];
    }
}

}  // namespace

int run_kv_evict(const EvictArgs &a, cudaStream_t st) {
    int rc = launch_pdl("qg_kv_evict", evict_select_kernel, dim3(a.n_seq * a.c.n_heads), kSelThreads, 0, st, a);
    if (rc != kOk) return rc;
    const int row_b = a.c.dim * (a.c.type == kE4m3 ? 1 : 2);
    const int most = a.max_len < a.budget ? a.max_len : a.budget;
    if (most == 0) return kOk;
    int per = 64;
    while ((most + per - 1) / per > 65535) per *= 2;
    return launch_pdl("qg_kv_evict", evict_move_kernel, dim3(a.n_seq * a.c.n_heads, (most + per - 1) / per),
                      kMoveThreads, 0, st, a, row_b, per);
}

}  // namespace qg
