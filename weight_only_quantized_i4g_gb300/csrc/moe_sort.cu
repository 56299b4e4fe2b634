// moe_sort.cu -- routed slots sorted by expert (qg_moe_sort).
//
//   offsets[e] = number of slots s with 0 <= ids[s] < e
//   place[s]   = offsets[ids[s]] + number of s' < s with ids[s'] = ids[s]
//   order[place[s]] = s
//
// A stable counting sort: every warp counts the experts of a stretch of
// slots, the counts before it (of lower experts, and of its own expert in
// earlier stretches) are added up, and a second pass over the stretch hands
// out the places in order.  No atomics: of the lanes that hold the same
// expert one counts for all, so the result never depends on timing.
#include "moe.cuh"

namespace qg {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortSmem = 200 * 1024;   // counts: a word a warp and expert
constexpr int kNone = 0x7FFFFFFF;

__device__ __forceinline__ int expert_of(const SortArgs &a, long long s) {
    if (s >= a.slots) return kNone;
    const int e = a.ids[s];
    return (unsigned)e < (unsigned)a.experts ? e : kNone;
}

// Exclusive prefix sums over the threads of a block; *total is their sum.
__device__ __forceinline__ int block_prefix(int v, int *s_warp, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < warps; ++w) {
        const int n = s_warp[w];
        before += w < warp ? n : 0;
        sum += n;
    }
    __syncthreads();
    *total = sum;
    return before + x - v;
}

__global__ void __launch_bounds__(kSortThreads) sort_one_kernel(const SortArgs a) {
    extern __shared__ int s_count[];               // [warps][experts]
    __shared__ int s_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = a.experts;
    int *mine = s_count + (size_t)warp * E;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) s_count[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const long long per = ((long long)(a.slots + warps - 1) / warps + 31) & ~31ll;
    const long long s0 = warp * per, s1 = min(s0 + per, (long long)a.slots);
    for (long long s = s0; s < s1; s += 32) {
        const int e = expert_of(a, s + lane);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e != kNone && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int sum = 0, total;
        if (e < E)
            for (int w = 0; w < warps; ++w) sum += s_count[(size_t)w * E + e];
        int at = carry + block_prefix(sum, s_warp, &total);
        if (e < E) {
            a.offsets[e] = at;
            for (int w = 0; w < warps; ++w) {
                const int n = s_count[(size_t)w * E + e];
                s_count[(size_t)w * E + e] = at;
                at += n;
            }
        }
        carry += total;
    }
    if (threadIdx.x == 0) a.offsets[E] = carry;
    __syncthreads();
    for (long long s = s0; s < s1; s += 32) {
        const int e = expert_of(a, s + lane);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int at = e != kNone ? mine[e] + __popc(same & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (e != kNone && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (s + lane < s1) {
            a.place[s + lane] = at;
            if (a.order && at >= 0) a.order[at] = (int)(s + lane);
        }
    }
}

}  // namespace

size_t ws_moe_sort(int, int) { return 0; }

int run_moe_sort(const SortArgs &a, void *, cudaStream_t st) {
    int warps = kSortThreads / 32;
    while (warps > 1 && (size_t)warps * a.experts * 4 > (size_t)kSortSmem) warps /= 2;
    const size_t smem = (size_t)warps * a.experts * 4;
    set_max_dynamic_smem(reinterpret_cast<const void *>(sort_one_kernel), kSortSmem);
    return launch_pdl("qg_moe_sort", sort_one_kernel, 1, warps * 32, smem, st, a);
}

}  // namespace qg
