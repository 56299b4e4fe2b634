// moe_sort.cu -- routed slots sorted by expert (qg_moe_sort).
//
//   offsets[e] = number of slots s with 0 <= ids[s] < e
//   place[s]   = offsets[ids[s]] + number of s' < s with ids[s'] = ids[s]
//   order[place[s]] = s
//
// A stable counting sort: every warp counts the experts of a stretch of
// slots, the counts before it (of lower experts, and of its own expert in
// earlier stretches) are added up, and a second pass over the stretch hands
// out the places in order: of the lanes that hold the same expert one counts
// for all.  The first kernel of a long list counts a block's stretch by atomic
// additions in shared memory, whole numbers whose sums are the same in any
// order, so the result never depends on timing.
#include <algorithm>

#include "moe.cuh"

namespace qg {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortSmem = 200 * 1024;   // counts: a word a warp and expert
constexpr size_t kPlainSmem = 48 * 1024 - 256;   // what a kernel may have without asking

// Experts of the 32 kBatch slots from s on (`experts` for none here), this
// lane's 32 apart: all loads in flight at once.  Past L1, which may hold what an earlier call left there.
constexpr int kBatch = 4;
__device__ __forceinline__ void load_experts(const SortArgs &a, long long s, long long s1, int lane, int (&e)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const long long at = s + 32 * i + lane;
        e[i] = at < s1 ? __ldcg(a.ids + at) : -1;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) e[i] = (unsigned)e[i] < (unsigned)a.experts ? e[i] : a.experts;
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

// The lanes with this lane's expert, a vote for each of its bits (the match
// instruction takes a third longer: 16384 x 8 slots 12.5 us against 9.2).
__device__ __forceinline__ unsigned lanes_of(int e, int bits) {
    unsigned same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const unsigned yes = __ballot_sync(0xffffffffu, e >> b & 1);
        same &= e >> b & 1 ? yes : ~yes;
    }
    return same;
}

// A warp counts the experts of a batch in its own row of counts.
__device__ __forceinline__ void count_batch(const SortArgs &a, const int (&e)[kBatch], long long s, long long s1, int lane,
                                            int *mine) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        if (s + 32 * i >= s1) break;
        const unsigned same = lanes_of(e[i], a.bits);
        if (e[i] != a.experts && lane == __ffs(same) - 1) mine[e[i]] += __popc(same);
        __syncwarp();
    }
}

// And gives each slot its place: `mine` holds the next place of each expert.
__device__ __forceinline__ void place_batch(const SortArgs &a, const int (&e)[kBatch], long long s, long long s1, int lane,
                                            int *mine) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        if (s + 32 * i >= s1) break;
        const long long slot = s + 32 * i + lane;
        const unsigned same = lanes_of(e[i], a.bits);
        const int at = e[i] != a.experts ? mine[e[i]] + __popc(same & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (e[i] != a.experts && lane == __ffs(same) - 1) mine[e[i]] += __popc(same);
        __syncwarp();
        if (slot < s1) {
            a.place[slot] = at;
            if (a.order && at >= 0) a.order[at] = (int)slot;
        }
    }
}

// Both passes over a warp's slots [s0, s1); `between` turns the counts into
// places.  One batch stays in registers for the second pass.
template <class F>
__device__ __forceinline__ void count_and_place(const SortArgs &a, long long s0, long long s1, int lane, int *mine, F between) {
    constexpr int kStep = 32 * kBatch;
    int e[kBatch];
    for (long long s = s0; s < s1; s += kStep) {
        load_experts(a, s, s1, lane, e);
        count_batch(a, e, s, s1, lane, mine);
    }
    between();
    const bool again = s1 - s0 > kStep;
    for (long long s = s0; s < s1; s += kStep) {
        if (again) load_experts(a, s, s1, lane, e);
        place_batch(a, e, s, s1, lane, mine);
    }
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
    count_and_place(a, s0, s1, lane, mine, [&] {
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
    });
}

// Long lists take two kernels: every block of the first counts one stretch,
// and every block of the second adds up the counts it needs (all experts' sums,
// and its own experts' before its stretch) and places its stretch.
constexpr int kPlaceThreads = 512;      // 16 warps
constexpr int kMaxCounts = 1 << 16;     // counts of all blocks and experts that every block reads

struct SortPlan {
    int blocks, warps, per_warp;        // a warp's slots, whole 32s
};
// A block for 1024 slots up to 64 blocks, whose counts every block reads in a
// few batches (16384 slots: 4.8 us, with 2048 a block 6.7; 131072 slots: 8.5 us
// with 64 blocks, 13 with 128), then one for 4096.  Never falls as the slots
// grow, so that the workspace of a long list serves its shorter ones.
long long most_blocks(int slots, int experts) {
    const long long by_size = std::min((slots + 1023LL) / 1024, std::max(64LL, slots / 4096LL));
    return std::min<long long>({by_size, std::max(1, kMaxCounts / experts), 1024});
}
SortPlan sort_plan(int slots, int experts) {
    long long blocks = most_blocks(slots, experts);
    int warps = kPlaceThreads / 32;        // a row of counts each in shared memory, and one more
    while ((warps + 1) * experts * 4 > kSortSmem) warps /= 2;
    long long per_warp = ((long long)slots + blocks * warps - 1) / (blocks * warps);
    per_warp = (per_warp + 31) / 32 * 32;
    blocks = ((long long)slots + per_warp * warps - 1) / (per_warp * warps);
    return SortPlan{(int)blocks, warps, (int)per_warp};
}

__global__ void __launch_bounds__(kPlaceThreads) sort_count_kernel(const SortArgs a, int per_warp, int *counts) {
    extern __shared__ int s_count[];               // [experts]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
    for (int i = threadIdx.x; i < E; i += blockDim.x) s_count[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const long long s0 = ((long long)blockIdx.x * (blockDim.x >> 5) + warp) * per_warp;
    const long long s1 = min(s0 + per_warp, (long long)a.slots);
    for (long long s = s0; s < s1; s += 32 * kBatch) {
        int e[kBatch];
        load_experts(a, s, s1, lane, e);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)           // sums of whole numbers: any order gives the same
            if (e[i] != E) atomicAdd(&s_count[e[i]], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < E; i += blockDim.x) counts[(size_t)blockIdx.x * E + i] = s_count[i];
}

__global__ void __launch_bounds__(kPlaceThreads) sort_place_kernel(const SortArgs a, int per_warp, const int *counts) {
    extern __shared__ int s_count[];               // [warps][experts], then [experts] places of the stretch's first
    __shared__ int s_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = a.experts;
    int *mine = s_count + (size_t)warp * E, *s_base = s_count + (size_t)warps * E;
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) s_count[i] = 0;
    __syncthreads();
    const long long s0 = ((long long)blockIdx.x * warps + warp) * per_warp;
    const long long s1 = min(s0 + per_warp, (long long)a.slots);
    // The counting kernel lets this one start after its own wait, so the ids
    // are there; its counts are after this kernel's.
    count_and_place(a, s0, s1, lane, mine, [&] {
        griddep_wait();
        griddep_launch_dependents();
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += blockDim.x) {
            const int e = e0 + threadIdx.x;
            int before = 0, all = 0, total;
            if (e < E) {
#pragma unroll 16
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int n = counts[(size_t)b * E + e];
                    all += n;
                    before += b < (int)blockIdx.x ? n : 0;
                }
            }
            const int at = carry + block_prefix(all, s_warp, &total);
            if (e < E) {
                s_base[e] = at + before;
                if (blockIdx.x == 0) a.offsets[e] = at;
            }
            carry += total;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = carry;
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int at = s_base[e];
            for (int w = 0; w < warps; ++w) {
                const int n = s_count[(size_t)w * E + e];
                s_count[(size_t)w * E + e] = at;
                at += n;
            }
        }
        __syncthreads();
    });
}

}  // namespace

// One block's 32 warps take up to this many slots.
constexpr int kOneBlock = 1024;

size_t ws_moe_sort(int slots, int experts) {
    return slots <= kOneBlock ? 0 : (size_t)most_blocks(slots, experts) * experts * sizeof(int);
}

int run_moe_sort(SortArgs a, void *ws, cudaStream_t st) {
    for (a.bits = 1; a.experts >> a.bits; ++a.bits) {}
    const char *what = "qg_moe_sort";
    if (a.slots <= kOneBlock) {
        // as many warps as there are 32s of slots, and counts in shared memory
        int warps = kSortThreads / 32;
        while (warps > 1 && ((size_t)warps * a.experts * 4 > (size_t)kSortSmem || warps * 16 >= a.slots)) warps /= 2;
        warps = std::max(warps, 4);
        const size_t smem = (size_t)warps * a.experts * 4;
        if (smem > kPlainSmem) set_max_dynamic_smem(reinterpret_cast<const void *>(sort_one_kernel), kSortSmem);
        return launch_pdl(what, sort_one_kernel, 1, warps * 32, smem, st, a);
    }
    const SortPlan p = sort_plan(a.slots, a.experts);
    int *counts = static_cast<int *>(ws);
    const size_t row = (size_t)a.experts * 4;
    if (row * (p.warps + 1) > kPlainSmem) set_max_dynamic_smem(reinterpret_cast<const void *>(sort_place_kernel), kSortSmem);
    const int rc = launch_pdl(what, sort_count_kernel, p.blocks, p.warps * 32, row, st, a, p.per_warp, counts);
    if (rc != kOk) return rc;
    return launch_pdl(what, sort_place_kernel, p.blocks, p.warps * 32, row * (p.warps + 1), st, a, p.per_warp,
                      (const int *)counts);
}

}  // namespace qg
