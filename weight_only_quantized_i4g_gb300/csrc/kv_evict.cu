// kv_evict.cu -- eviction by accumulated attention weight (qg_kv_evict).
//
// Per sequence and head, of L slots N = min(L, budget) are kept: the first
// `sinks`, the last `recent` and, of the slots between them, those of largest
// weight (equal weights: the lower slot).  A select kernel finds them with a
// radix select over order-preserving 32-bit keys and writes their slots in
// order; a move kernel copies K, V and weight of the kept slots to the new
// pages.  Selection reads 4 bytes a slot; the copies, 4 D bytes a kept slot
// and 16-bit element each way, are the bulk and bound by HBM.
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace qg {

namespace cg = cooperative_groups;

namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Order of weights: every NaN above +inf, -0 equal to +0; larger key = larger weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The ones of the low half of each byte, in that byte.
__device__ __forceinline__ unsigned ones_of_nibbles(unsigned v) {
    v &= 0x0F0F0F0Fu;
    v -= v >> 1 & 0x05050505u;
    return (v & 0x03030303u) + (v >> 2 & 0x03030303u);
}

// A cluster per sequence and head; its blocks share the slots in equal
// stretches and keep their keys in shared memory (`cap` of them; a longer
// stretch reads the rest again).  Three digits (11, 11, 10 bits) of the key of
// the last slot to keep are found from the top: each block counts its keys'
// digits, each rank adds up one slice of the bins over the blocks and hands
// the sums to all, and every block finds the same bin.  One block per head
// took 315 us for three sequences of 100k slots, 8 heads, two thirds of it
// here; the clusters spread that over the SMs.  A digit whose slots are all
// kept ends the search (distinct weights: mostly the second).
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a, int cap) {
    constexpr int kSelWarps = kSelThreads / 32;
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ int s_hist[kBins], s_total[kBins];
    __shared__ int s_warp[2][kSelWarps];
    __shared__ int2 s_block[kMaxCluster];
    __shared__ int s_digit, s_need, s_bin;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    griddep_wait();
    griddep_launch_dependents();                   // after the wait: the copies' kernel reads lengths and tables before its own
    const int bh = blockIdx.x / ranks, b = bh / a.c.n_heads, h = bh - b * a.c.n_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = seq_len(a.lens, b, a.max_len, tid == 0 && rank == 0 ? a.err : nullptr);
    const int N = L < a.budget ? L : a.budget;
    int *kept = a.kept + (size_t)bh * a.budget;
    const int first = rank * kSelThreads + tid, step = ranks * kSelThreads;
    if (h == 0 && first == 0) a.new_lens[b] = N;
    for (unsigned i = N + first; i < (unsigned)a.budget; i += step) kept[i] = -1;   // unsigned: the budget may be up to 2^31 - 1
    if (L <= a.budget) {                           // the same for every block of the cluster
        for (int i = first; i < N; i += step) kept[i] = i;
        return;
    }
    // sinks + recent <= budget < L: the protected ends do not meet
    const int *row = a.table + (size_t)b * a.table_stride;
    const int lo = a.sinks, hi = L - a.recent;
    int need = N - a.sinks - a.recent;             // to take from [lo, hi)
    const bool any = need > 0;
    const bool quads = a.c.page % 4 == 0 && reinterpret_cast<uintptr_t>(a.c.weight) % 16 == 0;
    // this block's stretch, and each warp's in it
    const int per_warp = ((L + ranks * kSelWarps - 1) / (ranks * kSelWarps) + 31) & ~31, per = per_warp * kSelWarps;
    const int r0 = rank * per < L ? rank * per : L, r1 = r0 + per < L ? r0 + per : L;
    auto key_in_cache = [&](int t) -> uint32_t {
        const SlotRef r = find_slot(a.c, row, t);
        return r.page < 0 ? 0u : weight_key(a.c.weight[slot_weight(a.c, r, h)]);
    };
    // four keys from t on (t - r0 and cap are multiples of four), 0 past the stretch
    auto keys_at = [&](int t, uint32_t (&k)[4]) {
        if (t - r0 < cap) {
            const uint4 v = *reinterpret_cast<const uint4 *>(s_key + (t - r0));
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) k[x] = t + x < r1 ? key_in_cache(t + x) : 0u;
        }
    };
    const int in_smem = r1 - r0 < cap ? r1 - r0 : cap;
    // of this block's stretch, the slots to choose from: m0 to m0 + m_n
    const int m0 = r0 > lo ? r0 : lo, m_n = (r1 < hi ? r1 : hi) > m0 ? (r1 < hi ? r1 : hi) - m0 : 0;
    auto count = [&](int t, uint32_t digit) {      // additions of one that a warp shares are combined in hardware
        if ((unsigned)(t - m0) < (unsigned)m_n) atomicAdd(&s_hist[digit], 1);
    };
    if (any) {
        // the keys, and the first digit's counts with them
        for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        if (quads) {
            // a page holds whole fours: one look-up and one load for four slots,
            // eight look-ups, then four loads in flight
            constexpr int kAhead = 8, kLoads = 4;
            for (int i = 4 * tid; i < in_smem; i += 4 * kAhead * kSelThreads) {
                int page[kAhead], off[kAhead];
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    int index;
                    split_slot(a.c, r0 + i + x * 4 * kSelThreads, &index, &off[x]);
                    page[x] = i + x * 4 * kSelThreads < in_smem ? row[index] : -1;
                }
#pragma unroll
                for (int x0 = 0; x0 < kAhead; x0 += kLoads) {
                    float4 wt[kLoads];
#pragma unroll
                    for (int x = 0; x < kLoads; ++x) {
                        const SlotRef r{page[x0 + x], off[x0 + x]};
                        if ((unsigned)r.page < (unsigned)a.c.n_pages)
                            wt[x] = *reinterpret_cast<const float4 *>(a.c.weight + slot_weight(a.c, r, h));
                    }
#pragma unroll
                    for (int x = 0; x < kLoads; ++x) {
                        const int at = i + (x0 + x) * 4 * kSelThreads;
                        if (at >= in_smem) break;
                        const bool ok = (unsigned)page[x0 + x] < (unsigned)a.c.n_pages;
                        const uint4 k = ok ? make_uint4(weight_key(wt[x].x), weight_key(wt[x].y), weight_key(wt[x].z),
                                                        weight_key(wt[x].w))
                                           : make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(s_key + at) = k;
                        count(r0 + at, k.x >> 21), count(r0 + at + 1, k.y >> 21);
                        count(r0 + at + 2, k.z >> 21), count(r0 + at + 3, k.w >> 21);
                    }
                }
            }
        } else {
            for (int i = tid; i < in_smem; i += kSelThreads) {
                const uint32_t k = key_in_cache(r0 + i);
                s_key[i] = k;
                count(r0 + i, k >> 21);
            }
        }
        for (int i = in_smem + tid; i < r1 - r0; i += kSelThreads) count(r0 + i, key_in_cache(r0 + i) >> 21);
    }
    __syncthreads();

    uint32_t prefix = 0;
    if (tid == 0) s_digit = s_need = s_bin = 0;
    if (any) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
            if (pass > 0) {
                const int done = pass == 1 ? 21 : 10;                         // low bits not yet fixed
                for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
                __syncthreads();
                for (int t = r0 + 4 * tid; t < r1; t += 4 * kSelThreads) {
                    uint32_t k[4];
                    keys_at(t, k);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if ((k[x] ^ prefix) < 1u << done) count(t + x, (k[x] >> shift) & (bins - 1));
                }
            }
            int *total = s_hist;
            if (ranks > 1) {
                total = s_total;
                cluster.sync();
                const int slice = bins / ranks;
                for (int i = tid; i < slice; i += kSelThreads) {
                    const int bin = rank * slice + i;
                    int sum = 0;
#pragma unroll
                    for (int x = 0; x < kMaxCluster; ++x)
                        if (x < ranks) sum += cluster.map_shared_rank(s_hist, x)[bin];
#pragma unroll
                    for (int x = 0; x < kMaxCluster; ++x)
                        if (x < ranks) cluster.map_shared_rank(s_total, x)[bin] = sum;
                }
                cluster.sync();
            } else {
                __syncthreads();
            }
            // from the top bin down: where the count reaches `need`
            const int each = bins / kSelThreads;
            int mine[kBins / kSelThreads], sum = 0;
#pragma unroll
            for (int i = 0; i < kBins / kSelThreads; ++i) {
                mine[i] = i < each ? total[bins - 1 - (tid * each + i)] : 0;
                sum += mine[i];
            }
            int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) s_warp[0][warp] = inc;
            __syncthreads();
            int before = inc - sum + __reduce_add_sync(~0u, lane < warp ? s_warp[0][lane] : 0);
            if (before < need && need <= before + sum) {
#pragma unroll
                for (int i = 0; i < kBins / kSelThreads; ++i) {
                    if (before < need && need <= before + mine[i])
                        s_digit = bins - 1 - (tid * each + i), s_need = need - before, s_bin = mine[i];
                    before += mine[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            need = s_need;                         // slots of this digit still to take
            const bool all_of_it = need == s_bin;
            __syncthreads();
            if (all_of_it && prefix > 0) {         // then those above the last key below the digit
                --prefix;
                need = 0;
                break;
            }
        }
    } else if (ranks > 1) {
        cluster.sync();                            // every block has started: its shared memory may be written (a search has met them)
    }
    // Emit in slot order, four neighbouring slots a lane: every warp counts its
    // stretch (kept for sure, and equal to the threshold), the counts before it
    // are summed, then it writes.
    const int t0 = r0 + warp * per_warp, t1 = t0 + per_warp < r1 ? t0 + per_warp : r1;
    // bits 0-3: slot t + x is kept for sure; bits 4-7: it ties with the threshold
    auto flags = [&](int t) {
        uint32_t k[4] = {0u, 0u, 0u, 0u};
        if (any && t < t1) keys_at(t, k);
        unsigned f = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool safe = (unsigned)(t + x - lo) >= (unsigned)(hi - lo);
            if (t + x < t1 && (safe || k[x] > prefix)) f |= 1u << x;
            if (t + x < t1 && !safe && k[x] == prefix) f |= 16u << x;
        }
        return f;
    };
    int sure_n = 0, tie_n = 0;
    unsigned long long seen = 0;                   // the flags of the first eight rounds of 128 slots
    int round = 0;
    for (int t = t0 + 4 * lane; t < t1; t += 128, ++round) {
        const unsigned f = flags(t);
        if (round < 8) seen |= (unsigned long long)f << (8 * round);
        sure_n += __popc(f & 15u), tie_n += __popc(f >> 4);
    }
    sure_n = __reduce_add_sync(~0u, sure_n), tie_n = __reduce_add_sync(~0u, tie_n);
    if (lane == 0) s_warp[0][warp] = sure_n, s_warp[1][warp] = tie_n;
    __syncthreads();
    const int of_sure = lane < kSelWarps ? s_warp[0][lane] : 0, of_tie = lane < kSelWarps ? s_warp[1][lane] : 0;
    const int all_sure = __reduce_add_sync(~0u, of_sure), all_tie = __reduce_add_sync(~0u, of_tie);
    int base_sure = __reduce_add_sync(~0u, lane < warp ? of_sure : 0);
    int base_tie = __reduce_add_sync(~0u, lane < warp ? of_tie : 0);
    if (ranks > 1) {
        if (tid < ranks) cluster.map_shared_rank(s_block, tid)[rank] = make_int2(all_sure, all_tie);
        cluster.sync();                            // also the last access to another block's memory
        for (int x = 0; x < rank; ++x) base_sure += s_block[x].x, base_tie += s_block[x].y;
    }
    // four rounds at a time: a count of a round is 128 at most and takes a byte
    const bool ties = need > 0 && tie_n > 0;       // the same in every lane
    for (int g = 0; t0 + 128 * g < t1; g += 4) {
        const int t = t0 + 128 * g + 4 * lane;
        unsigned f4 = 0;
        if (g < 8) {
            f4 = (unsigned)(seen >> (8 * g));
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) f4 |= flags(t + 128 * x) << (8 * x);
        }
        const unsigned sure4 = ones_of_nibbles(f4), tie4 = ties ? ones_of_nibbles(f4 >> 4) : 0u;
        unsigned sure_in = sure4, tie_in = tie4;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(~0u, sure_in, o);
            if (lane >= o) sure_in += v;
        }
        if (ties)
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(~0u, tie_in, o);
                if (lane >= o) tie_in += v;
            }
        const unsigned sure_all = __shfl_sync(~0u, sure_in, 31), tie_all = __shfl_sync(~0u, tie_in, 31);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            int sure = base_sure + ((sure_in - sure4) >> (8 * r) & 255u), tie = base_tie + ((tie_in - tie4) >> (8 * r) & 255u);
            // at < N always, unless the weights change under the call
            if (ties) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int at = sure + (tie < need ? tie : need);
                    const bool is_sure = f4 >> (8 * r + x) & 1u, is_tie = f4 >> (8 * r + 4 + x) & 1u;
                    if ((is_sure || (is_tie && tie < need)) && at < N) kept[at] = t + 128 * r + x;
                    sure += is_sure, tie += is_tie;
                }
            } else {
                int at = sure + (tie < need ? tie : need);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if ((f4 >> (8 * r + x) & 1u) && at < N) kept[at++] = t + 128 * r + x;
            }
            base_sure += sure_all >> (8 * r) & 255u, base_tie += tie_all >> (8 * r) & 255u;
        }
    }
}

// Copies kept slots, `slots` a block: their places are looked up once, then
// every thread has eight 16-byte loads in flight before its stores.  24
// sequences of 1500 to 8191 slots cut to 4096 (8 heads of 128, bf16): 106 us,
// the measured copy rate, after 13 of the select kernel.
constexpr int kMoveThreads = 256, kMoveSlots = 256, kMoveAhead = 4;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, FastDiv chunks,
                                                                  int slots) {
    __shared__ long long s_src[kMoveSlots], s_dst[kMoveSlots];
    griddep_launch_dependents();
    const int bh = blockIdx.x, b = bh / a.c.n_heads, h = bh - b * a.c.n_heads, tid = threadIdx.x;
    // before the wait, past L1: all but `kept` stands
    int len = __ldcg(a.lens + b);
    len = len < 0 ? 0 : len < a.max_len ? len : a.max_len;
    const int n = len < a.budget ? len : a.budget;
    auto place = [&](long long i) {                // of kept slot i in the new pages
        SlotRef r{-1, 0};
        if (tid < slots && i < n) {
            int index;
            split_slot(a.c, (int)i, &index, &r.off);
            const int page = __ldcg(a.dst_table + (size_t)b * a.dst_stride + index);
            if ((unsigned)page < (unsigned)a.c.n_pages) r.page = page;
        }
        return r;
    };
    SlotRef d = place((long long)blockIdx.y * slots + tid);
    griddep_wait();
    for (long long i0 = (long long)blockIdx.y * slots; i0 < n; i0 += (long long)gridDim.y * slots) {
        const int count = n - i0 < slots ? (int)(n - i0) : slots;
        float weight = 0.f;
        bool ok = false;
        __syncthreads();
        if (tid < count) {
            const int t = a.kept[(size_t)bh * a.budget + (int)i0 + tid];
            SlotRef s{-1, 0};
            if ((unsigned)t < (unsigned)len) s = find_slot(a.c, a.table + (size_t)b * a.table_stride, t);
            ok = s.page >= 0 && d.page >= 0;
            s_src[tid] = ok ? slot_bytes(a.c, s, h) : -1;
            s_dst[tid] = ok ? slot_bytes(a.c, d, h) : -1;
            if (ok) weight = a.c.weight[slot_weight(a.c, s, h)];
            else raise_device_error(a.err, kErrPage);
        }
        __syncthreads();
        const int work = count * (int)chunks.d;
        for (int w0 = tid; w0 < work; w0 += kMoveAhead * kMoveThreads) {
            uint4 k[kMoveAhead], v[kMoveAhead];
            long long to[kMoveAhead];
#pragma unroll
            for (int x = 0; x < kMoveAhead; ++x) {
                const int w = w0 + x * kMoveThreads;
                to[x] = -1;
                if (w >= work) continue;
                const int i = quotient(w, chunks), at = 16 * (w - i * (int)chunks.d);
                if (s_src[i] < 0) continue;
                to[x] = s_dst[i] + at;
                k[x] = *reinterpret_cast<const uint4 *>(a.c.k + s_src[i] + at);
                v[x] = *reinterpret_cast<const uint4 *>(a.c.v + s_src[i] + at);
            }
#pragma unroll
            for (int x = 0; x < kMoveAhead; ++x) {
                if (to[x] < 0) continue;
                *reinterpret_cast<uint4 *>(a.c.k + to[x]) = k[x];
                *reinterpret_cast<uint4 *>(a.c.v + to[x]) = v[x];
            }
        }
        if (ok) a.c.weight[slot_weight(a.c, d, h)] = weight;
        d = place(i0 + (long long)gridDim.y * slots + tid);
    }
}

}  // namespace

template <int THREADS>
int launch_select(const EvictArgs &a, int ranks, cudaStream_t st) {
    const int warps = ranks * (THREADS / 32);
    const long long keys = (((long long)a.max_len + warps - 1) / warps + 31) / 32 * THREADS;   // a block's stretch
    const int cap = keys < 49152 ? (int)keys : 49152;              // up to 192 KB of keys
    set_max_dynamic_smem(reinterpret_cast<const void *>(evict_select_kernel<THREADS>), 4 * 49152);
    return launch_clusters("qg_kv_evict", evict_select_kernel<THREADS>, dim3(a.n_seq * a.c.n_heads * ranks), THREADS,
                           ranks, (size_t)cap * 4, st, a, cap);
}

int run_kv_evict(const EvictArgs &a, cudaStream_t st) {
    // As many blocks per head as have an SM each and 1024 slots or more (two
    // an SM did not all start at once as clusters of eight: three sequences of
    // 100k slots 143 us against 130).  Their threads, where every head has an SM:
    // 1024 for many slots, else 512 (8 heads, 30000 slots on eight blocks each:
    // 14.0 us a call with 1024, 12.5 with 512).  With more heads than SMs several
    // blocks share one, the more the shorter they are; 8 heads a sequence, with
    // 1024 / 512 / 256 threads:
    //   200 sequences of 1000 slots: - / 173 / 156 us, 64 of 2000: - / 59 / 55
    //   24 of 3000 to 6000: 34.8 / 28.9 / 32.7, 64: 77 / 64 / 61
    //   40 of 1500 to 8191: 199 / 192 / 229, 24: 119.7 / 121.0 / 138.6
    //   64 of 16000: 92 / 79 / -, 24 of 30000: 54 / 64 / 92
    const long long heads = (long long)a.n_seq * a.c.n_heads;
    const bool room = heads <= num_sms();
    int ranks = 1;
    while (ranks < kMaxCluster && heads * ranks * 2 <= num_sms() && ranks * 2048LL <= a.max_len) ranks *= 2;
    const int stretch = a.max_len / ranks;
    int rc = stretch > (room ? 4096 : 16384) ? launch_select<1024>(a, ranks, st)
             : room || stretch > 2048        ? launch_select<512>(a, ranks, st) : launch_select<256>(a, ranks, st);
    const int most = a.max_len < a.budget ? a.max_len : a.budget;
    if (rc != kOk || most == 0) return rc;
    const int chunks = a.c.dim * (a.c.type == kE4m3 ? 1 : 2) / 16;
    int slots = kMoveAhead * kMoveThreads / chunks;               // one round of loads a block
    if (slots > kMoveSlots) slots = kMoveSlots;
    const int blocks = (most + slots - 1) / slots;
    return launch_pdl("qg_kv_evict", evict_move_kernel, dim3(a.n_seq * a.c.n_heads, blocks < 65535 ? blocks : 65535),
                      kMoveThreads, 0, st, a, fast_div(chunks), slots);
}

}  // namespace qg
