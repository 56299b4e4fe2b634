// gemm_e4m3_tc.cu -- products of e4m3 activations with e4m3 weights on the
// 5th-generation tensor cores (tcgen05 kind::f8f6f4, accumulators in tensor
// memory), for rows of whole 16-byte lines.
//
//   Y[m, o] = sum_b xs[m, b] ws[o/128, b] sum_{i in block b} X[m, i] W[o, i]
//
// A tile is 128 outputs (rows of W, MMA M) by up to BT tokens of one expert
// (MMA N, as many as the tile has, in sixteens).  One K step is one block of
// 128 elements: four MMAs of K = 32 leave the block's sums in one of several
// buffers of tensor memory, and the promoting warps add them, times the two
// scales, to f32 sums in registers.  The outputs of a tile share one weight
// scale, and the product of both scales comes from shared memory, a token
// each.  One persistent thread block per SM:
//   warp 0      TMA producer: per K step the 128 x 128 codes of W and the
//               tile's tokens x 128 of X, both 128-byte swizzled
//   warp 1      allocates tensor memory, issues the MMAs from one thread
//   warp 2      the scales' products, kChunk steps at a time
//   warps 4..   promote: tensor-memory lanes 32 (w % 4) .. + 31, columns in
//               sixteens shared by the one or two warps of a lane quarter
// Calls of few tiles split K over the blocks of a cluster, which add their
// sums over distributed shared memory, in rank order.
#include "gemm_tc.cuh"
#include "moe.cuh"

namespace qg {
namespace e8 {

using namespace tc;

constexpr int kChunk = 4;              // K steps of one slot of scales
constexpr int kSlots = 2;
constexpr int kWarpScale = 2, kWarpPromote = 4;
constexpr int kBoxRows = 32;           // tokens of one TMA box of X
constexpr int kMaxExperts = 1024;      // the tables of tiles and rows in shared memory
constexpr uint32_t kWBytes = 128 * 128;

template <int BT_>
struct Cfg8 {
    static constexpr int BT = BT_;
    static constexpr int kGroups = BT >= 256 ? 2 : 1;              // promoting warps of a lane quarter
    static constexpr int kWarps = 4 * kGroups;
    static constexpr int kThreads = 32 * (kWarpPromote + kWarps);
    static constexpr int kBufs = BT >= 256 ? 2 : 4;                // tensor-memory buffers
    static constexpr uint32_t kTmemCols = kBufs * BT < 32 ? 32 : kBufs * BT;
    static constexpr uint32_t kXBytes = BT * 128;
    static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
    static constexpr int kRedCols = BT >= 64 ? 32 : BT;            // columns of one round of the reduction
    static constexpr uint32_t kRedBytes = kRedCols * 128 * 4;
    static constexpr uint32_t kScaleBytes = kSlots * kChunk * BT * 4;
    static constexpr uint32_t kTableBytes = (3 * kMaxExperts + 2) * 4;   // first tiles [E + 1], first and last rows [E][2]
    static constexpr uint32_t kBarBytes = 512;
    static constexpr int kStages = (int)((kSmemBudget - 1024 - 256 - kRedBytes - kScaleBytes - kTableBytes - kBarBytes) / kStageBytes);
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 2;
    static constexpr uint32_t kScaleOff = kStages * kStageBytes;
    static constexpr uint32_t kRedOff = kScaleOff + kScaleBytes;
    static constexpr uint32_t kBarOff = kRedOff + kRedBytes;
    static constexpr uint32_t kTableOff = kBarOff + kBarBytes;
    static constexpr uint32_t kSmemBytes = 1024 + kTableOff + kTableBytes;
    static constexpr int kPieces = BT / 16 / kGroups;              // sixteens of columns a promoting warp holds
    static_assert(BT % 32 == 0 && BT <= 256, "whole boxes, one MMA");
    static_assert(kStages >= 3 && kNumBars * 8 + 16 <= (int)kBarBytes && kTmemCols <= 512, "");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0, "allocations are powers of two");
};

struct Args8 {
    void *Y;
    int y_type;
    const float *xs;
    const void *ws;
    const int *offsets;               // NULL: one expert, rows [0, M)
    int experts, M, O, KB, NB;        // K blocks, output tiles
    int *err;
};

// Instruction descriptor of kind::f8f6f4: f32 accumulator, e4m3 A and B (format code 0), K-major, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_e4m3(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kMmaM >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 columns of this warp's 32 lanes, to be read after tmem_landed on the same registers.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// a += (lo, hi) * f, two f32 at a time
__device__ __forceinline__ void fma2(uint64_t &a, uint32_t lo, uint32_t hi, uint64_t f) {
    asm("{.reg .b64 t; mov.b64 t, {%1, %2}; fma.rn.f32x2 %0, t, %3, %0;}" : "+l"(a) : "r"(lo), "r"(hi), "l"(f));
}
__device__ __forceinline__ float2 pair_of(uint64_t v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// Cluster helpers: the address of a local shared variable in another block, arrivals there, loads from there.
__device__ __forceinline__ uint32_t map_rank(uint32_t local, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float load_remote(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile uint32_t *abort) {
    const uint32_t a = smem_addr(bar);
    for (uint32_t it = 0; it < kSpinLimit; ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(parity)
            : "memory");
        if (done) return true;
        if ((it & 255u) == 255u && *abort) return false;
    }
    *abort = 1u;
    return false;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void store_y(const Args8 &a, size_t at, float v) {
    if (a.y_type == kF32) static_cast<float *>(a.Y)[at] = v;
    else if (a.y_type == kBf16) static_cast<uint16_t *>(a.Y)[at] = Elem<kBf16>::put(v);
    else static_cast<uint16_t *>(a.Y)[at] = Elem<kF16>::put(v);
}

struct Tile {
    int e, m0, rows, ot;              // expert, first row, its rows in the tile, output tile
};
// Tiles are numbered expert by expert, output tile by output tile, tokens
// fastest: blocks of one wave share weights.
template <int BT>
__device__ __forceinline__ Tile find_tile(const Args8 &a, const int *s_tile, const int *s_row, int t) {
    int lo = 0, hi = a.experts;       // the last e with s_tile[e] * NB <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tile[mid] * a.NB <= t) lo = mid;
        else hi = mid;
    }
    const int nt = s_tile[lo + 1] - s_tile[lo], local = t - s_tile[lo] * a.NB;
    Tile r;
    r.e = lo;
    r.ot = local / nt;
    r.m0 = s_row[2 * lo] + (local - r.ot * nt) * BT;
    r.rows = min(s_row[2 * lo + 1] - r.m0, BT);
    return r;
}

template <int BT, class SC>
__global__ void __launch_bounds__(Cfg8<BT>::kThreads, 1)
gemm_e4m3_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args8 a) {
    using C = Cfg8<BT>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    float *s_scale = reinterpret_cast<float *>(smem + C::kScaleOff);
    float *s_red = reinterpret_cast<float *>(smem + C::kRedOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *full = bars, *empty = full + C::kStages, *acc_full = empty + C::kStages, *acc_empty = acc_full + C::kBufs,
             *sc_full = acc_empty + C::kBufs, *sc_empty = sc_full + kSlots, *red_full = sc_empty + kSlots,
             *red_empty = red_full + 1;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + C::kNumBars);
    volatile uint32_t *abort = tmem_slot + 1;
    int *s_tile = reinterpret_cast<int *>(smem + C::kTableOff), *s_row = s_tile + kMaxExperts + 2;
    __shared__ int2 s_warp[C::kThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ranks, rank;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], C::kWarps);
        }
        for (int b = 0; b < kSlots; ++b) {
            mbar_init(&sc_full[b], 1);
            mbar_init(&sc_empty[b], C::kWarps);
        }
        mbar_init(red_full, ranks * C::kWarps);
        mbar_init(red_empty, ranks * C::kWarps);
        *abort = 0u;
        mbar_fence_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == kWarpMma) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr((const void *)tmem_slot)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    griddep_launch_dependents();
    // Tables of the experts' first tiles and rows.
    if (a.offsets == nullptr) {
        if (threadIdx.x == 0) {
            s_tile[0] = 0;
            s_tile[1] = (a.M + BT - 1) / BT;
            s_row[0] = 0;
            s_row[1] = a.M;
        }
    } else {
        // Row bounds held to [0, M] and to their order (a table that is
        // neither raises the error word): expert e has rows most[e] to
        // most[e+1] of the running maximum.
        int tiles_before = 0, most = min(max(a.offsets[0], 0), a.M);
        for (int e0 = 0; e0 < a.experts; e0 += C::kThreads) {
            const int e = e0 + threadIdx.x;
            int to = 0;
            if (e < a.experts) {
                const int lo = a.offsets[e], hi = a.offsets[e + 1];
                if ((lo < 0 || hi < lo || hi > a.M) && blockIdx.x == 0) raise_device_error(a.err, kErrExpert);
                to = min(max(hi, 0), a.M);
            }
            int top = to;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, top, d);
                if (lane >= d) top = max(top, y);
            }
            if (lane == 31) s_warp[warp].x = top;
            __syncthreads();
            int below = most;
            for (int w = 0; w < C::kThreads / 32; ++w) {
                if (w < warp) below = max(below, s_warp[w].x);
                most = max(most, s_warp[w].x);
            }
            int from = __shfl_up_sync(0xffffffffu, top, 1);
            from = lane == 0 ? below : max(from, below);
            to = max(top, below);
            const int n = e < a.experts ? (to - from + BT - 1) / BT : 0;
            int x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) s_warp[warp].y = x;
            __syncthreads();
            int before = tiles_before;
            for (int w = 0; w < C::kThreads / 32; ++w) {
                before += w < warp ? s_warp[w].y : 0;
                tiles_before += s_warp[w].y;
            }
            if (e < a.experts) {
                s_tile[e] = before + x - n;
                s_row[2 * e] = from;
                s_row[2 * e + 1] = to;
            }
            __syncthreads();
        }
        if (threadIdx.x == 0) s_tile[a.experts] = tiles_before;
    }
    tc_fence_before();
    __syncthreads();
    if (ranks > 1) cluster_barrier();      // every block's barriers are there before another arrives at them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int tiles = s_tile[a.experts] * a.NB, first = blockIdx.x / ranks, step = gridDim.x / ranks;
    const int k0 = (int)((long long)a.KB * rank / ranks), k1 = (int)((long long)a.KB * (rank + 1) / ranks);

    if (warp == kWarpTma) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int t = first; t < tiles; t += step) {
                const Tile L = find_tile<BT>(a, s_tile, s_row, t);
                const int boxes = (L.rows + kBoxRows - 1) / kBoxRows, wrow = L.e * a.O + L.ot * 128;
                for (int k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % C::kStages, r = it / C::kStages;
                    if (r > 0 && !mbar_wait_or_abort(&empty[s], (r & 1) ^ 1, abort))
                        raise_device_error(a.err, kErrTimeout);
                    const uint32_t st = sbase + s * C::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], kWBytes + boxes * (kBoxRows * 128));
                    tma_load_2d(st, &tmW, k * 128, wrow, &full[s]);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(st + kWBytes + b * (kBoxRows * 128), &tmX, k * 128, L.m0 + b * kBoxRows, &full[s]);
                }
            }
            // Every copy issued must have landed before the block exits.
            for (uint32_t j = it > (uint32_t)C::kStages ? it - C::kStages : 0; j < it; ++j)
                if (!mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1)) raise_device_error(a.err, kErrTimeout);
        }
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int t = first; t < tiles; t += step) {
                const Tile L = find_tile<BT>(a, s_tile, s_row, t);
                const uint32_t idesc = idesc_e4m3((L.rows + 15) & ~15);
                for (int k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % C::kStages, r = it / C::kStages, b = it % C::kBufs, rb = it / C::kBufs;
                    if (rb > 0 && !mbar_wait_or_abort(&acc_empty[b], (rb & 1) ^ 1, abort))
                        raise_device_error(a.err, kErrTimeout);
                    if (!mbar_wait_or_abort(&full[s], r & 1, abort)) raise_device_error(a.err, kErrTimeout);
                    tc_fence_after();
                    const uint32_t st = sbase + s * C::kStageBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_e4m3(tmem + b * BT, sw128_desc(st + kk * 32), sw128_desc(st + kWBytes + kk * 32), idesc,
                                 kk > 0 ? 1u : 0u);
                    mma_commit(&acc_full[b]);
                    mma_commit(&empty[s]);
                }
            }
        }
    } else if (warp == kWarpScale) {
        constexpr int kTok = BT / 32;
        uint32_t ch = 0;
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile<BT>(a, s_tile, s_row, t);
            const typename SC::T *ws = static_cast<const typename SC::T *>(a.ws) + ((size_t)L.e * a.NB + L.ot) * a.KB;
            for (int k = k0; k < k1; k += kChunk, ++ch) {
                const uint32_t s = ch % kSlots, r = ch / kSlots;
                float v[kTok][kChunk];
#pragma unroll
                for (int c = 0; c < kChunk; ++c) {
                    const float w = k + c < k1 ? SC::get(ws, k + c) : 0.f;
#pragma unroll
                    for (int i = 0; i < kTok; ++i) {
                        const int m = lane + 32 * i;
                        v[i][c] = m < L.rows && k + c < k1 ? a.xs[(size_t)(L.m0 + m) * a.KB + k + c] * w : 0.f;
                    }
                }
                if (r > 0) {
                    bool ok = true;
                    if (lane == 0) ok = mbar_wait_or_abort(&sc_empty[s], (r & 1) ^ 1, abort);
                    if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0) && lane == 0) raise_device_error(a.err, kErrTimeout);
                }
                float *dst = s_scale + s * kChunk * BT;
#pragma unroll
                for (int c = 0; c < kChunk; ++c)
#pragma unroll
                    for (int i = 0; i < kTok; ++i) dst[c * BT + lane + 32 * i] = v[i][c];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[s]);
            }
        }
    } else if (warp >= kWarpPromote) {
        const int pw = warp - kWarpPromote, q = warp & 3, grp = pw >> 2, pt = threadIdx.x - 32 * kWarpPromote;
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
        const int row = q * 32 + lane;
        uint32_t it = 0, ch = 0, round = 0;
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
            if (!mbar_wait_or_abort(bar, parity, abort) && lane == 0) raise_device_error(a.err, kErrTimeout);
            __syncwarp();
        };
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile<BT>(a, s_tile, s_row, t);
            const int pieces = (L.rows + 15) >> 4;             // sixteens of the tile; mine: grp, grp + kGroups, ...
            uint64_t acc[C::kPieces][8];
#pragma unroll
            for (int p = 0; p < C::kPieces; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[p][j] = 0;
            for (int k = k0; k < k1; ++k, ++it) {
                const int c = (k - k0) % kChunk;
                if (c == 0) wait_warp(&sc_full[ch % kSlots], (ch / kSlots) & 1);
                const uint32_t b = it % C::kBufs;
                wait_warp(&acc_full[b], (it / C::kBufs) & 1);
                tc_fence_after();
                const float *f = s_scale + ((ch % kSlots) * kChunk + c) * BT;
                uint32_t r[2][16];
                const uint32_t tb = tq + b * BT;
                if (grp < pieces) tmem_ld16_async(tb + grp * 16, r[0]);
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p) {
                    const int at = p * C::kGroups + grp;
                    if (at >= pieces) break;
                    tmem_landed(r[p & 1]);
                    if (p + 1 < C::kPieces && at + C::kGroups < pieces) tmem_ld16_async(tb + (at + C::kGroups) * 16, r[(p + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 g = *reinterpret_cast<const ulonglong2 *>(f + at * 16 + 4 * j);
                        fma2(acc[p][2 * j], r[p & 1][4 * j], r[p & 1][4 * j + 1], g.x);
                        fma2(acc[p][2 * j + 1], r[p & 1][4 * j + 2], r[p & 1][4 * j + 3], g.y);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
                if (c == kChunk - 1 || k + 1 == k1) {
                    if (lane == 0) mbar_arrive(&sc_empty[ch % kSlots]);
                    ++ch;
                }
            }
            const int o0 = L.ot * 128;
            if (ranks == 1) {
                const int o = o0 + row;
                if (o < a.O) {
#pragma unroll
                    for (int p = 0; p < C::kPieces; ++p) {
                        const int at = (p * C::kGroups + grp) * 16;
                        const size_t y = (size_t)(L.m0 + at) * a.O + o;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 v = pair_of(acc[p][j]);
                            if (at + 2 * j < L.rows) store_y(a, y + (size_t)(2 * j) * a.O, v.x);
                            if (at + 2 * j + 1 < L.rows) store_y(a, y + (size_t)(2 * j + 1) * a.O, v.y);
                        }
                    }
                }
                continue;
            }
            // Rounds of kRedCols columns: every block's sums into its shared
            // memory, then each rank adds its share of the columns over all
            // blocks, in rank order, and stores it.
            constexpr int kPer = C::kRedCols / 16 / C::kGroups;   // pieces a warp brings to a round
#pragma unroll
            for (int rd = 0; rd < BT / C::kRedCols; ++rd) {
                if (rd * C::kRedCols >= L.rows) break;
                if (round > 0) {
                    if (!wait_cluster(red_empty, (round - 1) & 1, abort) && lane == 0) raise_device_error(a.err, kErrTimeout);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int p = rd * kPer + i, col = (i * C::kGroups + grp) * 16;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = pair_of(acc[p][j]);
                        s_red[(col + 2 * j) * 128 + row] = v.x;
                        s_red[(col + 2 * j + 1) * 128 + row] = v.y;
                    }
                }
                __syncwarp();
                if (lane < (int)ranks) arrive_remote(map_rank(smem_addr(red_full), lane));
                if (!wait_cluster(red_full, round & 1, abort) && lane == 0) raise_device_error(a.err, kErrTimeout);
                __syncwarp();
                const int o = o0 + (pt & 127);
                for (int col = (int)rank + (pt >> 7) * (int)ranks; col < C::kRedCols; col += C::kGroups * (int)ranks) {
                    const int m = rd * C::kRedCols + col;
                    if (m >= L.rows) break;
                    const uint32_t local = smem_addr(s_red + col * 128 + (pt & 127));
                    float sum = 0.f;
                    for (int r = 0; r < (int)ranks; ++r) sum += load_remote(map_rank(local, r));
                    if (o < a.O) store_y(a, (size_t)(L.m0 + m) * a.O + o, sum);
                }
                __syncwarp();
                if (lane < (int)ranks) arrive_remote(map_rank(smem_addr(red_empty), lane));
                ++round;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols)
                     : "memory");
    }
    if (ranks > 1) cluster_barrier();      // no block leaves while another reads its sums
}

// Host side.

struct Plan8 {
    int bt, cluster, blocks;
};

template <int BT, class SC>
const void *kernel_of() { return reinterpret_cast<const void *>(gemm_e4m3_kernel<BT, SC>); }

// Clusters of 2, 4 or 8 blocks that run at once (both scale types take the
// same registers and shared memory).
int clusters_at_once(int bt, int cluster) {
    static PerContext<int> cache[4][3];
    const int i = bt == 32 ? 0 : bt == 64 ? 1 : bt == 128 ? 2 : 3, j = cluster == 2 ? 0 : cluster == 4 ? 1 : 2;
    int n = 0;
    const int rc = cache[i][j].get(&n, [&](int *out) {
        const void *k = i == 0 ? kernel_of<32, ScaleF32>() : i == 1 ? kernel_of<64, ScaleF32>()
                      : i == 2 ? kernel_of<128, ScaleF32>() : kernel_of<256, ScaleF32>();
        const uint32_t smem = i == 0 ? Cfg8<32>::kSmemBytes : i == 1 ? Cfg8<64>::kSmemBytes
                            : i == 2 ? Cfg8<128>::kSmemBytes : Cfg8<256>::kSmemBytes;
        set_max_dynamic_smem(k, (int)smem);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cluster);
        cfg.blockDim = dim3(i == 3 ? Cfg8<256>::kThreads : Cfg8<32>::kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(out, k, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return (int)kECuda;
        }
        return (int)kOk;
    });
    return rc == kOk ? n : 0;
}

inline Plan8 plan(int M, int I, int O, int experts) {
    const int P = num_sms(), KB = (I + 127) / 128, NB = (O + 127) / 128;
    Plan8 p;
    // as wide as the experts' rows would be in even shares, and twice that, as they are not even
    const int filled = std::min(experts, M);
    const long long want = experts == 1 ? M : 2LL * ((M + filled - 1) / filled);
    p.bt = want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : 256;
    const double tiles = (double)NB * (experts == 1 ? (M + p.bt - 1) / p.bt : filled + M / p.bt);
    // cycles of a K step and of one round of the reduction over a cluster
    const double step = p.bt == 256 ? 600.0 : 500.0, rounds = p.bt >= 64 ? p.bt / 32 : 1;
    double best = 0;
    for (int c = 1; c <= 8; c *= 2) {
        if (c > 1 && KB < 4 * c) break;
        const int n = c == 1 ? P : clusters_at_once(p.bt, c);
        if (n < 1) break;
        const double waves = std::ceil(tiles / n);
        const double cost = waves * (((KB + c - 1) / c) * step + (c > 1 ? 1500.0 * rounds : 0.0) + 1500.0);
        if (c == 1 || cost < best) {
            best = cost;
            p.cluster = c;
            p.blocks = n * c;
        }
    }
    return p;
}

inline bool encode_map(CUtensorMap *m, const void *p, long long rows, int I, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)I, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)I};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT, class SC>
int launch(const char *what, const Plan8 &p, const CUtensorMap &w, const CUtensorMap &x, const Args8 &a, cudaStream_t st) {
    using C = Cfg8<BT>;
    set_max_dynamic_smem(reinterpret_cast<const void *>(gemm_e4m3_kernel<BT, SC>), (int)C::kSmemBytes);
    return launch_clusters(what, gemm_e4m3_kernel<BT, SC>, p.blocks, C::kThreads, p.cluster, C::kSmemBytes, st, w, x, a);
}

template <class SC>
int launch_bt(const char *what, const Plan8 &p, const CUtensorMap &w, const CUtensorMap &x, const Args8 &a, cudaStream_t st) {
    switch (p.bt) {
        case 32: return launch<32, SC>(what, p, w, x, a, st);
        case 64: return launch<64, SC>(what, p, w, x, a, st);
        case 128: return launch<128, SC>(what, p, w, x, a, st);
        default: return launch<256, SC>(what, p, w, x, a, st);
    }
}

}  // namespace e8

bool gemm_e4m3_tc_takes(const E4m3Args &a) {
    const long long wrows = (long long)a.experts * a.O;
    const long long tiles = ((long long)a.M / 32 + a.experts) * ((a.O + 127) / 128);
    return a.I % 16 == 0 && (uintptr_t)a.X % 16 == 0 && (uintptr_t)a.w % 16 == 0 && a.experts <= e8::kMaxExperts &&
           wrows < (1ll << 31) - 256 && tiles < (1ll << 31) - 65536;
}

int run_gemm_e4m3_tc(const E4m3Args &g, cudaStream_t st) {
    const char *what = g.offsets ? "qgemm_e4m3_moe" : "qgemm_e4m3";
    if (!tc::encode_fn()) QG_REFUSE(kECuda, "%s: cuTensorMapEncodeTiled is not available from the driver", what);
    CUtensorMap w, x;
    if (!e8::encode_map(&w, g.w, (long long)g.experts * g.O, g.I, 128) || !e8::encode_map(&x, g.X, g.M, g.I, e8::kBoxRows))
        QG_REFUSE(kECuda, "%s: tensor map refused", what);
    const e8::Plan8 p = e8::plan(g.M, g.I, g.O, g.experts);
    const e8::Args8 a{g.Y, g.y_type, g.x_scale, g.w_scale, g.offsets, g.experts, g.M, g.O,
                      (g.I + 127) / 128, (g.O + 127) / 128, g.err};
    return g.w_power ? e8::launch_bt<ScaleE8M0>(what, p, w, x, a, st) : e8::launch_bt<ScaleF32>(what, p, w, x, a, st);
}

}  // namespace qg
