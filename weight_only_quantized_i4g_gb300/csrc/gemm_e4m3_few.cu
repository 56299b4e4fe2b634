// gemm_e4m3_few.cu -- products of e4m3 activations with e4m3 weights, few
// tokens an expert: the weights' bytes bound it.
//
// A tile is 128 outputs (rows of W, MMA M) by up to BT tokens of one expert
// (MMA N, as many as the tile has, in sixteens), so a token costs an MMA of
// sixteen and not of 128.  The outputs of a tile share one weight scale, and
// the product of both scales comes from shared memory, a token each.  One
// persistent thread block per SM:
//   warp 0      TMA producer: per K block the 128 x 128 codes of W and BT x
//               128 of X, both 128-byte swizzled
//   warps 1, 2  issue the MMAs, a thread each, stages in turn
//   warp 3      the scales' products, kChunk K blocks at a time
//   warps 4..   promote: tensor-memory lanes 32 (w % 4) .. + 31, columns
//               shared by the one or two warps of a lane quarter
// Calls of few tiles split K over the blocks of a cluster, which add their
// sums over distributed shared memory, in rank order.
#include "gemm_e4m3_tc.cuh"

namespace qg {
namespace e8 {

constexpr int kChunk = 4, kSlots = 2;  // K blocks of one slot of scales
constexpr int kWarpScale = 3, kWarpPromote = 4;
constexpr uint32_t kWBytes = 128 * 128;
constexpr int kRedStride = 132;        // words between the columns of a reduction: the fragments' rows and columns meet no bank twice
constexpr int kOutStride = 80;         // bytes between the tokens of a 32-output strip on its way out, for the same reason

template <int BT_>
struct Cfg8 {
    static constexpr int BT = BT_;
    static constexpr int kBlocks = BT <= 64 ? 2 : 1;               // K blocks of a stage
    static constexpr int kGroups = BT >= 128 ? 2 : 1;              // promoting warps of a lane quarter
    static constexpr int kWarps = 4 * kGroups;
    static constexpr int kThreads = 32 * (kWarpPromote + kWarps);
    static constexpr int kBufs = 4;                                // tensor-memory buffers, one a stage
    static constexpr int kBufCols = kBlocks * BT;
    static constexpr uint32_t kTmemCols = kBufs * kBufCols;
    static constexpr uint32_t kXBytes = BT * 128;
    static constexpr uint32_t kBlockBytes = kWBytes + kXBytes;
    static constexpr uint32_t kStageBytes = kBlocks * kBlockBytes;
    static constexpr int kRedCols = 32;                            // columns of one round of the reduction
    static constexpr uint32_t kRedBytes = kRedCols * kRedStride * 4;
    static constexpr uint32_t kScaleBytes = kSlots * kChunk * BT * 4;
    static constexpr uint32_t kBarBytes = 512;
    static constexpr int kStages = (int)((kSmemBudget - 1024 - 256 - kRedBytes - kScaleBytes - kTableBytes - kBarBytes) / kStageBytes);
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 2 * kSlots + 2;
    static constexpr uint32_t kScaleOff = kStages * kStageBytes;
    static constexpr uint32_t kRedOff = kScaleOff + kScaleBytes;
    static constexpr uint32_t kBarOff = kRedOff + kRedBytes;
    static constexpr uint32_t kTableOff = kBarOff + kBarBytes;
    static constexpr uint32_t kSmemBytes = 1024 + kTableOff + kTableBytes;
    static constexpr int kCols = BT < 64 ? BT : 64;                // columns a promoting warp loads at once
    static constexpr int kPieces = BT / kCols / kGroups;           // such pieces it holds
    static_assert(BT % 32 == 0 && BT <= 128, "one box of X, one MMA");
    static_assert(kStages >= 3 && kNumBars * 8 + 16 <= (int)kBarBytes && kTmemCols <= 512 && kTmemCols >= 32, "");
    static_assert((kTmemCols & (kTmemCols - 1)) == 0, "allocations are powers of two");
    // A wait tells one phase of a barrier from the next, not from the one
    // after that, so a stage must always be the same issuer's: with an odd
    // number of stages one thread could pass on a phase that the other had
    // not seen begin.
    static_assert(kStages % 2 == 0 && kBufs % 2 == 0, "a stage and a buffer belong to the same issuer every time");
    static_assert(kWarps * 16 * kOutStride <= (int)kRedBytes, "a strip of 16 tokens a warp on its way out");
};

// 8 R columns of 16 tensor-memory lanes, to be read after tmem_landed on the
// same registers: of columns 8 i + 2 (lane % 4) + {0, 1}, registers 4 i and
// 4 i + 1 hold tensor-memory lane lane / 4 and the next two lane / 4 + 8.
template <int R>
struct Frag {
    uint32_t r[4 * R];
};
__device__ __forceinline__ void tmem_load(uint32_t taddr, Frag<4> &f) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(f.r[0]), "=r"(f.r[1]), "=r"(f.r[2]), "=r"(f.r[3]), "=r"(f.r[4]), "=r"(f.r[5]), "=r"(f.r[6]),
          "=r"(f.r[7]), "=r"(f.r[8]), "=r"(f.r[9]), "=r"(f.r[10]), "=r"(f.r[11]), "=r"(f.r[12]), "=r"(f.r[13]),
          "=r"(f.r[14]), "=r"(f.r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, Frag<8> &f) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(f.r[0]), "=r"(f.r[1]), "=r"(f.r[2]), "=r"(f.r[3]), "=r"(f.r[4]), "=r"(f.r[5]), "=r"(f.r[6]),
          "=r"(f.r[7]), "=r"(f.r[8]), "=r"(f.r[9]), "=r"(f.r[10]), "=r"(f.r[11]), "=r"(f.r[12]), "=r"(f.r[13]),
          "=r"(f.r[14]), "=r"(f.r[15]), "=r"(f.r[16]), "=r"(f.r[17]), "=r"(f.r[18]), "=r"(f.r[19]),
          "=r"(f.r[20]), "=r"(f.r[21]), "=r"(f.r[22]), "=r"(f.r[23]), "=r"(f.r[24]), "=r"(f.r[25]),
          "=r"(f.r[26]), "=r"(f.r[27]), "=r"(f.r[28]), "=r"(f.r[29]), "=r"(f.r[30]), "=r"(f.r[31])
        : "r"(taddr));
}
// Waits for the loads; the registers pass through, so that nothing reads them before.
__device__ __forceinline__ void tmem_landed(Frag<4> &f) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(f.r[0]), "+r"(f.r[1]), "+r"(f.r[2]), "+r"(f.r[3]), "+r"(f.r[4]), "+r"(f.r[5]), "+r"(f.r[6]),
                   "+r"(f.r[7]), "+r"(f.r[8]), "+r"(f.r[9]), "+r"(f.r[10]), "+r"(f.r[11]), "+r"(f.r[12]),
                   "+r"(f.r[13]), "+r"(f.r[14]), "+r"(f.r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_landed(Frag<8> &f) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(f.r[0]), "+r"(f.r[1]), "+r"(f.r[2]), "+r"(f.r[3]), "+r"(f.r[4]), "+r"(f.r[5]), "+r"(f.r[6]),
                   "+r"(f.r[7]), "+r"(f.r[8]), "+r"(f.r[9]), "+r"(f.r[10]), "+r"(f.r[11]), "+r"(f.r[12]),
                   "+r"(f.r[13]), "+r"(f.r[14]), "+r"(f.r[15]), "+r"(f.r[16]), "+r"(f.r[17]), "+r"(f.r[18]),
                   "+r"(f.r[19]), "+r"(f.r[20]), "+r"(f.r[21]), "+r"(f.r[22]), "+r"(f.r[23]), "+r"(f.r[24]),
                   "+r"(f.r[25]), "+r"(f.r[26]), "+r"(f.r[27])
                 :
                 : "memory");
    asm volatile("" : "+r"(f.r[28]), "+r"(f.r[29]), "+r"(f.r[30]), "+r"(f.r[31])::"memory");
}
// Four 8 x 8 matrices of 16-bit fragments, transposed: row lane % 8 of matrix lane / 8 goes to this lane's address.
__device__ __forceinline__ void stmatrix4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
template <int BT, class SC>
__global__ void __launch_bounds__(Cfg8<BT>::kThreads, 1)
gemm_e4m3_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args8 a) {
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
        tmem_alloc(tmem_slot, C::kTmemCols);
    }
    griddep_wait();
    griddep_launch_dependents();
    build_tables<BT, C::kThreads>(a, s_tile, s_row, s_warp);
    tc_fence_before();
    __syncthreads();
    if (ranks > 1) cluster_barrier();      // every block's barriers are there before another arrives at them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int tiles = s_tile[a.experts] * a.NT, first = blockIdx.x / ranks, step = gridDim.x / ranks;
    const int k0 = (int)((long long)a.KB * rank / ranks), k1 = (int)((long long)a.KB * (rank + 1) / ranks);

    // Every lane waits: with one lane's wait and a vote the warp goes on 170 cycles later.
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
        mbar_wait_or_abort(bar, parity, abort);        // a wait that gives up sets *abort, which the block's end reports
        __syncwarp();
    };
    if (warp == kWarpTma) {
        uint32_t it = 0;
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile_warp<BT>(a, s_tile, s_row, t);
            const int wrow = L.e * a.O + L.ot * 128;
            for (int k = k0; k < k1; k += C::kBlocks, ++it) {
                const uint32_t s = it % C::kStages, r = it / C::kStages;
                const int n = min(C::kBlocks, k1 - k);
                if (r > 0) wait_warp(&empty[s], (r & 1) ^ 1);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], n * C::kBlockBytes);
                    for (int j = 0; j < n; ++j) {
                        const uint32_t st = sbase + s * C::kStageBytes + j * C::kBlockBytes;
                        tma_load_2d(st, &tmW, (k + j) * 128, wrow, &full[s]);
                        tma_load_2d(st + kWBytes, &tmX, (k + j) * 128, L.m0, &full[s]);
                    }
                }
                __syncwarp();
            }
        }
        // Every copy issued must have landed, and every commit arrived, before the block exits.
        for (uint32_t j = it > (uint32_t)C::kStages ? it - C::kStages : 0; j < it; ++j) {
            wait_warp(&full[j % C::kStages], (j / C::kStages) & 1);
            wait_warp(&empty[j % C::kStages], (j / C::kStages) & 1);
        }
    } else if (warp == kWarpMma || warp == kWarpMma2) {
        // No stage's sums depend on another's, so two warps issue them in
        // turn: each one's waits and commits pass while the other's MMAs run.
        uint32_t it = 0;
        const uint32_t mine = warp == kWarpMma ? 0u : 1u, lo = desc_lo(sbase);
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile_warp<BT>(a, s_tile, s_row, t);
            const uint32_t idesc = idesc_e4m3((L.rows + 15) & ~15);
            for (int k = k0; k < k1; k += C::kBlocks, ++it) {
                if ((it & 1u) != mine) continue;
                const uint32_t s = it % C::kStages, r = it / C::kStages, b = it % C::kBufs, rb = it / C::kBufs;
                const int n = min(C::kBlocks, k1 - k);
                wait_warp(&full[s], r & 1);
                if (rb > 0) wait_warp(&acc_empty[b], (rb & 1) ^ 1);
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t w_lo = lo + s * (C::kStageBytes >> 4);
#pragma unroll
                    for (int j = 0; j < C::kBlocks; ++j) {
                        if (j >= n) break;
                        mma_block(tmem + b * C::kBufCols + j * BT, w_lo + j * (C::kBlockBytes >> 4),
                                  w_lo + (j * C::kBlockBytes + kWBytes) / 16, idesc);
                    }
                    mma_commit(&acc_full[b]);
                    mma_commit(&empty[s]);
                }
                __syncwarp();
            }
        }
    } else if (warp == kWarpScale) {
        constexpr int kTok = BT / 32;
        uint32_t ch = 0;
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile_warp<BT>(a, s_tile, s_row, t);
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
                    wait_warp(&sc_empty[s], (r & 1) ^ 1);
                }
                float *dst = s_scale + s * kChunk * BT + lane;
#pragma unroll
                for (int c = 0; c < kChunk; ++c)
#pragma unroll
                    for (int i = 0; i < kTok; ++i) dst[c * BT + 32 * i] = v[i][c];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[s]);
            }
        }
    } else if (warp >= kWarpPromote) {
        const int pw = warp - kWarpPromote, q = warp & 3, grp = pw >> 2, pt = threadIdx.x - 32 * kWarpPromote;
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
        const int row = q * 32 + (lane >> 2), cl = 2 * (lane & 3);   // of the fragments: rows row + 8 i, columns 8 j + cl, + 1
        constexpr int kF = C::kCols / 8;
        uint32_t it = 0, ch = 0, round = 0;
        for (int t = first; t < tiles; t += step) {
            const Tile L = find_tile_warp<BT>(a, s_tile, s_row, t);
            // piece p: columns (p * kGroups + grp) * kCols; sums [upper half of the rows][fragment][row + 8]
            uint64_t acc[C::kPieces][2][kF][2];
#pragma unroll
            for (int p = 0; p < C::kPieces; ++p)
#pragma unroll
                for (int j = 0; j < kF; ++j) acc[p][0][j][0] = acc[p][0][j][1] = acc[p][1][j][0] = acc[p][1][j][1] = 0;
            for (int k = k0; k < k1; k += C::kBlocks, ++it) {
                const uint32_t b = it % C::kBufs;
#pragma unroll
                for (int x = 0; x < C::kBlocks; ++x) {
                    if (x > 0 && k + x >= k1) break;
                    const int c = (k + x - k0) % kChunk;
                    if (c == 0) wait_warp(&sc_full[ch % kSlots], (ch / kSlots) & 1);
                    if (x == 0) {
                        wait_warp(&acc_full[b], (it / C::kBufs) & 1);
                        tc_fence_after();
                    }
                    const float *f = s_scale + ((ch % kSlots) * kChunk + c) * BT + cl;
#pragma unroll
                    for (int p = 0; p < C::kPieces; ++p) {
                        const int col = (p * C::kGroups + grp) * C::kCols;
                        if (col < L.rows) {
                            Frag<kF> lo, hi;
                            const uint32_t ta = tq + b * C::kBufCols + x * BT + col;
                            tmem_load(ta, lo);
                            tmem_load(ta + (16u << 16), hi);
                            uint64_t g[kF];
#pragma unroll
                            for (int j = 0; j < kF; ++j) g[j] = *reinterpret_cast<const uint64_t *>(f + col + 8 * j);
                            tmem_landed(lo);
                            tmem_landed(hi);
#pragma unroll
                            for (int j = 0; j < kF; ++j) {
                                fma2(acc[p][0][j][0], lo.r[4 * j], lo.r[4 * j + 1], g[j]);
                                fma2(acc[p][0][j][1], lo.r[4 * j + 2], lo.r[4 * j + 3], g[j]);
                                fma2(acc[p][1][j][0], hi.r[4 * j], hi.r[4 * j + 1], g[j]);
                                fma2(acc[p][1][j][1], hi.r[4 * j + 2], hi.r[4 * j + 3], g[j]);
                            }
                        }
                    }
                    if (c == kChunk - 1 || k + x + 1 == k1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_empty[ch % kSlots]);
                        ++ch;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
            }
            const int o0 = L.ot * 128;
            if (ranks == 1) {
                if (a.y_type == kF32) {
                    // a warp's store: eight outputs, one sector, of four tokens
                    float *y = static_cast<float *>(a.Y) + (size_t)L.m0 * a.O + o0 + row;
#pragma unroll
                    for (int p = 0; p < C::kPieces; ++p)
#pragma unroll
                        for (int j = 0; j < kF; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int m = (p * C::kGroups + grp) * C::kCols + 8 * j + cl;
                                const float2 v = pair_of(acc[p][i >> 1][j][i & 1]);
                                if (o0 + row + 8 * i < a.O) {
                                    if (m < L.rows) y[(size_t)m * a.O + 8 * i] = v.x;
                                    if (m + 1 < L.rows) y[(size_t)(m + 1) * a.O + 8 * i] = v.y;
                                }
                            }
                    continue;
                }
                // 16-bit types: sixteen tokens of this warp's 32 outputs at a
                // time, transposed through shared memory to 64 bytes a token.
                const uint32_t strip = smem_addr(s_red) + pw * 16 * kOutStride;
                const int ow = o0 + q * 32, part = lane & 3;
                const bool lines = a.O % 8 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p)
#pragma unroll
                    for (int j = 0; j < kF; j += 2) {
                        const int m = (p * C::kGroups + grp) * C::kCols + 8 * j;
                        if (m >= L.rows) continue;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 v = pair_of(acc[p][i >> 1][j + x][i & 1]);
                                w[i] = pack_16(a.y_type, v.x, v.y);
                            }
                            // matrix i (outputs 8 i ..): row lane % 8 is token 8 x + lane % 8
                            stmatrix4_trans(strip + (8 * x + (lane & 7)) * kOutStride + (lane >> 3) * 16, w[0], w[1], w[2], w[3]);
                        }
                        __syncwarp();
                        const char *from = reinterpret_cast<const char *>(s_red) + pw * 16 * kOutStride;
                        uint16_t *y = static_cast<uint16_t *>(a.Y) + (size_t)(L.m0 + m) * a.O + ow;
                        if (lines) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int tok = 8 * x + (lane >> 2);
                                if (m + tok < L.rows && ow + part * 8 < a.O)
                                    *reinterpret_cast<uint4 *>(y + (size_t)tok * a.O + part * 8) =
                                        *reinterpret_cast<const uint4 *>(from + tok * kOutStride + part * 16);
                            }
                        } else if (ow + lane < a.O) {      // neighbouring lanes, neighbouring outputs
                            const int n = min(L.rows - m, 16);
#pragma unroll 4
                            for (int tok = 0; tok < n; ++tok)
                                y[(size_t)tok * a.O + lane] = *reinterpret_cast<const uint16_t *>(from + tok * kOutStride + 2 * lane);
                        }
                        __syncwarp();
                    }
                continue;
            }
            // Rounds of kRedCols columns: every block's sums into its shared
            // memory, then each rank adds its share of the columns over all
            // blocks, in rank order, and stores it.
            constexpr int kRounds = C::kCols / C::kRedCols;       // of a piece
#pragma unroll
            for (int rd = 0; rd < BT / C::kRedCols; ++rd) {
                if (rd * C::kRedCols >= L.rows) break;
                if (round > 0) {
                    wait_cluster(red_empty, (round - 1) & 1, abort);
                    __syncwarp();
                }
                // the round's columns are one group's
                const int piece = rd / kRounds, p = piece / C::kGroups, j0 = rd % kRounds * (C::kRedCols / 8);
                if (piece % C::kGroups == grp) {
#pragma unroll
                    for (int j = 0; j < C::kRedCols / 8; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 v = pair_of(acc[p][i >> 1][j0 + j][i & 1]);
                            s_red[(8 * j + cl) * kRedStride + row + 8 * i] = v.x;
                            s_red[(8 * j + cl + 1) * kRedStride + row + 8 * i] = v.y;
                        }
                }
                __syncwarp();
                if (lane < (int)ranks) arrive_remote(map_rank(smem_addr(red_full), lane));
                wait_cluster(red_full, round & 1, abort);
                __syncwarp();
                const int o = o0 + (pt & 127);
                for (int col = (int)rank + (pt >> 7) * (int)ranks; col < C::kRedCols; col += C::kGroups * (int)ranks) {
                    const int m = rd * C::kRedCols + col;
                    if (m >= L.rows) break;
                    const uint32_t local = smem_addr(s_red + col * kRedStride + (pt & 127));
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
    if (threadIdx.x == 0 && *abort) raise_device_error(a.err, kErrTimeout);
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_free(tmem, C::kTmemCols);
    }
    if (ranks > 1) cluster_barrier();      // no block leaves while another reads its sums
}

// Host side.

template <class SC, class F>
int by_width(int bt, F f) {
    switch (bt) {
        case 32: return f(gemm_e4m3_few_kernel<32, SC>, Cfg8<32>());
        case 64: return f(gemm_e4m3_few_kernel<64, SC>, Cfg8<64>());
        default: return f(gemm_e4m3_few_kernel<128, SC>, Cfg8<128>());
    }
}

// Both scale types take the same registers and shared memory.
int clusters_at_once(int bt, int cluster) {
    static PerContext<int> cache[3][3];
    if (cluster == 1) return num_sms();
    int n = 0;
    const int rc = cache[bt == 32 ? 0 : bt == 64 ? 1 : 2][cluster == 2 ? 0 : cluster == 4 ? 1 : 2].get(&n, [&](int *out) {
        return by_width<ScaleF32>(bt, [&](auto kernel, auto cfg) {
            using C = decltype(cfg);
            return count_clusters(kernel, C::kThreads, C::kSmemBytes, cluster, out);
        });
    });
    return rc == kOk ? n : 0;
}

FewPlan plan_few(int M, int I, int O, int experts) {
    const int KB = (I + 127) / 128, NB = (O + 127) / 128;
    // as wide as the experts' rows would be in even shares, and twice that, as they are not even
    const int filled = std::min(experts, M);
    const long long want = experts == 1 ? M : 2LL * ((M + filled - 1) / filled);
    FewPlan best{want <= 32 ? 32 : want <= 64 ? 64 : 128, 1, 0, 0.0};
    const double tiles = NB * token_tiles(M, experts, best.bt);
    for (int c = 1; c <= 8; c *= 2) {
        if (c > 1 && KB < 4 * c) break;
        const int n = clusters_at_once(best.bt, c);
        if (n < 1) break;
        // cycles of a K block, as measured with full tiles (32 tokens: what
        // 16 KB of weights take an SM at the card's bandwidth), and of one
        // round of the reduction over a cluster, which takes longer: with 2500
        // the estimate for 64 rows of 2048 x 7168 is 6 us and the call takes 17
        const double step = best.bt == 128 ? 1370.0 : best.bt == 64 ? 800.0 : 700.0, rounds = best.bt / 32;
        const double waves = std::ceil(tiles / n);
        const double cost = waves * (((KB + c - 1) / c) * step + (c > 1 ? 2500.0 * rounds : 0.0) + 1500.0);
        if (c == 1 || cost < best.cost) best = FewPlan{best.bt, c, n * c, cost};
    }
    return best;
}

template <class SC>
int launch_few_as(const char *what, const FewPlan &p, const CUtensorMap &w, const CUtensorMap &x, const Args8 &a,
                  cudaStream_t st) {
    return by_width<SC>(p.bt, [&](auto kernel, auto cfg) {
        using C = decltype(cfg);
        set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)C::kSmemBytes);
        return launch_clusters(what, kernel, p.blocks, C::kThreads, p.cluster, C::kSmemBytes, st, w, x, a);
    });
}

int launch_few(const char *what, const FewPlan &p, const E4m3Args &g, Args8 a, cudaStream_t st) {
    CUtensorMap w, x;
    if (!encode_map(&w, g.w, (long long)g.experts * g.O, g.I, 128) || !encode_map(&x, g.X, g.M, g.I, p.bt))
        QG_REFUSE(kECuda, "%s: tensor map refused", what);
    a.NT = a.NB;
    return g.w_power ? launch_few_as<ScaleE8M0>(what, p, w, x, a, st) : launch_few_as<ScaleF32>(what, p, w, x, a, st);
}

}  // namespace e8
}  // namespace qg
