// gemm_e4m3_many.cu -- products of e4m3 activations with e4m3 weights, many
// tokens an expert: the tensor cores and what feeds and empties them bound it.
//
// A tile is 128 tokens (MMA M) by 256 or 192 outputs, two halves of N = 128 or
// 96, so a promoting thread holds one token and scales 32 columns by one
// factor.  (With the tokens along N a factor a column has to be read from
// shared memory: 64 columns then take a warp 290 cycles instead of 134, and a
// K block 1800 instead of the MMAs' 512.)  Shared memory bounds it: a K block's
// MMAs read 64 KB and TMA writes 48, which takes 875 cycles at 128 bytes a
// cycle; it takes 880.  Block pairs that share an MMA (half the weights a
// block) were built and measured 0 to 10% slower: their signals cross SMs.
// One persistent thread block per SM:
//   warps 0, 1   TMA producers, K blocks in turn: 128 x 128 codes of X and both
//                halves' of W, 128-byte swizzled
//   warps 2..5   issue the MMAs, each every second K block of one half; its four leave the half's sums in one of four
//                buffers (one producer and two issuers took 81 us where these
//                take 50, without the promotion)
//   warps 8..15  promote: tensor-memory lanes 32 (w % 4) .. + 31, one half
//                each, so that a scheduler's two warps are at different points
//                of their K blocks; a thread loads its token's scales and its
//                half's (of the one or two 128-blocks it lies in) four K blocks
//                ahead
#include "gemm_e4m3_tc.cuh"

namespace qg {
namespace e8 {
namespace {

constexpr int kPrefetchAhead = 8;
constexpr int kAhead = 4;              // K blocks of scales in a thread's registers
constexpr int kWarpIssue = 2, kWarpPromote = 4, kWarps = 8, kThreads = 32 * (kWarpPromote + kWarps);
constexpr int kBufs = 2;               // tensor-memory buffers of 256 columns
constexpr int kOutStride = 80;         // bytes between the tokens (64 each) of a strip on its way out: eight lanes' 16 bytes meet no bank twice

template <int HALF>                    // outputs of half a tile
struct CfgMany {
    static constexpr uint32_t kXBytes = 128 * 128, kWBytes = HALF * 128;
    static constexpr uint32_t kStageBytes = kXBytes + 2 * kWBytes;
    static constexpr uint32_t kOutAll = kWarps * 16 * kOutStride;   // strips of 16 tokens
    static constexpr uint32_t kBarBytes = 256;
    static constexpr int kStages = ~1 & (int)((kSmemBudget - 1024 - 256 - kOutAll - kTableBytes - kBarBytes) / kStageBytes);
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs;
    static constexpr uint32_t kOutOff = kStages * kStageBytes;
    static constexpr uint32_t kBarOff = kOutOff + kOutAll;
    static constexpr uint32_t kTableOff = kBarOff + kBarBytes;
    static constexpr uint32_t kSmemBytes = 1024 + kTableOff + kTableBytes;
    static_assert(kStages >= 3 && kNumBars * 8 + 16 <= (int)kBarBytes, "");
    // A wait tells one phase of a barrier from the next, not from the one
    // after that, so a stage must always be the same warps': with an odd
    // number of stages one could pass on a phase that the other had not seen
    // begin.
    static_assert(kStages % 2 == 0 && kBufs == 2, "a stage and a buffer belong to the same producer and issuer every time");
};

// 32 columns of this warp's 32 lanes, to be read after landed() on the same registers.
struct Sums {
    uint32_t r[32];
};
__device__ __forceinline__ void load(uint32_t taddr, Sums &s) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19,"
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(s.r[0]), "=r"(s.r[1]), "=r"(s.r[2]), "=r"(s.r[3]), "=r"(s.r[4]), "=r"(s.r[5]), "=r"(s.r[6]),
          "=r"(s.r[7]), "=r"(s.r[8]), "=r"(s.r[9]), "=r"(s.r[10]), "=r"(s.r[11]), "=r"(s.r[12]),
          "=r"(s.r[13]), "=r"(s.r[14]), "=r"(s.r[15]), "=r"(s.r[16]), "=r"(s.r[17]), "=r"(s.r[18]),
          "=r"(s.r[19]), "=r"(s.r[20]), "=r"(s.r[21]), "=r"(s.r[22]), "=r"(s.r[23]), "=r"(s.r[24]),
          "=r"(s.r[25]), "=r"(s.r[26]), "=r"(s.r[27]), "=r"(s.r[28]), "=r"(s.r[29]), "=r"(s.r[30]),
          "=r"(s.r[31])
        : "r"(taddr));
}
// Sixteen registers pass through, so that nothing reads them before.
__device__ __forceinline__ void pass(uint32_t *r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void landed(Sums &s) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    pass(s.r);
    pass(s.r + 16);
}

template <int HALF, class SC>
__global__ void __launch_bounds__(kThreads, 1)
gemm_e4m3_many_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args8 a) {
    using C = CfgMany<HALF>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *full = bars, *empty = full + C::kStages, *acc_full = empty + C::kStages, *acc_empty = acc_full + kBufs;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + C::kNumBars);
    volatile uint32_t *abort = tmem_slot + 1;
    int *s_tile = reinterpret_cast<int *>(smem + C::kTableOff), *s_row = s_tile + kMaxExperts + 2;
    __shared__ int2 s_warp[kThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kWarps);
        }
        *abort = 0u;
        mbar_fence_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmW)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmX)) : "memory");
    }
    if (warp == kWarpIssue) {
        __syncwarp();
        tmem_alloc(tmem_slot, kBufs * 256);
    }
    griddep_wait();
    griddep_launch_dependents();
    build_tables<128, kThreads>(a, s_tile, s_row, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = s_tile[a.experts] * a.NT, first = blockIdx.x, step = gridDim.x;

    // 384 threads start with 168 registers each, 64512 in all, of which the
    // promoting warps take 8 x 32 x 224 and the others 4 x 32 x 56.
    // Every lane waits: with one lane's wait and a vote the warp goes on 170 cycles later.
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
        if (!mbar_wait_or_abort(bar, parity, abort) && lane == 0) raise_device_error(a.err, kErrTimeout);
        __syncwarp();
    };
    if (warp < kWarpPromote) {
        regs_down<56>();
        if (warp < kWarpIssue) {
            uint32_t it = 0;
            for (int t = first; t < tiles; t += step) {
                const Tile L = find_tile<128>(a, s_tile, s_row, t);
                const int wrow = L.e * a.O + L.ot * 2 * HALF;
                for (int k = 0; k < a.KB; ++k, ++it) {
                    if ((it & 1u) != (uint32_t)warp) continue;
                    const uint32_t s = it % C::kStages, r = it / C::kStages;
                    if (r > 0) wait_warp(&empty[s], (r & 1) ^ 1);
                    if (lane == 0) {
                        const uint32_t st = sbase + s * C::kStageBytes;
                        mbar_arrive_expect_tx(&full[s], C::kStageBytes);
                        tma_load_2d(st, &tmX, k * 128, L.m0, &full[s]);
                        for (int h = 0; h < 2; ++h)
                            tma_load_2d(st + C::kXBytes + h * C::kWBytes, &tmW, k * 128, wrow + h * HALF, &full[s]);
                        if (k + kPrefetchAhead < a.KB && L.m0 == s_row[2 * L.e])
                            for (int h = 0; h < 2; ++h) prefetch_tile(&tmW, (k + kPrefetchAhead) * 128, wrow + h * HALF);
                    }
                    __syncwarp();
                }
            }
            // Every copy issued must have landed, and every commit arrived, before the block exits.
            for (uint32_t j = it > (uint32_t)C::kStages ? it - C::kStages : 0; j < it; ++j) {
                if ((j & 1u) != (uint32_t)warp) continue;
                wait_warp(&full[j % C::kStages], (j / C::kStages) & 1);
                wait_warp(&empty[j % C::kStages], (j / C::kStages) & 1);
            }
        } else {
            // No K block's sums depend on another's, so two warps issue them in
            // turn: each one's waits and commits pass while the other's MMAs run.
            uint32_t it = 0;
            const uint32_t odd = warp - kWarpIssue, d = tmem + odd * 256, idesc = idesc_e4m3(2 * HALF);
            const uint32_t x_lo = desc_lo(sbase), w_lo = desc_lo(sbase + C::kXBytes);
            for (int t = first; t < tiles; t += step) {
                for (int k = 0; k < a.KB; ++k, ++it) {
                    if ((it & 1u) != odd) continue;
                    const uint32_t s = it % C::kStages, r = it / C::kStages, rb = it / 2;
                    const uint32_t at = s * (C::kStageBytes >> 4);
                    wait_warp(&full[s], r & 1);
                    if (rb > 0) wait_warp(&acc_empty[odd], (rb & 1) ^ 1);
                    tc_fence_after();
                    if (lane == 0) {
                        mma_block(d, x_lo + at, w_lo + at, idesc);
                        mma_commit(&acc_full[odd]);
                        mma_commit(&empty[s]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        regs_up<224>();
        const int pw = warp - kWarpPromote, q = warp & 3, half = pw >> 2, m = q * 32 + lane;
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + half * HALF;
        uint32_t it = 0;
        float acc[HALF / 32][32];          // token m of the tile, the half's columns 32 x .. + 31
        // A half of 96 outputs may lie in two blocks of weight scales: its first
        // `split` columns in one, the others in the next.
        constexpr int kParts = HALF % 128 ? 2 : 1;
        float next_x[kAhead], next_w[kParts][kAhead];
        const float *xs;
        const typename SC::T *ws;
        bool here, there[kParts];          // whether the tile has this token, and the blocks are there
        int split = HALF;
        // Whole fours of scales at 16-byte addresses (4-byte ones of UE8M0) come in one load.
        const bool fours = a.KB % kAhead == 0 && reinterpret_cast<uintptr_t>(a.xs) % 16 == 0 &&
                           reinterpret_cast<uintptr_t>(a.ws) % (kAhead * sizeof(typename SC::T)) == 0;
        auto fetch = [&](int k) {
            if (fours) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (here && k < a.KB) v = *reinterpret_cast<const float4 *>(xs + k);
                next_x[0] = v.x, next_x[1] = v.y, next_x[2] = v.z, next_x[3] = v.w;
#pragma unroll
                for (int p = 0; p < kParts; ++p) SC::get4(next_w[p], ws + (size_t)p * a.KB + k, there[p] && k < a.KB);
                return;
            }
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
                next_x[c] = here && k + c < a.KB ? xs[k + c] : 0.f;
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    next_w[p][c] = there[p] && k + c < a.KB ? SC::get(ws, (size_t)p * a.KB + k + c) : 0.f;
            }
        };
        auto begin = [&](int t) {          // the tile's first scales are on their way
            const Tile N = find_tile<128>(a, s_tile, s_row, t);
            const int o = (2 * N.ot + half) * HALF, block = o / 128;
            here = m < N.rows;
            if (kParts > 1) split = min(HALF, 128 * (block + 1) - o);
#pragma unroll
            for (int p = 0; p < kParts; ++p) there[p] = block + p < a.NB;
            xs = a.xs + (size_t)(N.m0 + m) * a.KB;
            ws = static_cast<const typename SC::T *>(a.ws) + ((size_t)N.e * a.NB + block) * a.KB;
            fetch(0);
        };
        // One K block: the half's sums, times both scales, onto acc.  Scalar
        // FMAs: packed ones need their operands moved into pairs, 79 us
        // against 70 for 512 tokens of 16384 x 7168.
        auto promote = [&](const float (&f)[kParts]) {
            const uint32_t odd = it & 1u, tb = tq + odd * 256;
            wait_warp(&acc_full[odd], (it >> 1) & 1);
            tc_fence_after();
            Sums v[2];
            load(tb, v[0]);
#pragma unroll
            for (int x = 0; x < HALF / 32; ++x) {
                landed(v[x & 1]);
                if (x < HALF / 32 - 1) {
                    load(tb + 32 * (x + 1), v[(x + 1) & 1]);
                } else {
                    // the sums are in registers: the next MMAs may have the buffer
                    tc_fence_before();
                    __syncwarp();
                    arrive_if(lane == 0, &acc_empty[odd]);
                }
                const float fx = kParts == 1 || 32 * x < split ? f[0] : f[kParts - 1];
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[x][j] = fmaf(__uint_as_float(v[x & 1].r[j]), fx, acc[x][j]);
            }
            ++it;
        };
        auto tile_sums = [&]() {
            for (int k = 0; k < a.KB; k += kAhead) {
                float f[kAhead][kParts];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int p = 0; p < kParts; ++p) f[i][p] = next_x[i] * next_w[p][i];
                fetch(k + kAhead);
                const int n = min(kAhead, a.KB - k);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (i >= n) break;
                    promote(f[i]);
                }
            }
        };
        unsigned char *strip = smem + C::kOutOff + pw * 16 * kOutStride;
        // 64 bytes a token through shared memory, so that four lanes store a token's.
        auto store_strip = [&](const uint32_t (&w)[16], const Tile &L, int o) {
            const int esz = a.y_type == kF32 ? 4 : 2, per16 = 16 / esz;
            const bool lines = a.O % per16 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
            const int part = lane & 3, at = o + part * per16;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (lane >> 4 == x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(strip + (lane & 15) * kOutStride + 16 * i) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = 8 * i + (lane >> 2), mt = q * 32 + 16 * x + tok;
                    const uint4 v = *reinterpret_cast<const uint4 *>(strip + tok * kOutStride + 16 * part);
                    if (mt >= L.rows || at >= a.O) continue;
                    unsigned char *y = static_cast<unsigned char *>(a.Y) + ((size_t)(L.m0 + mt) * a.O + at) * esz;
                    if (lines) {
                        *reinterpret_cast<uint4 *>(y) = v;
                        continue;
                    }
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    if (esz == 4) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (at + e < a.O) reinterpret_cast<uint32_t *>(y)[e] = u[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (at + e < a.O) reinterpret_cast<uint16_t *>(y)[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
                    }
                }
                __syncwarp();
            }
        };
        if (first < tiles) begin(first);
        for (int t = first; t < tiles; t += step) {
#pragma unroll
            for (int x = 0; x < HALF / 32; ++x)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[x][j] = 0.f;
            tile_sums();
            if (t + step < tiles) begin(t + step);
            const Tile L = find_tile<128>(a, s_tile, s_row, t);    // looked up again: no register holds it over the sums
            if (q * 32 >= L.rows) continue;
#pragma unroll
            for (int y = 0; y < HALF / 32; ++y) {
                const int o = (2 * L.ot + half) * HALF + y * 32;
                if (o >= a.O) continue;
                uint32_t w[16];
                if (a.y_type == kF32) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(acc[y][16 * x + j]);
                        store_strip(w, L, o + 16 * x);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = pack_16(a.y_type, acc[y][2 * j], acc[y][2 * j + 1]);
                    store_strip(w, L, o);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpIssue) {
        tc_fence_after();
        tmem_free(tmem, kBufs * 256);
    }
}

template <int HALF, class SC>
int launch_as(const char *what, int blocks, const CUtensorMap &w, const CUtensorMap &x, const Args8 &a, cudaStream_t st) {
    using C = CfgMany<HALF>;
    set_max_dynamic_smem(reinterpret_cast<const void *>(gemm_e4m3_many_kernel<HALF, SC>), (int)C::kSmemBytes);
    return launch_pdl(what, gemm_e4m3_many_kernel<HALF, SC>, blocks, kThreads, C::kSmemBytes, st, w, x, a);
}

}  // namespace

ManyPlan plan_many(int M, int I, int O, int experts) {
    const int KB = (I + 127) / 128, n = num_sms(), filled = std::min(experts, M);
    const double per_output = token_tiles(M, experts, 128);
    ManyPlan best{128, n, 0.0};
    for (int half = 128; half >= 96; half -= 32) {
        const double tiles = (double)((O + 2 * half - 1) / (2 * half)) * per_output;
        // cycles of a K block, as measured; where an expert's weights serve one
        // tile alone, what a tile's take an SM at the card's bandwidth
        const double step = per_output < 1.5 * (experts == 1 ? 1 : filled) ? 2 * half * 5.5 : half == 128 ? 880.0 : 680.0;
        const double cost = std::ceil(tiles / n) * (KB * step + 3000.0);
        if (half == 128 || cost < best.cost) best = ManyPlan{half, n, cost};
    }
    return best;
}

int launch_many(const char *what, const ManyPlan &p, const E4m3Args &g, Args8 a, cudaStream_t st) {
    CUtensorMap w, x;
    if (!encode_map(&w, g.w, (long long)g.experts * g.O, g.I, p.half) || !encode_map(&x, g.X, g.M, g.I, 128))
        QG_REFUSE(kECuda, "%s: tensor map refused", what);
    a.NT = (g.O + 2 * p.half - 1) / (2 * p.half);
    if (p.half == 96)
        return g.w_power ? launch_as<96, ScaleE8M0>(what, p.blocks, w, x, a, st)
                         : launch_as<96, ScaleF32>(what, p.blocks, w, x, a, st);
    return g.w_power ? launch_as<128, ScaleE8M0>(what, p.blocks, w, x, a, st)
                     : launch_as<128, ScaleF32>(what, p.blocks, w, x, a, st);
}

}  // namespace e8
}  // namespace qg
