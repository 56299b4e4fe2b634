// gemm_e4m3_many.cu -- products of e4m3 activations with e4m3 weights, many
// tokens an expert: the tensor cores and the warps that empty them bound it.
//
// A tile is 128 tokens (MMA M) by 256 outputs (N), two halves with a weight
// scale each, so a promoting thread holds one token and scales a half's sums by
// one factor.  (With the tokens along N a factor a column has to be read from
// shared memory: 64 columns then take a warp 290 cycles instead of 134, and a K
// block 1800 instead of the MMAs' 512.)  4096 x 7168 x 7168 with normal codes:
// 157 us, 2685 TFLOP/s, about 770 cycles a K block.  What bounds it is the promoting warps,
// two a scheduler with 128 additions a thread and the wait and loads before
// them: without the additions it took 133 us (157 with them at the time), with
// one of a K block's four MMAs 146, without the copies 152.  As two MMAs of N =
// 128 a K block took 880 cycles: the tokens' codes are read twice.  Measured and
// left out: block pairs that share an MMA (half the weights a block; 0 to 10%
// slower, their signals cross SMs), tiles of 192 outputs (a K block takes the
// same time), and the next K block's first sums loaded before this one's last
// additions (164 us: the wait for its MMAs then stands before the additions).
// One persistent thread block per SM:
//   warps 0, 1   TMA producers, K blocks in turn: 128 x 128 codes of X and
//                256 x 128 of W, 128-byte swizzled
//   warps 2, 3   issue the MMAs, K blocks in turn; a block's four leave its sums
//                in one of two buffers of tensor memory
//   warps 4..11  promote: tensor-memory lanes 32 (w % 4) .. + 31, one half
//                each; a thread loads its token's scales and its half's four K
//                blocks ahead
#include "gemm_e4m3_tc.cuh"

namespace qg {
namespace e8 {
namespace {

constexpr int kPrefetchAhead = 8;
constexpr int kAhead = 4;              // K blocks of scales in a thread's registers
constexpr int kWarpIssue = 2, kWarpPromote = 4, kWarps = 8, kThreads = 32 * (kWarpPromote + kWarps);
constexpr int kBufs = 2;               // tensor-memory buffers of 256 columns
constexpr int kOutStride = 80;         // bytes between the tokens (64 each) of a strip on its way out: eight lanes' 16 bytes meet no bank twice

constexpr uint32_t kXBytes = 128 * 128, kWBytes = 256 * 128, kStageBytes = kXBytes + kWBytes;
constexpr uint32_t kOutAll = kWarps * 32 * kOutStride;             // strips of 64 bytes of a warp's tokens
constexpr uint32_t kBarBytes = 256;
constexpr int kStages = ~1 & (int)((kSmemBudget - 1024 - 256 - kOutAll - kTableBytes - kBarBytes) / kStageBytes);
constexpr int kNumBars = 2 * kStages + 2 * kBufs;
constexpr uint32_t kOutOff = kStages * kStageBytes, kBarOff = kOutOff + kOutAll, kTableOff = kBarOff + kBarBytes;
constexpr uint32_t kSmemBytes = 1024 + kTableOff + kTableBytes;
static_assert(kStages >= 3 && kNumBars * 8 + 16 <= (int)kBarBytes, "");
// A wait tells one phase of a barrier from the next, not from the one after
// that, so a stage must always be the same warps': with an odd number of
// stages one could pass on a phase that the other had not seen begin.
static_assert(kStages % 2 == 0 && kBufs == 2, "a stage and a buffer belong to the same producer and issuer every time");

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

template <class SC>
__global__ void __launch_bounds__(kThreads, 1)
gemm_e4m3_many_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Args8 a) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw);
    unsigned char *smem = smem_raw + ((1024u - (raw_base & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBarOff);
    uint64_t *full = bars, *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + kBufs;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bars + kNumBars);
    volatile uint32_t *abort = tmem_slot + 1;
    int *s_tile = reinterpret_cast<int *>(smem + kTableOff), *s_row = s_tile + kMaxExperts + 2;
    __shared__ int2 s_warp[kThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
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
    // promoting warps take 8 x 32 x 232 and the others 4 x 32 x 40.
    // Every lane waits: with one lane's wait and a vote the warp goes on 170 cycles later.
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
        mbar_wait_or_abort(bar, parity, abort);        // a wait that gives up sets *abort, which the block's end reports
        __syncwarp();
    };
    if (warp < kWarpPromote) {
        regs_down<40>();
        if (warp < kWarpIssue) {
            // What comes from memory goes to L2 kPrefetchAhead K blocks before
            // its copy, over the tile's end: weights by the tile that holds an
            // expert's first tokens, activations by the one of its first outputs.
            auto prefetch = [&](const Tile &L, int k) {
                if (L.m0 == s_row[2 * L.e]) prefetch_tile(&tmW, k * 128, L.e * a.O + L.ot * 256);
                if (L.ot == 0) prefetch_tile(&tmX, k * 128, L.m0);
            };
            uint32_t it = 0;
            Tile L, next;
            if (first < tiles) next = find_tile_warp<128>(a, s_tile, s_row, first);
            for (int t = first; t < tiles; t += step) {
                L = next;
                if (t + step < tiles) next = find_tile_warp<128>(a, s_tile, s_row, t + step);
                const int wrow = L.e * a.O + L.ot * 256;
                for (int k = 0; k < a.KB; ++k, ++it) {
                    if ((it & 1u) != (uint32_t)warp) continue;
                    const uint32_t s = it % kStages, r = it / kStages;
                    if (r > 0) wait_warp(&empty[s], (r & 1) ^ 1);
                    if (lane == 0) {
                        const uint32_t st = sbase + s * kStageBytes;
                        mbar_arrive_expect_tx(&full[s], kStageBytes);
                        tma_load_2d(st, &tmX, k * 128, L.m0, &full[s]);
                        tma_load_2d(st + kXBytes, &tmW, k * 128, wrow, &full[s]);
                        const int ahead = k + kPrefetchAhead;
                        if (ahead < a.KB) prefetch(L, ahead);
                        else if (t + step < tiles && ahead - a.KB < a.KB) prefetch(next, ahead - a.KB);
                    }
                    __syncwarp();
                }
            }
            // Every copy issued must have landed, and every commit arrived, before the block exits.
            for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j) {
                if ((j & 1u) != (uint32_t)warp) continue;
                wait_warp(&full[j % kStages], (j / kStages) & 1);
                wait_warp(&empty[j % kStages], (j / kStages) & 1);
            }
        } else {
            // No K block's sums depend on another's, so two warps issue them in
            // turn: each one's waits and commits pass while the other's MMAs run.
            uint32_t it = 0;
            const uint32_t odd = warp - kWarpIssue, d = tmem + odd * 256, idesc = idesc_e4m3(256);
            const uint32_t x_lo = desc_lo(sbase), w_lo = desc_lo(sbase + kXBytes);
            for (int t = first; t < tiles; t += step) {
                for (int k = 0; k < a.KB; ++k, ++it) {
                    if ((it & 1u) != odd) continue;
                    const uint32_t s = it % kStages, r = it / kStages, rb = it / 2;
                    const uint32_t at = s * (kStageBytes >> 4);
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
        regs_up<232>();
        const int pw = warp - kWarpPromote, q = warp & 3, half = pw >> 2, m = q * 32 + lane;
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
        uint32_t it = 0;
        float acc[4][32];          // token m of the tile, the half's columns 32 x .. + 31
        float next_x[kAhead];
        typename SC::Four next_w;
        const float *xs;
        const typename SC::T *ws;
        bool here, there;                  // whether the tile has this token and this half
        // Whole fours of scales at 16-byte addresses (4-byte ones of UE8M0) come in one load.
        const bool fours = a.KB % kAhead == 0 && reinterpret_cast<uintptr_t>(a.xs) % 16 == 0 &&
                           reinterpret_cast<uintptr_t>(a.ws) % (kAhead * sizeof(typename SC::T)) == 0;
        auto fetch = [&](int k) {
            if (fours) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (here && k < a.KB) v = *reinterpret_cast<const float4 *>(xs + k);
                next_x[0] = v.x, next_x[1] = v.y, next_x[2] = v.z, next_x[3] = v.w;
            } else {
#pragma unroll
                for (int c = 0; c < kAhead; ++c) next_x[c] = here && k + c < a.KB ? xs[k + c] : 0.f;
            }
            next_w.load(ws + k, there ? a.KB - k : 0, fours);
        };
        auto begin = [&](int t) {          // the tile's first scales are on their way
            const Tile N = find_tile_warp<128>(a, s_tile, s_row, t);
            const int block = 2 * N.ot + half;
            here = m < N.rows;
            there = block < a.NB;
            xs = a.xs + (size_t)(N.m0 + m) * a.KB;
            ws = static_cast<const typename SC::T *>(a.ws) + ((size_t)N.e * a.NB + block) * a.KB;
            fetch(0);
        };
        // One K block: the half's sums, times both scales, onto acc.  Scalar
        // FMAs: packed ones need their operands moved into pairs, 79 us
        // against 70 for 512 tokens of 16384 x 7168.
        auto promote = [&](float f) {
            const uint32_t odd = it & 1u, tb = tq + odd * 256;
            wait_warp(&acc_full[odd], (it >> 1) & 1);
            tc_fence_after();
            Sums v[2];
            load(tb, v[0]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                landed(v[x & 1]);
                if (x < 3) {
                    load(tb + 32 * (x + 1), v[(x + 1) & 1]);
                } else {
                    // the sums are in registers: the next MMAs may have the buffer
                    tc_fence_before();
                    __syncwarp();
                    arrive_if(lane == 0, &acc_empty[odd]);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[x][j] = fmaf(__uint_as_float(v[x & 1].r[j]), f, acc[x][j]);
            }
            ++it;
        };
        auto tile_sums = [&]() {
            for (int k = 0; k < a.KB; k += kAhead) {
                float f[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) f[i] = next_x[i] * next_w.get(i);
                fetch(k + kAhead);
                const int n = min(kAhead, a.KB - k);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (i >= n) break;
                    promote(f[i]);
                }
            }
        };
        // 64 bytes a token go through shared memory, so that four lanes store a
        // token's.  Where these are no whole lines neighbouring lanes store
        // neighbouring elements (19757 x 144 x 2023: 168 us with a lane's 16
        // bytes element by element, 45 so).
        unsigned char *strip = smem + kOutOff + pw * 32 * kOutStride;
        const int esz = a.y_type == kF32 ? 4 : 2, per16 = 16 / esz, part = lane & 3;
        const bool lines = a.O % per16 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
        // w: this lane's token's 64 bytes; at: the strip's first output; y: where this lane's first element goes
        auto store_strip = [&](const uint32_t (&w)[16], unsigned char *y, int at, int rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(strip + lane * kOutStride + 16 * i) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            __syncwarp();
            if (lines) {
#pragma unroll
                for (int i = 0; i < 4; ++i, y += (size_t)8 * a.O * esz) {
                    const int tok = 8 * i + (lane >> 2);
                    const uint4 v = *reinterpret_cast<const uint4 *>(strip + tok * kOutStride + 16 * part);
                    if (tok < rows && at + part * per16 < a.O) *reinterpret_cast<uint4 *>(y) = v;
                }
            } else if (esz == 4) {
                const int e = lane & 15, n = at + e < a.O ? min(rows, 32) : 0;
#pragma unroll 4
                for (int tok = lane >> 4; tok < n; tok += 2, y += (size_t)8 * a.O)
                    *reinterpret_cast<uint32_t *>(y) = *reinterpret_cast<const uint32_t *>(strip + tok * kOutStride + 4 * e);
            } else {
                const int n = at + lane < a.O ? min(rows, 32) : 0;
#pragma unroll 4
                for (int tok = 0; tok < n; ++tok, y += (size_t)2 * a.O)
                    *reinterpret_cast<uint16_t *>(y) = *reinterpret_cast<const uint16_t *>(strip + tok * kOutStride + 2 * lane);
            }
            __syncwarp();
        };
        if (first < tiles) begin(first);
        for (int t = first; t < tiles; t += step) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[x][j] = 0.f;
            tile_sums();
            if (t + step < tiles) begin(t + step);
            const Tile L = find_tile_warp<128>(a, s_tile, s_row, t);    // looked up again: no register holds it over the sums
            const int m0 = L.m0 + q * 32, rows = L.rows - q * 32, o0 = L.ot * 256 + half * 128;
            if (rows <= 0) continue;
            const int tok0 = lane >> (lines ? 2 : esz == 4 ? 4 : 5), e0 = lines ? part * per16 : lane & (esz == 4 ? 15 : 31);
            unsigned char *y = static_cast<unsigned char *>(a.Y) + ((size_t)(m0 + tok0) * a.O + o0 + e0) * esz;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if (o0 + 32 * z >= a.O) break;
                uint32_t w[16];
                if (a.y_type == kF32) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(acc[z][16 * x + j]);
                        store_strip(w, y + (32 * z + 16 * x) * 4, o0 + 32 * z + 16 * x, rows);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = pack_16(a.y_type, acc[z][2 * j], acc[z][2 * j + 1]);
                    store_strip(w, y + 32 * z * 2, o0 + 32 * z, rows);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort) raise_device_error(a.err, kErrTimeout);
    if (warp == kWarpIssue) {
        tc_fence_after();
        tmem_free(tmem, kBufs * 256);
    }
}

template <class SC>
int launch_as(const char *what, int blocks, const CUtensorMap &w, const CUtensorMap &x, const Args8 &a, cudaStream_t st) {
    set_max_dynamic_smem(reinterpret_cast<const void *>(gemm_e4m3_many_kernel<SC>), (int)kSmemBytes);
    return launch_pdl(what, gemm_e4m3_many_kernel<SC>, blocks, kThreads, kSmemBytes, st, w, x, a);
}

}  // namespace

ManyPlan plan_many(int M, int I, int O, int experts) {
    const int KB = (I + 127) / 128, n = num_sms(), filled = experts == 1 ? 1 : std::min(experts, M);
    const double per_output = token_tiles(M, experts, 128), tiles = (double)((O + 255) / 256) * per_output;
    // cycles of a K block, as measured; where an expert's weights serve one
    // tile alone, what 32 KB of them take an SM at the card's bandwidth
    const double step = per_output < 1.5 * filled ? 1400.0 : 800.0;
    return ManyPlan{n, std::ceil(tiles / n) * (KB * step + 5000.0)};
}

int launch_many(const char *what, const ManyPlan &p, const E4m3Args &g, Args8 a, cudaStream_t st) {
    CUtensorMap w, x;
    if (!encode_map(&w, g.w, (long long)g.experts * g.O, g.I, 256) || !encode_map(&x, g.X, g.M, g.I, 128))
        QG_REFUSE(kECuda, "%s: tensor map refused", what);
    a.NT = (g.O + 255) / 256;
    return g.w_power ? launch_as<ScaleE8M0>(what, p.blocks, w, x, a, st) : launch_as<ScaleF32>(what, p.blocks, w, x, a, st);
}

}  // namespace e8
}  // namespace qg
