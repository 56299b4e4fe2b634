// gemm_e4m3_tc.cuh -- what the tensor-core kernels of the e4m3 x e4m3 products
// share (tcgen05 kind::f8f6f4, f32 accumulators in tensor memory):
//
//   Y[m, o] = sum_b xs[m, b] ws[o/128, b] sum_{i in block b} X[m, i] W[o, i]
//
// A K step is one block of 128 elements: four MMAs of K = 32 leave the
// block's sums in a buffer of tensor memory, and "promoting" warps add them,
// times the two scales, to f32 sums in registers.  gemm_e4m3_few.cu has the
// tokens along the MMA's N (as few as sixteen: decode), gemm_e4m3_many.cu
// along its M (prompts).
#pragma once

#include "gemm_tc.cuh"
#include "moe.cuh"

namespace qg {
namespace e8 {

using namespace tc;

constexpr int kWarpMma2 = 2;           // a second issuing warp: they take the stages in turn
constexpr int kMaxExperts = 1024;      // of one launch: the tables of tiles and rows in shared memory
constexpr uint32_t kTableBytes = (3 * kMaxExperts + 2) * 4;   // first tiles [E + 1], first and last rows [E][2]

struct Args8 {
    void *Y;
    int y_type;
    const float *xs;
    const void *ws;
    const int *offsets;               // NULL: one expert, rows [0, M)
    int before;                       // experts of the launches before this one: offsets[-before] is the table's first
    int experts, M, O, KB, NB, NT;    // K blocks, 128-output blocks, output tiles (set by the launch)
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

// The two words of sw128_desc: where an operand starts, in 16 bytes (32 bytes
// further along K: + 2), and what never changes.  One thread issues the MMAs,
// and every instruction before them is on the K step's way.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
// Four MMAs along K, the first of which starts the sums.
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
#pragma unroll
    for (uint32_t kk = 0; kk < 4; ++kk)
        mma_e4m3(d_tmem, (uint64_t)kDescHi << 32 | (a_lo + 2 * kk), (uint64_t)kDescHi << 32 | (b_lo + 2 * kk), idesc,
                 kk > 0 ? 1u : 0u);
}
// A box of a tensor map on its way from memory to L2.
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tmem_alloc(volatile uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr((const void *)slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// a += (lo, hi) * f, two f32 at a time
__device__ __forceinline__ void fma2(uint64_t &a, uint32_t lo, uint32_t hi, uint64_t f) {
    asm("{.reg .b64 t; mov.b64 t, {%1, %2}; fma.rn.f32x2 %0, t, %3, %0;}" : "+l"(a) : "r"(lo), "r"(hi), "l"(f));
}
__device__ __forceinline__ float2 pair_of(uint64_t v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Cluster helpers: the address of a local shared variable in another block, arrivals there, loads from there.
__device__ __forceinline__ uint32_t map_rank(uint32_t local, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One lane's arrival without a branch (a branch costs the warp some 100 cycles).
__device__ __forceinline__ void arrive_if(bool yes, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"((int)yes),
        "r"(smem_addr(bar))
        : "memory");
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

// Tables of the experts' first tiles (of BT tokens) and rows; ends with the
// writes of every thread, before a barrier.
template <int BT, int kThreads>
__device__ __forceinline__ void build_tables(const Args8 &a, int *s_tile, int *s_row, int2 *s_warp) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.offsets == nullptr) {
        if (threadIdx.x == 0) {
            s_tile[0] = 0;
            s_tile[1] = (a.M + BT - 1) / BT;
            s_row[0] = 0;
            s_row[1] = a.M;
        }
    } else {
        // The rule of next_rows: expert e has rows most[e] to most[e+1] of the running maximum.
        int tiles_before = 0, most = held_row(a.offsets[0], a.M);
        if (a.before > 0) {
            for (int i = threadIdx.x; i < a.before; i += kThreads) most = max(most, held_row(a.offsets[i - a.before], a.M));
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) s_warp[warp].x = most;
            __syncthreads();
            for (int w = 0; w < kThreads / 32; ++w) most = max(most, s_warp[w].x);
            __syncthreads();
        }
        for (int e0 = 0; e0 < a.experts; e0 += kThreads) {
            const int e = e0 + threadIdx.x;
            int to = 0;
            if (e < a.experts) {
                const int hi = a.offsets[e + 1];
                if (blockIdx.x == 0) check_offsets(a.offsets[e], hi, a.M, a.err);
                to = held_row(hi, a.M);
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
            for (int w = 0; w < kThreads / 32; ++w) {
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
            for (int w = 0; w < kThreads / 32; ++w) {
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
}

struct Tile {
    int e, m0, rows, ot;              // expert, first row, its rows in the tile, output tile
};
// Tiles are numbered expert by expert, output tile by output tile, tokens
// fastest: blocks of one wave share weights.
template <int BT>
__device__ __forceinline__ Tile tile_of(const Args8 &a, const int *s_tile, const int *s_row, int t, int e) {
    const int nt = s_tile[e + 1] - s_tile[e], local = t - s_tile[e] * a.NT;
    Tile r;
    r.e = e;
    r.ot = local / nt;
    r.m0 = s_row[2 * e] + (local - r.ot * nt) * BT;
    r.rows = min(s_row[2 * e + 1] - r.m0, BT);
    return r;
}
// Tile t, by a whole warp in two votes: the last e with s_tile[e] * NT <= t.
template <int BT>
__device__ __forceinline__ Tile find_tile_warp(const Args8 &a, const int *s_tile, const int *s_row, int t) {
    static_assert(kMaxExperts <= 32 * 32, "two votes of 32 lanes");
    const int lane = threadIdx.x & 31, apart = (a.experts + 31) / 32;
    const int far = lane * apart;
    unsigned yes = __ballot_sync(0xffffffffu, far < a.experts && s_tile[min(far, a.experts)] * a.NT <= t);
    const int from = (31 - __clz(yes)) * apart, near = from + lane;      // lane 0 votes yes: s_tile[0] = 0
    yes = __ballot_sync(0xffffffffu, lane < apart && near < a.experts && s_tile[min(near, a.experts)] * a.NT <= t);
    return tile_of<BT>(a, s_tile, s_row, t, from + 31 - __clz(yes));
}

// Host side: a map of [rows][I] codes in 128-byte swizzled boxes of box_rows x 128.
inline bool encode_map(CUtensorMap *m, const void *p, long long rows, int I, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)I, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)I};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `cluster` blocks of this kernel that run at once.
template <class K>
inline int count_clusters(K kernel, int threads, uint32_t smem, int cluster, int *out) {
    set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(out, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return kECuda;
    }
    return kOk;
}

// About how many tiles of bt tokens the experts' rows make (the host knows
// their sum alone): an expert's last tile is half empty.
inline double token_tiles(int M, int experts, int bt) {
    if (experts == 1) return (M + bt - 1) / bt;
    const double filled = std::min(experts, M);
    return std::max(filled, (double)M / bt + 0.5 * filled);
}

// The two kernels.  `cost` receives an estimate of the call's cycles.
struct FewPlan {
    int bt, cluster, blocks;
    double cost;
};
struct ManyPlan {
    int blocks;
    double cost;
};
FewPlan plan_few(int M, int I, int O, int experts);
ManyPlan plan_many(int M, int I, int O, int experts);
int launch_few(const char *what, const FewPlan &p, const E4m3Args &g, Args8 a, cudaStream_t st);
int launch_many(const char *what, const ManyPlan &p, const E4m3Args &g, Args8 a, cudaStream_t st);

}  // namespace e8
}  // namespace qg
