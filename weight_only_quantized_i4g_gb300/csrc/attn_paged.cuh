// attn_paged.cuh -- attention of a few new tokens over a paged key-value cache
// (qattn_paged): the streaming kernel.
//
// Row (b, s, h) sees the slots t < len_b - S + 1 + s:
//   z_t = scale q . k_t,   o = sum_t exp(z_t - lse) v_t,   lse = log sum_t exp(z_t).
// The cache is read once and little is computed per byte, so the call is bound
// by HBM and everything serves keeping its reads in flight.
//
// Work.  The rows of one sequence that share a key-value head, R = S * group,
// form tiles; a (sequence, head, tile) is a segment of steps of up to 16 slots
// of one page.  A warp does 8 * NT rows; where there are more, GW warps share a
// ring and each does its rows of the same steps (so K and V come from HBM and
// L2 once for up to 64 rows).  Below, a warp stands for such a group.
// All segments' steps, laid end to end, are cut into one equal range per block
// (one block an SM) and each range into one per warp: unequal lengths balance
// without the host knowing them.  A segment counts kSegmentCost steps more than
// it has, for its Q and its end.  A warp keeps the running maximum and sum of
// each row and O in registers (online softmax).
// A segment that ends inside its warp is finished there; pieces of one that
// does not are joined in shared memory after the block's ranges are done, and
// across blocks by a second kernel, always in slot order.  Where every segment
// is short and has an SM or several to itself, a block or a thread-block cluster
// takes one whole segment instead, the cluster's blocks join their pieces over
// the workspace, and the second kernel is not needed.
//
// Loads.  Each warp keeps a ring of steps in shared memory, filled by TMA
// tensor copies (boxes of 16 slots by 128 bytes, 128-byte swizzle) that one
// lane issues NS steps ahead; the copies pad odd head sizes and page ends with
// zeros and take any strides.  Fragments are read 16 bytes a thread without
// bank conflicts: a fragment's k indices are the 8 (or 16) consecutive
// elements of a chunk, since the contraction over d may run in any order, and
// the chunks are dealt to the threads so that the swizzle spreads them.
// (cp.async in fragment order, 64 to 128 bytes a row and instruction, read 5.2
// TB/s; in runs of 512 bytes 6.8, but it took a code path each for pages that
// end inside a step, strides and padded heads, at the same issue cost, 450 to
// 600 cycles a warp and step.)
//
// Products.  S^T = K Q^T with the 16 slots as M and 8 rows as N (a decode step
// has few rows), then O^T = V^T P^T; P^T's fragment is the transpose of
// S^T's (movmatrix), V^T's pairs of slots are byte permutes of two loads.
// mma.sync suffices: at the HBM rate 16 slots of 128 dimensions arrive per SM
// every ~350 cycles and need 24 MMAs per 8 rows, a twelfth of its rate.
// Precision: products of 16-bit operands are exact and summed in f32.  P is
// not rounded to one 16-bit value but split into a sum of two (three for f32
// or f16 output of a bf16 cache), so it keeps 16 to 24 bits.  bf16 parts have
// f32's range.  f16 parts do not: P (and l) are scaled by 2^11 and the second
// part by 2^12 more, which its product's sum or V takes back, so that weights
// keep 16 bits down to 2^-32 of the row's largest and add nothing to O below
// 2^-48.  (With both parts scaled by 2^6 alone O was 1e-4 off where a slot with a
// zero v outweighs the others by 2^26, and most of it was lost at 2^32.)
// Where `fresh`, O itself is summed outside the MMAs, which round towards zero.
// Softmax.  Each row's exponents are taken against a reference that follows
// the running maximum only when a score passes it by more than 2^8 (f16 parts:
// 2^4, so p stays <= 2^15): a step then needs one vote instead of a maximum
// over lanes.
// e4m3 codes are exact in f16; q over them is scaled per row by a power of two
// into f16's range, which is exact for bf16 values within 2^29 of the largest.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kv_cache.cuh"

namespace qg {

constexpr int kAttnMaxSeq = 2048;     // sequences per launch (their lengths sit in shared memory)
constexpr int kMaxRanks = 8;          // blocks of a cluster
constexpr int kSegmentCost = 2;       // what starting and ending a segment takes, in steps (~5000 cycles against ~2000)

// Workspace of one launch.
struct AttnWork {
    float *part_o;      // [ctas][2][rows][DP]: pieces a block leaves open, at its start (0) and end (1)
    float2 *part_ml;    // [ctas][2][rows]: their maxima (log2 units) and sums
    float *head_o;      // [ctas][warps][its rows][DP]: pieces a warp finishes before its range ends
    int2 *open;         // [ctas]: {segment a block leaves open at its end or -1, blocks it spans}
    int2 *span;         // accumulate: [segment]: {its first block, blocks it spans}
    float *scores;      // accumulate: z in log2 units, [segment][slot][score_rows]
    int score_slots, score_rows;   // slots per segment; rows, a multiple of four
    int row_tiles;
    int tiles;          // segments per sequence: heads times row tiles
    int ranks;          // blocks (a cluster) that take one whole segment; 0: equal ranges of all steps
    int ctas;           // blocks of the streaming kernel
    int page_steps;     // steps of a page
    int box_rows;       // slots a copy moves: 16, or a smaller page
    FastDiv tiles_div, row_tiles_div, group_div, page_steps_div;
};

constexpr int warps_for(int regs) { return regs <= 128 ? 16 : regs <= 168 ? 12 : 8; }

// FINE: the output is of more bits than a bf16 or e4m3 cache's kernels have
// otherwise (f32, f16).  With bf16 P then has three parts.
template <int TYPE, int DP_, int NT_, int GW_, bool FINE>
struct AttnCfg {
    static constexpr int DP = DP_, NT = NT_, GW = GW_;
    static constexpr bool THIRD = FINE && TYPE == kBf16;
    // An MMA rounds its sum towards zero: O shrinks by about 2^-24.4 a step that
    // is summed in the accumulators (measured: 2.2e-6 after 50 steps, 1e-7
    // without).  So a step's product is summed alone and then added
    // to O, which rounds to nearest.  Only where a warp has 16 rows and more and
    // the output is bf16 the sum stays in the accumulators: 600,000 slots of one
    // warp would make that half a unit of bf16, and 48 ragged sequences take
    // 222 us for 242 (32 rows at 128 dimensions; 420 for 460 with 64 rows; with
    // e4m3 214 for 291).  With 8 rows there is no difference in time.
    static constexpr bool fresh = FINE || TYPE == kF16 || (NT == 1 && GW == 1);
    // where the second f16 part of P gets its scale of 2^12 back: in its
    // product's sum where that starts empty, else in V (exact for e4m3 codes).
    // 64 e4m3 sequences of 6000 to 16384, 7 rows: 233 us with the sum, 241 with V,
    // 232 with an unscaled part.
    static constexpr bool LOW_SUM = fresh && TYPE != kBf16, LOW_V = !fresh && TYPE == kE4m3;
    static_assert(LOW_SUM || TYPE != kF16, "V of a f16 cache cannot be scaled exactly");
    static constexpr int ESZ = TYPE == kE4m3 ? 1 : 2;
    static constexpr int warp_rows = 8 * NT, rows = GW * warp_rows;   // of a warp, of a segment
    static constexpr int KE = 16 / ESZ;               // elements of a K chunk
    static constexpr int NI = DP * ESZ / 64;          // K chunks a thread holds per slot (4 threads a slot)
    static constexpr int E = DP / 8 < KE ? DP / 8 : KE;   // elements of a V chunk (8 threads a slot)
    static constexpr int VB = E * ESZ;                // its bytes: 16, or 8
    static constexpr int NQ = DP / (8 * E);           // V chunks a thread holds per slot
    static constexpr int MT = DP / 16;                // 16-row tiles of O^T
    static constexpr int BB = DP * ESZ < 128 ? DP * ESZ : 128;   // bytes of a row in one box: 64 or 128
    static constexpr int NB = DP * ESZ / BB;          // boxes of a row
    static constexpr int box = 16 * BB;
    static constexpr int stage = 2 * NB * box;        // 16 slots of K, then of V
    // as many warps as the registers of O, Q and S allow (16, 12 or 8 an SM);
    // groups keep Q in shared memory where that makes it more: 12 for 8 (48
    // ragged bf16 sequences, 32 rows at 128 dimensions: 236 -> 222 us; f16 264 ->
    // 258, e4m3 238 -> 214), 16 for 12 (64 dimensions, f16: 158 -> 147; with four
    // drafted tokens, lengths to 4099, 29.6 -> 26.9).  Not where FINE needs more
    // registers (e4m3 243 -> 251, bf16 with its third part of P 287 -> 283)
    static constexpr int regs0 = (ESZ == 1 ? 85 : 70) + 4 * MT * NT + 8 * NT, regs_q = NT * NI * (ESZ == 1 ? 8 : 4);
    static constexpr bool QS = GW > 1 && DP <= 128 && NT == 2 && !FINE && warps_for(regs0) > warps_for(regs0 + regs_q);
    static constexpr int W0 = warps_for(regs0 + (QS ? 0 : regs_q));
    static constexpr int W = GW == 1 && stage > 8192 ? 4 : W0;
    static constexpr int q_bytes = QS ? NT * NI * (ESZ == 1 ? 2 : 1) * 512 : 0;   // of a warp
    static constexpr int G = W / GW;                  // groups, a ring each
    // 8 rows of O on their way out; a lone warp takes the stage it has just read
    static constexpr int slab = GW > 1 ? 32 * DP : 0;
    // up to 192 KB of copies in flight
    static constexpr int NS0 = (196608 - W * (slab + q_bytes)) / (G * stage);
    static constexpr int NS = GW == 1 ? (NS0 > 6 ? 6 : NS0) : (NS0 > 8 ? 8 : NS0);
    static constexpr int ring = NS * stage;           // per group
    static_assert(ring >= rows * DP * 4, "an open piece takes the place of its ring");
    static constexpr int threads = 32 * W;
};

// The ring: byte offset of 16-byte chunk `chunk` of slot `row` in a step's K or
// V, as the copies' swizzle leaves it.
template <class C>
__host__ __device__ __forceinline__ constexpr int chunk_place(int row, int chunk) {
    constexpr int per = C::BB / 16;
    const int b = chunk / per, x = chunk % per;
    return b * C::box + row * C::BB + 16 * (per == 8 ? x ^ (row & 7) : x ^ (row >> 1 & 3));
}
// Which chunk of its slot a thread (c = lane % 4) holds as its i-th of K: with
// rows of 128 bytes neighbouring ones, so that the swizzle of even and odd rows
// parts the eight lanes of a read.
template <class C>
__host__ __device__ __forceinline__ constexpr int k_chunk(int i, int c) {
    return C::BB == 128 ? 8 * (i >> 1) + 2 * c + (i & 1) : 4 * i + c;
}
// Pieces of 8 rows of O in shared memory: place (in float4) of quad x of row r.
// The exchange by row parts the eight lanes of a store (two g, four c).
template <class C>
__host__ __device__ __forceinline__ constexpr int slab_place(int r, int x) {
    return r * (C::DP / 4) + (x ^ ((r >> 1 & 1) | (r >> 2 & 1) << 2));
}

template <class C>
__host__ __device__ constexpr size_t attn_fixed_smem() {
    // 1 KB for the copies' alignment, then as laid out in the kernel
    return 1024 + (size_t)C::G * C::ring + C::W * (C::slab + C::q_bytes) + C::G * C::NS * (8 + 8 + 16) +
           C::G * 2 * C::rows * sizeof(float2) + C::G * 2 * 8;
}

// Box at element x, slot t, head h of page p.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int t, int h, int p,
                                            uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(t), "r"(h), "r"(p), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {       // 2^x, 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

template <int TYPE>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (TYPE == kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A B, nothing added.
template <int TYPE>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    if (TYPE == kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// An f16 pair by 2^-12.
__device__ __forceinline__ uint32_t f16x2_down12(uint32_t v) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x0C000C00u));
    return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Elements 4 at a time of an output row: normalised, in the output's type.
__device__ __forceinline__ void store_out4(const AttnArgs &a, size_t at, float4 v, float f) {
    v.x *= f, v.y *= f, v.z *= f, v.w *= f;
    if (a.o_type == kF32)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + at) =
            make_uint2(pack_16(a.o_type, v.x, v.y), pack_16(a.o_type, v.z, v.w));
}

// A row's statistics: reference m (log2 units) and sum l of 2^(z - m).  A row
// that has seen nothing has l = 0 and m = kNoRef, whose differences are finite.
constexpr float kNoRef = -3e38f;
__device__ __forceinline__ float row_factor(float l, float v_scale) { return l == 0.f ? 0.f : v_scale / l; }
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Row r of a (sequence, key-value head): new token s, q head, and their index
// in q, o and lse.
struct RowRef { bool real; int s, q_head; size_t head; };
__device__ __forceinline__ RowRef row_ref(const AttnArgs &a, const AttnWork &w, int b, int kh, int r) {
    RowRef x;
    x.real = r < a.S * a.group;
    x.s = quotient(r, w.group_div);
    x.q_head = kh * a.group + (r - x.s * a.group);
    x.head = ((size_t)b * a.S + x.s) * a.n_q_heads + x.q_head;
    return x;
}

// Elements d .. d + 3 of the sum of a row with weight l, over a cache of 16 bits.
// An infinity in V times a part of P that is zero or negative is NaN where its
// product with P is infinite.  So where elements are NaN and the weights are not,
// the infinities that the row sees stand for them: the sign that they agree on.
__device__ __forceinline__ float4 with_infinities(const AttnArgs &a, const RowRef &row, int b, int kh, int d, float4 sum,
                                                  float l) {
    int open = (sum.x != sum.x) | (sum.y != sum.y) << 1 | (sum.z != sum.z) << 2 | (sum.w != sum.w) << 3;
    if (__builtin_expect(open == 0 || !(l > 0.f), 1)) return sum;
    const int end = seq_len(a.lens, b, a.max_len, nullptr) - a.S + 1 + row.s, ex = a.c.type == kBf16 ? 0x7F80 : 0x7C00;
    int up = 0, down = 0;                             // a bit an element: +inf, -inf seen (a NaN: both)
#pragma unroll 1
    for (int t = 0; t < end && (open & ~(up & down)); ++t) {
        const SlotRef r = find_slot(a.c, a.table + (size_t)b * a.table_stride, t);
        if (r.page < 0) continue;
        const uint2 w = *reinterpret_cast<const uint2 *>(a.c.v + slot_bytes(a.c, r, kh) + 2 * d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int v = (e < 2 ? w.x : w.y) >> (16 * (e & 1)) & 0xFFFF;
            if ((v & 0x7FFF) < ex) continue;
            if (v != (ex | 0x8000)) up |= 1 << e;
            if (v != ex) down |= 1 << e;
        }
    }
    open &= up ^ down;                                // the infinities agree
    auto pick = [&](float x, int e) { return open >> e & 1 ? up >> e & 1 ? INFINITY : -INFINITY : x; };
    return make_float4(pick(sum.x, 0), pick(sum.y, 1), pick(sum.z, 2), pick(sum.w, 3));
}

// Steps of a sequence of len slots: 16 slots of a page each, fewer at the ends
// of pages and of the sequence.
__host__ __device__ __forceinline__ int seq_steps(const KvView &c, const AttnWork &w, int len) {
    const int full = quotient(len, c.page_div);
    return full * w.page_steps + ((len - full * c.page + 15) >> 4);
}

// Lengths of all sequences, and the running sums (n + 1) of their segments'
// costs (a sequence without slots has none), into shared memory; THREADS
// threads, `s_sum` one int per warp.
template <int THREADS>
__device__ __forceinline__ void scan_costs(const AttnArgs &a, const AttnWork &w, int *s_len, int *s_prefix, int *s_sum, int *err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_seq;
    const int per = (n + THREADS - 1) / THREADS;
    int sum = 0;
    for (int i = tid * per; i < (tid + 1) * per && i < n; ++i) {
        const int len = seq_len(a.lens, i, a.max_len, err);
        s_len[i] = len;
        if (len > 0) sum += seq_steps(a.c, w, len) + kSegmentCost;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i)
        if (i < warp) base += s_sum[i];
    int at = base + inc - sum;
    for (int i = tid * per; i < (tid + 1) * per && i < n; ++i) {
        s_prefix[i] = at;
        if (s_len[i] > 0) at += seq_steps(a.c, w, s_len[i]) + kSegmentCost;
    }
    if (tid == THREADS - 1) s_prefix[n] = at;
    __syncthreads();
}

// Cost units per block where all are cut into equal ranges: a step per warp at least.
__host__ __device__ __forceinline__ int units_per_block(int total, int ctas, int warps) {
    const int chunk = (total + ctas - 1) / ctas;
    return chunk < warps + kSegmentCost ? warps + kSegmentCost : chunk;
}

// A step: sequence, segment there, step of that (page of the sequence and step
// inside it) and steps of the segment.
struct Place { int b, seg, i, n, page, sub; };
// The first step at or after unit u; a segment's first kSegmentCost units have none.
__host__ __device__ __forceinline__ Place locate(int u, const int *s_prefix, int n, const AttnWork &w) {
    Place p = {n, 0, 0, 1, 0, 0};
    const int x = quotient(u, w.tiles_div);
    if (x >= s_prefix[n]) return p;
    int lo = 0, hi = n - 1;                          // the last b with prefix[b] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    const int cost = s_prefix[lo + 1] - s_prefix[lo], rem = u - s_prefix[lo] * w.tiles;
    p.b = lo;
    p.n = cost - kSegmentCost;
    p.seg = rem / cost;
    p.i = rem - p.seg * cost - kSegmentCost;
    if (p.i < 0) p.i = 0;
    p.page = quotient(p.i, w.page_steps_div);
    p.sub = p.i - p.page * w.page_steps;
    return p;
}
// Steps from place x up to place y.
__host__ __device__ __forceinline__ int steps_between(const Place &x, const Place &y, const int *s_prefix, int tiles) {
    int steps = y.seg * y.n + y.i - (x.seg * x.n + x.i);
    for (int b = x.b; b < y.b; ++b) {
        const int cost = s_prefix[b + 1] - s_prefix[b];
        if (cost) steps += tiles * (cost - kSegmentCost);
    }
    return steps;
}
// The step after p (the sequence n, segment 0, step 0 after the last).
__host__ __device__ __forceinline__ void advance(Place &p, const int *s_prefix, int n, const AttnWork &w) {
    if (++p.sub == w.page_steps) p.sub = 0, ++p.page;
    if (++p.i < p.n) return;
    p.i = p.page = p.sub = 0;
    if (++p.seg < w.tiles) return;
    p.seg = 0;
    do ++p.b;
    while (p.b < n && s_prefix[p.b + 1] == s_prefix[p.b]);
    p.n = p.b < n ? s_prefix[p.b + 1] - s_prefix[p.b] - kSegmentCost : 1;
}
// Unit where part x of `parts` of the range [c0, c1) begins.
__host__ __device__ __forceinline__ int part_of(int c0, int c1, int x, int parts) {
    return c0 + (int)((long long)(c1 - c0) * x / parts);
}
// Steps per block where `ranks` of them take a segment of n steps: a step per
// warp (or group of warps) at least.
__host__ __device__ __forceinline__ int steps_per_rank(int n, int ranks, int groups) {
    const int each = (n + ranks - 1) / ranks;
    return each < groups ? groups : each;
}
// Blocks that the segment (sequence b, number sg) spans, from the block that holds its first step.
__host__ __device__ __forceinline__ int blocks_spanned(int b, int sg, int first, int chunk, const int *s_prefix,
                                                       int tiles) {
    const int end_unit = s_prefix[b] * tiles + (sg + 1) * (s_prefix[b + 1] - s_prefix[b]);
    return (end_unit - 1) / chunk - first + 1;
}

// DRAFT: several new tokens a sequence, the last of which some rows do not see.
// (Without the code for those the calls of one token are 2% faster.)
template <int TYPE, int DP_, int NT_, int GW_, bool FINE, bool DRAFT>
__global__ void __launch_bounds__(AttnCfg<TYPE, DP_, NT_, GW_, FINE>::threads, 1)
    attn_stream_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnWork w,
                       const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = AttnCfg<TYPE, DP_, NT_, GW_, FINE>;
    constexpr int DP = C::DP, NT = C::NT, W = C::W, GW = C::GW, G = C::G, NS = C::NS, NI = C::NI, E = C::E, NQ = C::NQ;
    constexpr int rows = C::rows, warp_rows = C::warp_rows;
    // flags of a step: its page is not in the pool; first and last of its segment
    constexpr int kMissing = 32, kFirst = 64, kLast = 128;
    extern __shared__ char smem_raw[];
    char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *s_bar = reinterpret_cast<uint64_t *>(smem + G * C::ring + W * (C::slab + C::q_bytes));   // [G][NS]: a step has landed
    uint64_t *s_free = s_bar + G * NS;                                        // [G][NS]: all warps have read it
    float2 *s_ml = reinterpret_cast<float2 *>(s_free + G * NS);               // [G][2][rows]
    int2 *s_piece = reinterpret_cast<int2 *>(s_ml + G * 2 * rows);            // [G][2]: {segment or -1, 1: ended | 2: in head_o}
    // [G][NS] of a step in the ring: its slots and flags, its first slot, its
    // segment, the first slot that some row of the sequence does not see
    int4 *s_state = reinterpret_cast<int4 *>(s_piece + G * 2);
    int *s_prefix = reinterpret_cast<int *>(s_state + G * NS);                // [n + 1]
    int *s_len = s_prefix + a.n_seq + 1;                                      // [n]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n = a.n_seq, D = a.c.dim;
    const int tiles = w.tiles;
    const int group = warp / GW, mate = warp % GW, my_rows = mate * warp_rows;   // rows of the segment before the warp's
    if (tid < G * NS) mbar_init(&s_bar[tid], 1), mbar_init(&s_free[tid], GW);
    if (tid < G * 2) s_piece[tid] = make_int2(-1, 0);
    mbar_fence_init();
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&k_map)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&v_map)) : "memory");
    }

    // the second kernel may start once lengths, tables and weights are final: it reads them before its own wait
    griddep_wait();
    griddep_launch_dependents();

    scan_costs<C::threads>(a, w, s_len, s_prefix, reinterpret_cast<int *>(s_state),
                           blockIdx.x == 0 ? a.err : nullptr);
    int c0, c1, chunk, shared_by = 1;                                         // in cost units
    const int rank = w.ranks > 1 ? blockIdx.x % w.ranks : 0;
    if (w.ranks > 0) {
        const int seg = blockIdx.x / w.ranks, b = quotient(seg, w.tiles_div), cost = s_prefix[b + 1] - s_prefix[b];
        const int steps = cost ? cost - kSegmentCost : 0, base = s_prefix[b] * tiles + (seg - b * tiles + 1) * cost - steps;
        chunk = steps_per_rank(steps, w.ranks, G);
        shared_by = (steps + chunk - 1) / chunk;
        c0 = base + (rank * chunk < steps ? rank * chunk : steps);
        c1 = base + ((rank + 1) * chunk < steps ? (rank + 1) * chunk : steps);
    } else {
        const int total = s_prefix[n] * tiles;
        chunk = units_per_block(total, gridDim.x, G);
        c0 = (int)(blockIdx.x * chunk) < total ? blockIdx.x * chunk : total;
        c1 = c0 + chunk < total ? c0 + chunk : total;
        if (tid == 0) w.open[blockIdx.x] = make_int2(-1, 0);
    }

    // sequences without a slot have no steps: their rows are empty
#pragma unroll 1
    for (int b = blockIdx.x; b < n; b += gridDim.x) {
        if (s_len[b] != 0) continue;
        const int quads = D / 4, count = a.S * a.n_q_heads;
#pragma unroll 1
        for (int i = tid; i < count * quads; i += C::threads)
            store_out4(a, ((size_t)b * count) * D + 4 * (size_t)i, make_float4(0.f, 0.f, 0.f, 0.f), 1.f);
        if (a.lse)
            for (int i = tid; i < count; i += C::threads) a.lse[(size_t)b * count + i] = -INFINITY;
    }
    if (c0 >= c1 && w.ranks <= 1) return;

    // the warp's first step, and how many it has
    Place ip = locate(part_of(c0, c1, group, G), s_prefix, n, w);
    int left = steps_between(ip, locate(part_of(c0, c1, group + 1, G), s_prefix, n, w), s_prefix, tiles);
    char *ring = smem + group * C::ring;
    const uint32_t ring_a = smem_addr(ring);

    // ---- loads: the page of the next step is looked up one step early ----
    // K and V are read once per row tile: marked first to leave L2 where there is but one
    uint64_t policy;
    if (w.row_tiles == 1) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    int to_issue = mate == 0 ? left : 0, istage = 0, look_page = 0;
    auto look = [&]() {
        if (to_issue == 0) return;
        look_page = a.table[(size_t)ip.b * a.table_stride + ip.page];
    };
    // reuse: wait until the group's other warps have read what the stage held
    auto issue = [&](bool reuse, uint32_t phase) {
        if (to_issue > 0) {
            if (lane == 0 && (GW == 1 || !reuse || mbar_wait(&s_free[group * NS + istage], phase))) {
                const int slot = 16 * ip.sub, before = ip.page * a.c.page, len = s_len[ip.b];
                int count = (len - before < a.c.page ? len - before : a.c.page) - slot;
                if (count > 16) count = 16;
                uint64_t *bar = &s_bar[group * NS + istage];
                const uint32_t dst = ring_a + istage * C::stage;
                const int kh = quotient(ip.seg, w.row_tiles_div);
                const bool there = (unsigned)look_page < (unsigned)a.c.n_pages;
                s_state[group * NS + istage] =
                    make_int4(count | (there ? 0 : kMissing) | (ip.i == 0 ? kFirst : 0) | (ip.i + 1 == ip.n ? kLast : 0),
                              before + slot, ip.b * tiles + ip.seg, len - a.S + 1);
                if (there) {
                    mbar_arrive_expect_tx(bar, 2 * C::NB * C::BB * w.box_rows);
#pragma unroll
                    for (int x = 0; x < C::NB; ++x)
                        tma_load_4d(dst + x * C::box, &k_map, x * (C::BB / C::ESZ), slot, kh, look_page, bar, policy);
#pragma unroll
                    for (int x = 0; x < C::NB; ++x)
                        tma_load_4d(dst + (C::NB + x) * C::box, &v_map, x * (C::BB / C::ESZ), slot, kh, look_page, bar,
                                    policy);
                } else {
                    raise_device_error(a.err, kErrPage);
                    mbar_arrive(bar);
                }
            }
            --to_issue;
            advance(ip, s_prefix, n, w);
            look();
        }
        if (++istage == NS) istage = 0;
    };
    look();
#pragma unroll 1
    for (int i = 0; i < NS; ++i) issue(false, 0u);

    // ---- the warp's range ----
    float o[C::MT][NT][4];
    float m[NT][2], l[NT][2];
    constexpr int QW = C::ESZ == 1 ? 8 : 4;           // words of Q per chunk
    uint32_t qf[C::QS ? 1 : NT][NI][QW];              // or in shared memory, each lane's own
    const uint32_t q_mem = smem_addr(smem) + G * C::ring + W * C::slab + warp * C::q_bytes + lane * 16;
    float rs[NT][2];                                  // score factor of the thread's rows (e4m3: per row)
    const float factor = a.scale * 1.44269504088896340736f;
    constexpr float shift = TYPE == kBf16 ? 0.f : 11.f, lag = TYPE == kBf16 ? 8.f : 4.f;
    bool fresh = true;                                // at the start of a piece
    bool began_here = false;
    int stage = 0;
    uint32_t phase = 0;

#pragma unroll 1
    for (; left > 0; --left) {
        // a lone warp can load Q while the step is on its way
        bool landed = true;
        if (GW > 1) landed = __all_sync(~0u, mbar_wait(&s_bar[group * NS + stage], phase));
        if (fresh && landed) {
            __syncwarp();                             // lane 0 wrote the state
            const int4 state = s_state[group * NS + stage];
            const int b = quotient(state.z, w.tiles_div), sg = state.z - b * tiles;
            const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
            fresh = false;
            began_here = state.x & kFirst;
            // Q as the B operand: row g of each 8, the thread's chunks
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t(&qn)[NI][QW] = qf[C::QS ? 0 : nt];
                const RowRef r = row_ref(a, w, b, kh, tile * rows + my_rows + 8 * nt + g);
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + ((size_t)b * a.S + r.s) * a.q_stride +
                                    (size_t)r.q_head * D;
                if constexpr (TYPE != kE4m3) {
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int d = k_chunk<C>(i, c) * 8;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (r.real && d < D) v = *reinterpret_cast<const uint4 *>(q + d);
                        qn[i][0] = v.x, qn[i][1] = v.y, qn[i][2] = v.z, qn[i][3] = v.w;
                    }
                } else {
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int d = k_chunk<C>(i, c) * 16;
                        uint4 v[2] = {};
                        if (r.real && d < D)
                            v[0] = *reinterpret_cast<const uint4 *>(q + d),
                            v[1] = *reinterpret_cast<const uint4 *>(q + d + 8);
                        const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            qn[i][u] = x[u];
                            const float2 f = a.q_type == kF16 ? unpack_f16(x[u]) : unpack_bf16(x[u]);
                            if (fabsf(f.x) < INFINITY) top = fmaxf(top, fabsf(f.x));
                            if (fabsf(f.y) < INFINITY) top = fmaxf(top, fabsf(f.y));
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    // largest |q| of the row into [2^14, 2^15): by 2^-113 for the largest
                    // numbers, by 2^126 at most (2^-126 is the last normal inverse)
                    int ex = 141 - (int)(__float_as_uint(top) >> 23);
                    ex = top == 0.f ? 0 : ex > 126 ? 126 : ex;
                    const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float2 f = a.q_type == kF16 ? unpack_f16(qn[i][u]) : unpack_bf16(qn[i][u]);
                            qn[i][u] = pack_f16(f.x * up, f.y * up);
                        }
                    const float down = factor * __uint_as_float((uint32_t)(127 - ex) << 23) * a.c.k_scale[kh];
                    rs[nt][0] = __shfl_sync(~0u, down, 8 * c);
                    rs[nt][1] = __shfl_sync(~0u, down, 8 * c + 4);
                }
                if constexpr (C::QS) {
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int u = 0; u < QW; u += 4)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q_mem + ((nt * NI + i) * QW + u) * 128),
                                         "r"(qn[i][u]), "r"(qn[i][u + 1]), "r"(qn[i][u + 2]), "r"(qn[i][u + 3])
                                         : "memory");
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nt][e] = kNoRef;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int t = 0; t < C::MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
            }
        }

        if (GW == 1) landed = __all_sync(~0u, mbar_wait(&s_bar[group * NS + stage], phase));
        if (!landed) {
            // a copy did not land in time: no result, but let those in flight land before the block ends
            if (lane == 0) raise_device_error(a.err, kErrTimeout);
            for (; mate == 0 && left > to_issue; --left) {
                mbar_wait(&s_bar[group * NS + stage], phase);
                if (++stage == NS) stage = 0, phase ^= 1u;
            }
            break;
        }
        // published by the arrival that the wait has seen
        const int4 state = s_state[group * NS + stage];
        const int count = state.x & 31, t0 = state.y, hidden_from = state.w;
        const uint32_t src = ring_a + stage * C::stage, src_v = src + C::NB * C::box;

        // ---- S^T = K Q^T, in two chains ----
        float s[NT][4], s1[NT][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            // slots g and g + 8
            const uint4 x = lds128(src + chunk_place<C>(g, k_chunk<C>(i, c)));
            const uint4 y = lds128(src + chunk_place<C>(g + 8, k_chunk<C>(i, c)));
            const uint32_t kx[4] = {x.x, x.y, x.z, x.w}, ky[4] = {y.x, y.y, y.z, y.w};
            uint32_t qi[NT][QW];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < QW; u += 4) {
                    if constexpr (C::QS) {
                        const uint4 v = lds128(q_mem + ((nt * NI + i) * QW + u) * 128);
                        qi[nt][u] = v.x, qi[nt][u + 1] = v.y, qi[nt][u + 2] = v.z, qi[nt][u + 3] = v.w;
                    } else {
#pragma unroll
                        for (int z = 0; z < 4; ++z) qi[nt][u + z] = qf[nt][i][u + z];
                    }
                }
#pragma unroll
            for (int u = 0; u < C::KE / 4; ++u) {
                uint32_t a0, a1, a2, a3;
                if constexpr (TYPE != kE4m3) {
                    a0 = kx[2 * u], a1 = ky[2 * u], a2 = kx[2 * u + 1], a3 = ky[2 * u + 1];
                } else {
                    e4m3x4_to_f16x2(kx[u], &a0, &a2);
                    e4m3x4_to_f16x2(ky[u], &a1, &a3);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&d)[4] = u & 1 ? s1[nt] : s[nt];
                    if (i == 0 && u < 2) mma16816_first<TYPE>(d, a0, a1, a2, a3, qi[nt][2 * u], qi[nt][2 * u + 1]);
                    else mma16816<TYPE>(d, a0, a1, a2, a3, qi[nt][2 * u], qi[nt][2 * u + 1]);
                }
            }
        }

        // ---- exponents against the rows' references; thread: slots g, g + 8 by rows 2c, 2c + 1 ----
        const bool partial = (state.x & 63) != 16 || (DRAFT && a.S > 1 && t0 + 16 > hidden_from);
        // slots that row nt, e of the thread sees of this step and before it
        auto limit = [&](int nt, int e) {
            const int sg = state.z - quotient(state.z, w.tiles_div) * tiles;
            const int tile = sg - quotient(sg, w.row_tiles_div) * w.row_tiles;
            const int s = quotient(tile * rows + my_rows + 8 * nt + 2 * c + (e & 1), w.group_div);
            return hidden_from + (s < a.S ? s : a.S - 1);
        };
        // no weight for slots that the step has not, or that the row does not see; NaN for a missing page
        auto masked = [&](float z, int nt, int e) {
            const int j = g + 8 * (e >> 1);
            if (j >= count || (DRAFT && a.S > 1 && t0 + j >= limit(nt, e))) return -INFINITY;
            return state.x & kMissing ? NAN : z;
        };
        // one vote for all rows: the tiles' chains then run side by side
        float x[NT][4];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] += s1[nt][e];
                x[nt][e] = fmaf(s[nt][e], TYPE == kE4m3 ? rs[nt][e & 1] : factor, -m[nt][e & 1]);
                if (__builtin_expect(partial, 0)) x[nt][e] = masked(x[nt][e], nt, e);
                over |= x[nt][e] > shift + lag;
            }
        if (__builtin_expect(__any_sync(~0u, over), 0)) {
            // raise the references to the maxima; l and O follow
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[e] = s[nt][e] * (TYPE == kE4m3 ? rs[nt][e & 1] : factor);
                    if (partial) z[e] = masked(z[e], nt, e);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(z[e], z[2 + e]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                    const float ref = fmaxf(m[nt][e], top - shift), f = ex2(m[nt][e] - ref);
                    m[nt][e] = ref;
                    l[nt][e] *= f;
#pragma unroll
                    for (int t = 0; t < C::MT; ++t) o[t][nt][e] *= f, o[t][nt][2 + e] *= f;
                    x[nt][e] = z[e] - ref;
                    x[nt][2 + e] = z[2 + e] - ref;
                }
            }
        }
        if (__builtin_expect(a.accumulate, 0)) {
            float *dst = w.scores + ((size_t)state.z * w.score_slots + t0) * w.score_rows + my_rows + 2 * c;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (my_rows + 8 * nt + 2 * c >= w.score_rows) continue;
                if (g < count)
                    *reinterpret_cast<float2 *>(dst + g * w.score_rows + 8 * nt) =
                        make_float2(x[nt][0] + m[nt][0], x[nt][1] + m[nt][1]);
                if (g + 8 < count)
                    *reinterpret_cast<float2 *>(dst + (g + 8) * w.score_rows + 8 * nt) =
                        make_float2(x[nt][2] + m[nt][0], x[nt][3] + m[nt][1]);
            }
        }
        uint32_t ph[NT][2], pl[NT][2], pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = ex2(x[nt][e]);
            l[nt][0] += x[nt][0] + x[nt][2];
            l[nt][1] += x[nt][1] + x[nt][3];
            // P as a sum of 16-bit parts, transposed into B fragments
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float u = x[nt][2 * half], v = x[nt][2 * half + 1];
                if constexpr (TYPE == kBf16) {
                    const uint32_t h = pack_bf16(u, v);
                    float2 f = unpack_bf16(h);
                    u -= f.x, v -= f.y;
                    const uint32_t r = pack_bf16(u, v);
                    ph[nt][half] = transpose8x8(h);
                    pl[nt][half] = transpose8x8(r);
                    if constexpr (C::THIRD) {
                        f = unpack_bf16(r);
                        pt[nt][half] = transpose8x8(pack_bf16(u - f.x, v - f.y));
                    }
                } else {
                    const uint32_t h = pack_f16(u, v);
                    const float2 f = unpack_f16(h);
                    ph[nt][half] = transpose8x8(h);
                    pl[nt][half] = transpose8x8(pack_f16((u - f.x) * 4096.f, (v - f.y) * 4096.f));
                }
            }
        }

        // ---- O^T += V^T P^T ----
        // V^T's A fragments: tile t of chunk q covers elements t (rows g) and t + E/2 (rows g + 8) of the chunk
        auto v_chunk = [&](int q, uint32_t (&x)[4][4]) {
            // slots 2c, 2c + 1, 2c + 8, 2c + 9, the thread's chunk 8 q + g (of 8 bytes where a row has but 64)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 2 * c + (j & 1) + 8 * (j >> 1);
                if (C::VB == 16) {
                    const uint4 v = lds128(src_v + chunk_place<C>(row, 8 * q + g));
                    x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
                } else {
                    const uint2 v = lds64(src_v + chunk_place<C>(row, g >> 1) + 8 * (g & 1));
                    x[j][0] = v.x, x[j][1] = v.y, x[j][2] = x[j][3] = 0u;
                }
            }
            if (__builtin_expect((state.x & 63) != 16, 0)) {   // what lies past the step's slots, or where no copy landed
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (state.x & kMissing || 2 * c + (j & 1) + 8 * (j >> 1) >= count)
                        x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0u;
            }
        };
        // elements e and e + 1 (e even) of two slots, each pair a half-word pair of an A fragment
        auto v_pairs = [&](uint32_t lo, uint32_t hi, int e, uint32_t *x0, uint32_t *x1) {
            if constexpr (TYPE != kE4m3) *x0 = __byte_perm(lo, hi, 0x5410), *x1 = __byte_perm(lo, hi, 0x7632);
            else e4m3x4_to_f16x2(__byte_perm(lo, hi, e & 2 ? 0x7362 : 0x5140), x0, x1);
        };
        // sum += V^T by the second part of P^T; LOW_SUM: the sum holds nothing else yet
        auto add_low = [&](float (&sum)[4], const uint32_t (&v)[4], int nt) {
            mma16816<TYPE>(sum, v[0], v[1], v[2], v[3], pl[nt][0], pl[nt][1]);
            if constexpr (C::LOW_SUM)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] *= 1.f / 4096.f;
        };
        constexpr int per_word = 4 / C::ESZ;
        bool careful = false;
        if (DRAFT && __builtin_expect(a.S > 1 && partial, 0)) {
            // a slot hidden from some rows: 0 * NaN and 0 * inf must not reach them
            bool odd = false;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                uint32_t x[4][4];
                v_chunk(q, x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = x[j][e];
                        if constexpr (TYPE == kE4m3) {
                            const uint32_t y = ~v & 0x7F7F7F7Fu;          // a zero byte: NaN
                            odd |= ((y - 0x01010101u) & ~y & 0x80808080u) != 0u;
                        } else {
                            constexpr uint32_t ex = TYPE == kBf16 ? 0x7F80u : 0x7C00u;
                            odd |= (v & ex) == ex || (v >> 16 & ex) == ex;
                        }
                    }
            }
            careful = __any_sync(~0u, odd);
        }
        if (!DRAFT || __builtin_expect(!careful, 1)) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                uint32_t x[4][4];
                v_chunk(q, x);
#pragma unroll
                for (int t = 0; t < E / 2; t += 2) {
                    const int e0 = t, e1 = t + E / 2;
                    uint32_t f[2][4];
                    v_pairs(x[0][e0 / per_word], x[1][e0 / per_word], e0, &f[0][0], &f[1][0]);
                    v_pairs(x[0][e1 / per_word], x[1][e1 / per_word], e1, &f[0][1], &f[1][1]);
                    v_pairs(x[2][e0 / per_word], x[3][e0 / per_word], e0, &f[0][2], &f[1][2]);
                    v_pairs(x[2][e1 / per_word], x[3][e1 / per_word], e1, &f[0][3], &f[1][3]);
                    uint32_t low[2][4];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int z = 0; z < 4; ++z) low[y][z] = C::LOW_V ? f16x2_down12(f[y][z]) : f[y][z];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float(&acc)[4] = o[q * (E / 2) + t + y][nt];
                            const uint32_t(&v)[4] = f[y];
                            float part[4] = {0.f, 0.f, 0.f, 0.f};
                            float(&sum)[4] = C::fresh ? part : acc;
                            if constexpr (C::THIRD) mma16816<TYPE>(sum, v[0], v[1], v[2], v[3], pt[nt][0], pt[nt][1]);
                            add_low(sum, low[y], nt);
                            mma16816<TYPE>(sum, v[0], v[1], v[2], v[3], ph[nt][0], ph[nt][1]);
                            if (C::fresh)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[e] += part[e];
                        }
                }
            }
        } else {
            // one slot at a time, added only to the rows that see it
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
                const uint32_t m0 = (j == 2 * c ? 0xFFFFu : 0u) | (j == 2 * c + 1 ? 0xFFFF0000u : 0u);
                const uint32_t m1 = (j == 2 * c + 8 ? 0xFFFFu : 0u) | (j == 2 * c + 9 ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    uint32_t x[4][4];
                    v_chunk(q, x);
#pragma unroll
                    for (int t = 0; t < E / 2; t += 2) {
                        const int e0 = t, e1 = t + E / 2;
                        uint32_t f[2][4];
                        v_pairs(x[0][e0 / per_word], x[1][e0 / per_word], e0, &f[0][0], &f[1][0]);
                        v_pairs(x[0][e1 / per_word], x[1][e1 / per_word], e1, &f[0][1], &f[1][1]);
                        v_pairs(x[2][e0 / per_word], x[3][e0 / per_word], e0, &f[0][2], &f[1][2]);
                        v_pairs(x[2][e1 / per_word], x[3][e1 / per_word], e1, &f[0][3], &f[1][3]);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t a0 = f[y][0] & m0, a1 = f[y][1] & m0, a2 = f[y][2] & m1, a3 = f[y][3] & m1;
                                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                                if constexpr (C::THIRD) mma16816<TYPE>(acc, a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                                uint32_t low[4] = {a0, a1, a2, a3};
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    if (C::LOW_V) low[z] = f16x2_down12(low[z]);
                                add_low(acc, low, nt);
                                mma16816<TYPE>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (t0 + j < limit(nt, e)) o[q * (E / 2) + t + y][nt][e] += acc[e];
                            }
                    }
                }
            }
        }
        __syncwarp();                                 // every lane has read its chunks and the state
        if (GW > 1 && lane == 0) mbar_arrive(&s_free[group * NS + stage]);

        // ---- end of a piece ----
        const bool ended = state.x & kLast, last = left == 1;
        if (__builtin_expect(ended || last, 0)) {
            fresh = true;
            const int here = state.z, b = quotient(here, w.tiles_div), sg = here - b * tiles;
            const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
            const float vs = TYPE == kE4m3 ? a.c.v_scale[kh] : 1.f;
            const bool whole = ended && began_here;
            const int slot = 2 * group + (began_here ? 1 : 0), row0 = slot * rows + my_rows;
            if (whole && a.accumulate && lane == 0 && mate == 0) w.span[here] = make_int2(blockIdx.x, 1);
            if (!whole && lane == 0 && mate == 0) s_piece[slot] = make_int2(here, (ended ? 1 : 0) | (last ? 0 : 2));
            // 8 rows at a time through shared memory: the stage just read (a group's
            // warps: a place of their own), or, with the range done and read by the
            // whole group, the ring, where an open piece stays for the join
            if (GW > 1 && last && !mbar_wait(&s_free[group * NS + stage], phase) && lane == 0)
                raise_device_error(a.err, kErrTimeout);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float4 *slab = reinterpret_cast<float4 *>(last     ? ring + my_rows * DP * 4 + nt * 32 * DP
                                                          : GW > 1 ? smem + G * C::ring + warp * C::slab
                                                                   : ring + stage * C::stage);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
                    if (g == 0) s_ml[row0 + 8 * nt + 2 * c + e] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int x = 0; x < E; x += 4) {
                            auto at = [&](int y) {
                                return y < E / 2 ? o[q * (E / 2) + y][nt][e] : o[q * (E / 2) + y - E / 2][nt][2 + e];
                            };
                            slab[slab_place<C>(2 * c + e, ((8 * q + g) * E + x) / 4)] =
                                make_float4(at(x), at(x + 1), at(x + 2), at(x + 3));
                        }
                }
                __syncwarp();
                if (whole) {
#pragma unroll 1
                    for (int i = lane; i < 8 * (DP / 4); i += 32) {
                        const int r = i / (DP / 4), d = 4 * (i - r * (DP / 4));
                        const RowRef ref = row_ref(a, w, b, kh, tile * rows + my_rows + 8 * nt + r);
                        const float2 ml = s_ml[row0 + 8 * nt + r];
                        if (!ref.real) continue;
                        if (d < D) {
                            float4 v = slab[slab_place<C>(r, d / 4)];
                            if constexpr (TYPE != kE4m3) v = with_infinities(a, ref, b, kh, d, v, ml.y);
                            store_out4(a, ref.head * D + d, v, row_factor(ml.y, vs));
                        }
                        if (d == 0 && a.lse) a.lse[ref.head] = row_lse(ml.x, ml.y);
                    }
                } else if (!last) {
                    float4 *keep = reinterpret_cast<float4 *>(w.head_o) +
                                   (((size_t)blockIdx.x * W + warp) * NT + nt) * 2 * DP;
#pragma unroll 1
                    for (int i = lane; i < 2 * DP; i += 32) keep[i] = slab[i];
                }
                __syncwarp();
            }
            // the stage is written next by a copy, another proxy
            if (GW == 1 && !last) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
        }
        issue(true, phase);
        if (++stage == NS) stage = 0, phase ^= 1u;
    }

    // ---- join the block's open pieces, in order: a segment has at most one per group ----
    __syncthreads();
    const int2 piece = lane < 2 * G ? s_piece[lane] : make_int2(-1, 0);
    const uint32_t before = __ballot_sync(~0u, piece.x >= 0) & ((1u << lane) - 1u);
    static_assert(2 * G <= 32, "a lane per piece");
    const int prior = __shfl_sync(~0u, piece.x, before ? 31 - __clz(before) : lane);
    uint32_t leaders = __ballot_sync(~0u, piece.x >= 0 && (before == 0u || prior != piece.x));
    const uint32_t in_work = __ballot_sync(~0u, piece.y & 2);
    for (; leaders; leaders &= leaders - 1u) {
        const int first = __ffs(leaders) - 1, seg = __shfl_sync(~0u, piece.x, first);
        const uint32_t members = __ballot_sync(~0u, piece.x == seg);
        const bool starts = first & 1, ends = __shfl_sync(~0u, piece.y, 31 - __clz(members)) & 1;
        const bool whole = starts && ends;
        const int b = quotient(seg, w.tiles_div), sg = seg - b * tiles;
        const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
        const float vs = TYPE == kE4m3 ? a.c.v_scale[kh] : 1.f;
        const size_t out = ((size_t)blockIdx.x * 2 + (starts ? 1 : 0)) * rows;
#pragma unroll 1
        for (int i = tid; i < rows * (DP / 4); i += C::threads) {
            const int r = i / (DP / 4), d = 4 * (i - r * (DP / 4));
            const RowRef ref = row_ref(a, w, b, kh, tile * rows + r);
            if (!ref.real) continue;
            float mm = kNoRef, ll = 0.f;
#pragma unroll 1
            for (uint32_t y = members; y; y &= y - 1u) mm = fmaxf(mm, s_ml[(__ffs(y) - 1) * rows + r].x);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (uint32_t y = members; y; y &= y - 1u) {
                const int x = __ffs(y) - 1;
                const float2 ml = s_ml[x * rows + r];
                const float f = ex2(ml.x - mm);
                ll += ml.y * f;
                // rows lie as the group's warps left them, 8 at a time
                const float4 *src = in_work >> x & 1u
                                        ? reinterpret_cast<const float4 *>(w.head_o) +
                                              ((size_t)blockIdx.x * G + (x >> 1)) * rows * (DP / 4)
                                        : reinterpret_cast<const float4 *>(smem + (x >> 1) * C::ring);
                const float4 v = src[(r >> 3) * 2 * DP + slab_place<C>(r & 7, d / 4)];
                sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
            }
            if (whole) {
                if constexpr (TYPE != kE4m3)
                    if (d < D) sum = with_infinities(a, ref, b, kh, d, sum, ll);
                if (d < D) store_out4(a, ref.head * D + d, sum, row_factor(ll, vs));
                if (d == 0 && a.lse) a.lse[ref.head] = row_lse(mm, ll);
            } else {
                *reinterpret_cast<float4 *>(w.part_o + (out + r) * DP + d) = sum;
                if (d == 0) w.part_ml[out + r] = make_float2(mm, ll);
            }
        }
        if (tid == 0 && starts) {
            const int2 span = make_int2(blockIdx.x, whole       ? 1
                                                    : w.ranks > 0 ? shared_by
                                                                  : blocks_spanned(b, sg, blockIdx.x, chunk, s_prefix, tiles));
            if (!whole && w.ranks == 0) w.open[blockIdx.x] = make_int2(seg, span.y);
            if (a.accumulate) w.span[seg] = span;
        }
    }

    // ---- a cluster's blocks join their pieces of the segment, some rows each ----
    if (w.ranks > 1) {
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        if (shared_by < 2) return;
        const int seg = blockIdx.x / w.ranks, b = quotient(seg, w.tiles_div), sg = seg - b * tiles;
        const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
        const float vs = TYPE == kE4m3 ? a.c.v_scale[kh] : 1.f;
#pragma unroll 1
        for (int i = tid; i < (rows + w.ranks - 1 - rank) / w.ranks * (DP / 4); i += C::threads) {
            const int y = i / (DP / 4), r = rank + y * w.ranks, d = 4 * (i - y * (DP / 4));
            const RowRef ref = row_ref(a, w, b, kh, tile * rows + r);
            if (!ref.real) continue;
            float2 ml[kMaxRanks];
            float4 v[kMaxRanks];
            float mm = kNoRef, ll = 0.f;
#pragma unroll
            for (int x = 0; x < kMaxRanks; ++x) {
                const size_t at = ((size_t)(blockIdx.x - rank + x) * 2 + (x == 0 ? 1 : 0)) * rows + r;
                ml[x] = make_float2(kNoRef, 0.f);
                v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x < shared_by) {
                    ml[x] = __ldcg(w.part_ml + at);
                    v[x] = __ldcg(reinterpret_cast<const float4 *>(w.part_o + at * DP + d));
                }
            }
#pragma unroll
            for (int x = 0; x < kMaxRanks; ++x) mm = fmaxf(mm, ml[x].x);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kMaxRanks; ++x) {
                const float f = ex2(ml[x].x - mm);
                ll += ml[x].y * f;
                sum.x += v[x].x * f, sum.y += v[x].y * f, sum.z += v[x].z * f, sum.w += v[x].w * f;
            }
            if constexpr (TYPE != kE4m3)
                if (d < D) sum = with_infinities(a, ref, b, kh, d, sum, ll);
            if (d < D) store_out4(a, ref.head * D + d, sum, row_factor(ll, vs));
            if (d == 0 && a.lse) a.lse[ref.head] = row_lse(mm, ll);
        }
    }
}

}  // namespace qg
