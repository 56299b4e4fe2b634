// attn_paged.cuh -- attention of a few new tokens over a paged key-value cache
// (qattn_paged): the streaming kernel.
//
// Row (b, s, h) sees the slots t < len_b - S + 1 + s:
//   z_t = scale q . k_t,   o = sum_t exp(z_t - lse) v_t,   lse = log sum_t exp(z_t).
// The cache is read once and little is computed per byte, so the call is bound
// by HBM and everything serves keeping its reads in flight.
//
// Work.  The rows of one sequence that share a key-value head, R = S * group,
// form tiles of 8 * NT rows; a (sequence, head, tile) is a segment of
// ceil(len / 16) steps of 16 slots.  All segments' steps, laid end to end, are
// cut into one equal range per block (one block an SM) and each range into one
// per warp: unequal lengths balance without the host knowing them.  A warp
// keeps the running maximum and sum of each row and O in registers (online
// softmax).  A segment that ends inside its warp is finished there; pieces of
// one that does not are joined in shared memory after the block's ranges are
// done, and across blocks by a second kernel, always in slot order.  Where
// every segment is short and has an SM to itself, each block takes one whole
// segment instead and the second kernel is not needed.
//
// Loads.  Each warp copies its steps into a ring of its own in shared memory
// (cp.async, NS steps ahead; no block barrier), 512 consecutive bytes of a
// page per instruction.  Copying straight in fragment order (64 and 128 byte
// pieces of many rows per instruction) read 5.2 TB/s where this order reads
// 6.8.  The 16-byte chunks of a row are swizzled so that both the copies and
// the fragment reads (16 bytes a thread) are free of bank conflicts.  A
// fragment's k indices are the 8 (or 16) consecutive elements of a chunk: the
// contraction over d may run in any order.
//
// Products.  S^T = K Q^T with the 16 slots as M and 8 rows as N (a decode step
// has few rows), then O^T = V^T P^T; P^T's fragment is the transpose of
// S^T's (movmatrix), V^T's pairs of slots are byte permutes of two loads.
// mma.sync suffices: at the HBM rate 16 slots of 128 dimensions arrive per SM
// every ~350 cycles and need 24 MMAs per 8 rows, a twelfth of its rate.
// Precision: products of 16-bit operands are exact and summed in f32.  P is
// not rounded to one 16-bit value but split into a sum of two (three for f32
// output of a bf16 cache), so it keeps 16 to 24 bits; f16 parts are scaled by
// 2^6 (as are the sums they are divided by) against its subnormals.
// Softmax.  Each row's exponents are taken against a reference that follows
// the running maximum only when a score passes it by more than 2^8: a step
// then needs one vote instead of a maximum over lanes, and p stays <= 2^14.
// e4m3 codes are exact in f16; q over them is scaled per row by a power of two
// into f16's range, which is exact for bf16 values within 2^29 of the largest.
#pragma once

#include <type_traits>

#include "kv_cache.cuh"

namespace qg {

constexpr int kAttnMaxSeq = 2048;     // sequences per launch (their lengths sit in shared memory)

// Workspace of one launch.
struct AttnWork {
    float *part_o;      // [ctas][2][rows][DP]: pieces a block leaves open, at its start (0) and end (1)
    float2 *part_ml;    // [ctas][2][rows]: their maxima (log2 units) and sums
    float *head_o;      // [ctas][warps][rows][DP]: pieces a warp finishes before its range ends
    float *scores;      // accumulate: z in log2 units, [segment][slot][rows]
    int score_slots;    // slots per segment in scores
    int row_tiles;
    int tiles;          // segments per sequence: heads times row tiles
    int whole;          // one block per segment (else equal ranges of steps)
    int ctas;           // blocks of the streaming kernel
    FastDiv tiles_div, row_tiles_div, group_div;
};

template <int TYPE, int DP_, int NT_>
struct AttnCfg {
    static constexpr int DP = DP_, NT = NT_;
    static constexpr int ESZ = TYPE == kE4m3 ? 1 : 2;
    static constexpr int rows = 8 * NT;
    static constexpr int KE = 16 / ESZ;               // elements of a K chunk
    static constexpr int NI = DP * ESZ / 64;          // K chunks a thread holds per slot (4 threads a slot)
    static constexpr int E = DP / 8 < KE ? DP / 8 : KE;   // elements of a V chunk (8 threads a slot)
    static constexpr int VB = E * ESZ;                // its bytes: 16, or 8
    static constexpr int NQ = DP / (8 * E);           // V chunks a thread holds per slot
    static constexpr int MT = DP / 16;                // 16-row tiles of O^T
    static constexpr int RB = DP * ESZ;               // bytes of a row
    static constexpr int NC = RB / 16;                // 16-byte chunks of a row: 4, 8, 16 or 32
    static constexpr int NL = NC / 2;                 // copies of 512 bytes for 16 rows
    static constexpr int RPL = 32 / NC;               // rows one covers
    static constexpr int k_bytes = 16 * RB;
    static constexpr int stage = 2 * k_bytes;         // 16 slots of K and V
    // 192 KB in flight per SM at most; eight warps, four where a stage is 16 KB
    static constexpr int W = stage > 8192 ? 4 : 8;
    static constexpr int NS0 = 196608 / (W * stage);
    static constexpr int NS = NS0 > 8 ? 8 : NS0;
    static constexpr int ring = NS * stage;           // per warp
    static_assert(ring >= rows * DP * 4, "a warp's open piece takes the place of its ring");
    static constexpr int threads = 32 * W;
};

// dynamic shared memory: rings, row statistics of open pieces, step masks,
// piece descriptors, then prefix [n + 1] and lengths [n]
// Where chunk u = row * NC + chunk of a step sits: the low three bits (its bank
// group) are exchanged by row.  A fragment read takes, per eight lanes, chunks
// x .. x + 3 of two neighbouring rows of K, two neighbouring chunks of four
// even (or odd) rows of V.
template <class C>
__device__ __forceinline__ constexpr int k_place(int row, int chunk) {
    return (row * C::NC + chunk) ^ (C::NC >= 8 ? (row & 1) << 2 : 0);
}
template <class C>
__device__ __forceinline__ constexpr int v_place(int row, int chunk) {
    return (row * C::NC + chunk) ^ (row >> 1 & 3) << 1;
}

template <class C>
__host__ __device__ constexpr size_t attn_fixed_smem() {
    return (size_t)C::W * C::ring + C::W * 2 * C::rows * sizeof(float2) + C::W * C::NS * 4 + C::W * 2 * 8;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int S>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const char *src) {   // [dst] <- [src + S]
    asm volatile("cp.async.cg.shared.global [%0], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(S) : "memory");
}
// fn(integral_constant<int, 0>) .. fn(integral_constant<int, N - 1>): unrolled, with the index a constant
template <int N, int I = 0, class Fn>
__device__ __forceinline__ void unrolled(Fn fn) {
    if constexpr (I < N) {
        fn(std::integral_constant<int, I>());
        unrolled<N, I + 1>(fn);
    }
}
__device__ __forceinline__ float ex2(float x) {       // 2^x, 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Steps of 16 slots of all sequences: lengths and their running sums (n + 1)
// into shared memory; THREADS threads, `s_sum` one int per warp.
template <int THREADS>
__device__ __forceinline__ void scan_steps(const AttnArgs &a, int *s_len, int *s_prefix, int *s_sum, int *err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n_seq;
    const int per = (n + THREADS - 1) / THREADS;
    int sum = 0;
    for (int i = tid * per; i < (tid + 1) * per && i < n; ++i) {
        const int len = seq_len(a.lens, i, a.max_len, err);
        s_len[i] = len;
        sum += (len + 15) >> 4;
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
        at += (s_len[i] + 15) >> 4;
    }
    if (tid == THREADS - 1) s_prefix[n] = at;
    __syncthreads();
}

// Steps per block where all are cut into equal ranges: at least one per warp.
__device__ __forceinline__ int steps_per_block(int total, int ctas, int warps) {
    const int chunk = (total + ctas - 1) / ctas;
    return chunk < warps ? warps : chunk;
}

// Place of a global step: its sequence, segment there, step of that and steps of the segment.
struct Place { int b, seg, i, n; };
__device__ __forceinline__ Place locate(int step, const int *s_prefix, int n, const AttnWork &w) {
    Place p;
    const int x = quotient(step, w.tiles_div);
    int lo = 0, hi = n - 1;                          // the last b with prefix[b] <= x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    p.b = lo;
    p.n = s_prefix[lo + 1] - s_prefix[lo];
    const int rem = step - s_prefix[lo] * w.tiles;
    p.seg = rem / p.n;
    p.i = rem - p.seg * p.n;
    return p;
}

template <int TYPE, int DP_, int NT_>
__global__ void __launch_bounds__(AttnCfg<TYPE, DP_, NT_>::threads, 1)
    attn_stream_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnWork w) {
    using C = AttnCfg<TYPE, DP_, NT_>;
    constexpr int DP = C::DP, NT = C::NT, W = C::W, NS = C::NS, NI = C::NI, E = C::E, NQ = C::NQ, rows = C::rows;
    extern __shared__ __align__(128) char smem[];
    float2 *s_ml = reinterpret_cast<float2 *>(smem + W * C::ring);            // [W][2][rows]
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_ml + W * 2 * rows);     // [W][NS]
    int2 *s_piece = reinterpret_cast<int2 *>(s_mask + W * NS);                // [W][2]: {segment or -1, 1: ended | 2: in head_o}
    int *s_prefix = reinterpret_cast<int *>(s_piece + W * 2);                 // [n + 1]
    int *s_len = s_prefix + a.n_seq + 1;                                      // [n]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int n = a.n_seq, D = a.c.dim;
    const int tiles = w.tiles;

    // dependents may start once the lengths are final: the second kernel reads them before its own wait
    griddep_wait();
    griddep_launch_dependents();

    scan_steps<C::threads>(a, s_len, s_prefix, reinterpret_cast<int *>(smem), blockIdx.x == 0 ? a.err : nullptr);
    int c0, c1;
    if (w.whole) {
        const int b = quotient(blockIdx.x, w.tiles_div), steps = s_prefix[b + 1] - s_prefix[b];
        c0 = s_prefix[b] * tiles + (blockIdx.x - b * tiles) * steps;
        c1 = c0 + steps;
    } else {
        const int total = s_prefix[n] * tiles, chunk = steps_per_block(total, gridDim.x, W);
        c0 = (int)(blockIdx.x * chunk) < total ? blockIdx.x * chunk : total;
        c1 = c0 + chunk < total ? c0 + chunk : total;
    }

    // sequences without a slot have no steps: their rows are empty
    for (int b = blockIdx.x; b < n; b += gridDim.x) {
        if (s_len[b] != 0) continue;
        const int quads = D / 4, count = a.S * a.n_q_heads;
        for (int i = tid; i < count * quads; i += C::threads)
            store_out4(a, ((size_t)b * count) * D + 4 * (size_t)i, make_float4(0.f, 0.f, 0.f, 0.f), 1.f);
        if (a.lse)
            for (int i = tid; i < count; i += C::threads) a.lse[(size_t)b * count + i] = -INFINITY;
    }
    if (c0 >= c1) return;

    const int w0 = c0 + (int)((long long)(c1 - c0) * warp / W);
    const int w1 = c0 + (int)((long long)(c1 - c0) * (warp + 1) / W);
    char *ring = smem + warp * C::ring;
    const uint32_t ring_a = smem_addr(ring);
    if (lane < 2) s_piece[2 * warp + lane] = make_int2(-1, 0);

    auto advance = [&](Place &p) {
        if (++p.i < p.n) return;
        p.i = 0;
        if (++p.seg < tiles) return;
        p.seg = 0;
        do ++p.b;
        while (p.b < n && s_prefix[p.b + 1] == s_prefix[p.b]);
        p.n = p.b < n ? s_prefix[p.b + 1] - s_prefix[p.b] : 1;
    };

    // ---- loads ----
    // `simple`: the 16 slots of a step lie in one page and rows fill the padded size
    const bool simple = D == DP && a.c.page % 16 == 0;
    Place ip = locate(w0 < w1 ? w0 : c0, s_prefix, n, w), p = ip;
    int ip_kh = quotient(ip.seg, w.row_tiles_div);
    int issued = w0, istage = 0;
    // the page of the next step to load is looked up one step early: of its
    // first slot where the step is simple, else of slot `lane` by lanes 0-15
    int look_page = 0, look_off = 0;
    auto look = [&]() {
        if (issued >= w1) return;
        const int t = 16 * ip.i + (simple ? 0 : lane);
        if (simple || (lane < 16 && t < s_len[ip.b])) {
            int index;
            split_slot(a.c, t, &index, &look_off);
            look_page = __ldg(a.table + (size_t)ip.b * a.table_stride + index);
        }
    };
    // copy n of a step moves chunk lane % NC of row n * RPL + lane / NC
    const int l_row = lane / C::NC, l_chunk = lane % C::NC;
    const long long l_off = l_row * a.c.token_b + 16 * l_chunk, copy_b = C::RPL * a.c.token_b;
    const bool in_row = 16 * l_chunk < D * C::ESZ;
    auto issue = [&]() {
        if (issued < w1) {
            const uint32_t dst = ring_a + istage * C::stage;
            const int t0 = 16 * ip.i, len = s_len[ip.b];
            if (simple && t0 + 16 <= len && (unsigned)look_page < (unsigned)a.c.n_pages) {
                if (lane == 0) s_mask[warp * NS + istage] = 0xFFFFu;
                const long long base =
                    look_page * a.c.page_b + ip_kh * a.c.head_b + look_off * a.c.token_b + l_off;
                const char *k = a.c.k + base, *v = a.c.v + base;
                if (copy_b == 512) {
                    unrolled<C::NL>([&](auto n) {
                        cp_async16_at<512 * n>(dst + 16 * k_place<C>(n * C::RPL + l_row, l_chunk), k);
                    });
                    unrolled<C::NL>([&](auto n) {
                        cp_async16_at<512 * n>(dst + C::k_bytes + 16 * v_place<C>(n * C::RPL + l_row, l_chunk), v);
                    });
                } else {
#pragma unroll
                    for (int n = 0; n < C::NL; ++n) {
                        cp_async16_at<0>(dst + 16 * k_place<C>(n * C::RPL + l_row, l_chunk), k);
                        cp_async16_at<0>(dst + C::k_bytes + 16 * v_place<C>(n * C::RPL + l_row, l_chunk), v);
                        k += copy_b, v += copy_b;
                    }
                }
            } else {
                const bool in = lane < 16 && t0 + lane < len;
                const bool ok = in && (unsigned)look_page < (unsigned)a.c.n_pages;
                const uint32_t good = __ballot_sync(~0u, ok), bad = __ballot_sync(~0u, in && !ok);
                if (lane == 0) {
                    s_mask[warp * NS + istage] = good | bad << 16;
                    if (bad) raise_device_error(a.err, kErrPage);
                }
                const long long off = ok ? look_page * a.c.page_b + ip_kh * a.c.head_b +
                                               (look_off + (simple ? lane : 0)) * a.c.token_b
                                         : 0;
#pragma unroll
                for (int n = 0; n < C::NL; ++n) {
                    const int row = n * C::RPL + l_row;
                    const long long at = __shfl_sync(~0u, off, row) + (in_row ? 16 * l_chunk : 0);
                    const bool take = in_row && (good >> row & 1u);
                    cp_async16(dst + 16 * k_place<C>(row, l_chunk), a.c.k + at, take);
                    cp_async16(dst + C::k_bytes + 16 * v_place<C>(row, l_chunk), a.c.v + at, take);
                }
            }
            ++issued;
            advance(ip);
            if (ip.i == 0) ip_kh = quotient(ip.seg, w.row_tiles_div);
            look();
        }
        cp_async_commit();
        if (++istage == NS) istage = 0;
    };
    look();
#pragma unroll 1
    for (int i = 0; i < NS; ++i) issue();

    // ---- the warp's range ----
    float o[C::MT][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t qf[NT][NI][C::ESZ == 1 ? 8 : 4];
    float rs[NT][2];                                  // score factor of the thread's rows (e4m3: per row)
    int lim[NT][2];                                   // slots they see
    const float factor = a.scale * 1.44269504088896340736f;
    constexpr float shift = TYPE == kBf16 ? 0.f : 6.f;
    const bool third = TYPE == kBf16 && a.o_type == kF32;
    int hidden_from = 0;                              // first slot that some row does not see
    bool fresh = true;                                // at the start of a piece
    int stage = 0;
    bool began_here = false;

#pragma unroll 1
    for (int step = w0; step < w1; ++step) {
        if (fresh) {
            const int kh = quotient(p.seg, w.row_tiles_div), tile = p.seg - kh * w.row_tiles, len = s_len[p.b];
            hidden_from = len - a.S + 1;
            fresh = false;
            began_here = p.i == 0;
            // Q as the B operand: row g of each 8, the thread's chunks
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const RowRef r = row_ref(a, w, p.b, kh, tile * rows + 8 * nt + g);
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + ((size_t)p.b * a.S + r.s) * a.q_stride +
                                    (size_t)r.q_head * D;
                if constexpr (TYPE != kE4m3) {
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int d = (4 * i + c) * 8;
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (r.real && d < D) v = *reinterpret_cast<const uint4 *>(q + d);
                        qf[nt][i][0] = v.x, qf[nt][i][1] = v.y, qf[nt][i][2] = v.z, qf[nt][i][3] = v.w;
                    }
                } else {
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int d = (4 * i + c) * 16;
                        uint4 v[2] = {};
                        if (r.real && d < D)
                            v[0] = *reinterpret_cast<const uint4 *>(q + d),
                            v[1] = *reinterpret_cast<const uint4 *>(q + d + 8);
                        const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            qf[nt][i][u] = x[u];
                            const float2 f = a.q_type == kF16 ? unpack_f16(x[u]) : unpack_bf16(x[u]);
                            if (fabsf(f.x) < INFINITY) top = fmaxf(top, fabsf(f.x));
                            if (fabsf(f.y) < INFINITY) top = fmaxf(top, fabsf(f.y));
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    // largest |q| of the row into [2^14, 2^15)
                    int ex = 141 - (int)(__float_as_uint(top) >> 23);
                    ex = top == 0.f ? 0 : ex > 100 ? 100 : ex < -100 ? -100 : ex;
                    const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float2 f = a.q_type == kF16 ? unpack_f16(qf[nt][i][u]) : unpack_bf16(qf[nt][i][u]);
                            qf[nt][i][u] = pack_f16(f.x * up, f.y * up);
                        }
                    const float down = factor * __ldg(a.c.k_scale + kh) * __uint_as_float((uint32_t)(127 - ex) << 23);
                    rs[nt][0] = __shfl_sync(~0u, down, 8 * c);
                    rs[nt][1] = __shfl_sync(~0u, down, 8 * c + 4);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int s = quotient(tile * rows + 8 * nt + 2 * c + e, w.group_div);
                    lim[nt][e] = len - a.S + 1 + (s < a.S ? s : a.S - 1);
                    m[nt][e] = kNoRef;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int t = 0; t < C::MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
            }
        }

        cp_async_wait<NS - 1>();
        __syncwarp();
        const uint32_t mask = s_mask[warp * NS + stage];
        const uint32_t src = ring_a + stage * C::stage;

        // ---- S^T = K Q^T, in two chains ----
        float s[NT][4], s1[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = s1[nt][e] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            // slots g and g + 8, chunk c + 4 i
            const uint4 x = lds128(src + 16 * k_place<C>(g, 4 * i + c)), y = lds128(src + 16 * k_place<C>(g + 8, 4 * i + c));
            const uint32_t kx[4] = {x.x, x.y, x.z, x.w}, ky[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int u = 0; u < C::KE / 4; ++u) {
                uint32_t a0, a1, a2, a3;
                if constexpr (TYPE != kE4m3) {
                    a0 = kx[2 * u], a1 = ky[2 * u], a2 = kx[2 * u + 1], a3 = ky[2 * u + 1];
                } else {
                    a0 = e4m3x2_to_f16x2(kx[u]), a2 = e4m3x2_to_f16x2(kx[u] >> 16);
                    a1 = e4m3x2_to_f16x2(ky[u]), a3 = e4m3x2_to_f16x2(ky[u] >> 16);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<TYPE>(u & 1 ? s1[nt] : s[nt], a0, a1, a2, a3, qf[nt][i][2 * u], qf[nt][i][2 * u + 1]);
            }
        }

        // ---- exponents against the rows' references; thread: slots g, g + 8 by rows 2c, 2c + 1 ----
        const int t0 = 16 * p.i;
        const bool partial = mask != 0xFFFFu || (a.S > 1 && t0 + 16 > hidden_from);
        // slots past the end are past every limit; NaN where the slot's page is not in the pool
        auto masked = [&](float z, int nt, int e) {
            const int j = g + 8 * (e >> 1);
            if (t0 + j >= lim[nt][e & 1]) return -INFINITY;
            return mask >> (16 + j) & 1u ? NAN : z;
        };
        uint32_t ph[NT][2], pl[NT][2], pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] += s1[nt][e];
                x[e] = fmaf(s[nt][e], TYPE == kE4m3 ? rs[nt][e & 1] : factor, -m[nt][e & 1]);
                if (partial) x[e] = masked(x[e], nt, e);
            }
            constexpr float most = shift + 8.f;
            if (__any_sync(~0u, x[0] > most || x[1] > most || x[2] > most || x[3] > most)) {
                // raise the references to the maxima; l and O follow
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
                    x[e] = z[e] - ref;
                    x[2 + e] = z[2 + e] - ref;
                }
            }
            if (a.accumulate) {
                float *dst = w.scores + ((size_t)(p.b * tiles + p.seg) * w.score_slots + t0) * rows + 8 * nt + 2 * c;
                *reinterpret_cast<float2 *>(dst + (size_t)g * rows) = make_float2(x[0] + m[nt][0], x[1] + m[nt][1]);
                *reinterpret_cast<float2 *>(dst + (size_t)(g + 8) * rows) = make_float2(x[2] + m[nt][0], x[3] + m[nt][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ex2(x[e]);
            l[nt][0] += x[0] + x[2];
            l[nt][1] += x[1] + x[3];
            // P as a sum of 16-bit parts, transposed into B fragments
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float u = x[2 * half], v = x[2 * half + 1];
                if constexpr (TYPE == kBf16) {
                    const uint32_t h = pack_bf16(u, v);
                    float2 f = unpack_bf16(h);
                    u -= f.x, v -= f.y;
                    const uint32_t r = pack_bf16(u, v);
                    ph[nt][half] = transpose8x8(h);
                    pl[nt][half] = transpose8x8(r);
                    if (third) {
                        f = unpack_bf16(r);
                        pt[nt][half] = transpose8x8(pack_bf16(u - f.x, v - f.y));
                    }
                } else {
                    const uint32_t h = pack_f16(u, v);
                    const float2 f = unpack_f16(h);
                    ph[nt][half] = transpose8x8(h);
                    pl[nt][half] = transpose8x8(pack_f16(u - f.x, v - f.y));
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
                    const uint4 v = lds128(src + C::k_bytes + 16 * v_place<C>(row, 8 * q + g));
                    x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
                } else {
                    const uint2 v = lds64(src + C::k_bytes + 16 * v_place<C>(row, g >> 1) + 8 * (g & 1));
                    x[j][0] = v.x, x[j][1] = v.y, x[j][2] = x[j][3] = 0u;
                }
            }
        };
        auto v_pair = [&](uint32_t lo, uint32_t hi, int e) -> uint32_t {   // element e of two slots' words
            if constexpr (TYPE != kE4m3) return __byte_perm(lo, hi, e & 1 ? 0x7632 : 0x5410);
            const uint32_t two = __byte_perm(lo, hi, e & 2 ? 0x7362 : 0x5140);
            return e4m3x2_to_f16x2(e & 1 ? two >> 16 : two);
        };
        constexpr int per_word = 4 / C::ESZ;
        bool careful = false;
        if (a.S > 1 && partial) {
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
        auto add_pv = [&](auto with_third) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                uint32_t x[4][4];
                v_chunk(q, x);
#pragma unroll
                for (int t = 0; t < E / 2; ++t) {
                    const int e0 = t, e1 = t + E / 2;
                    const uint32_t a0 = v_pair(x[0][e0 / per_word], x[1][e0 / per_word], e0);
                    const uint32_t a1 = v_pair(x[0][e1 / per_word], x[1][e1 / per_word], e1);
                    const uint32_t a2 = v_pair(x[2][e0 / per_word], x[3][e0 / per_word], e0);
                    const uint32_t a3 = v_pair(x[2][e1 / per_word], x[3][e1 / per_word], e1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float(&acc)[4] = o[q * (E / 2) + t][nt];
                        if constexpr (with_third) mma16816<TYPE>(acc, a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                        mma16816<TYPE>(acc, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                        mma16816<TYPE>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                    }
                }
            }
        };
        if (!careful) {
            if (TYPE == kBf16 && third) add_pv(std::true_type());
            else add_pv(std::false_type());
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
                    for (int t = 0; t < E / 2; ++t) {
                        const int e0 = t, e1 = t + E / 2;
                        const uint32_t a0 = v_pair(x[0][e0 / per_word], x[1][e0 / per_word], e0) & m0;
                        const uint32_t a1 = v_pair(x[0][e1 / per_word], x[1][e1 / per_word], e1) & m0;
                        const uint32_t a2 = v_pair(x[2][e0 / per_word], x[3][e0 / per_word], e0) & m1;
                        const uint32_t a3 = v_pair(x[2][e1 / per_word], x[3][e1 / per_word], e1) & m1;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            if (TYPE == kBf16 && third) mma16816<TYPE>(acc, a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                            mma16816<TYPE>(acc, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                            mma16816<TYPE>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (t0 + j < lim[nt][e & 1]) o[q * (E / 2) + t][nt][e] += acc[e];
                        }
                    }
                }
            }
        }
        __syncwarp();                                 // every lane has read the mask and its chunks
        issue();
        if (++stage == NS) stage = 0;

        // ---- end of a piece ----
        const bool ended = p.i + 1 == p.n;
        if (ended || step + 1 == w1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
            const int kh = quotient(p.seg, w.row_tiles_div), tile = p.seg - kh * w.row_tiles;
            const float vs = TYPE == kE4m3 ? __ldg(a.c.v_scale + kh) : 1.f;
            const bool whole = ended && began_here;
            // an open piece waits in the ring when the range is done with it, else in the workspace
            float *keep = step + 1 == w1 ? reinterpret_cast<float *>(ring)
                                         : w.head_o + ((size_t)blockIdx.x * W + warp) * rows * DP;
            const int slot = began_here ? 1 : 0;
            if (step + 1 == w1) {
                cp_async_wait<0>();
                __syncwarp();
            }
            if (!whole) {
                if (lane == 0)
                    s_piece[2 * warp + slot] = make_int2(p.b * tiles + p.seg, (ended ? 1 : 0) | (step + 1 == w1 ? 0 : 2));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nt + 2 * c + e;
                    const RowRef ref = row_ref(a, w, p.b, kh, tile * rows + r);
                    if (!ref.real) continue;
                    const float f = row_factor(l[nt][e], vs);
                    if (g == 0) {
                        if (whole) {
                            if (a.lse) a.lse[ref.head] = row_lse(m[nt][e], l[nt][e]);
                        } else {
                            s_ml[(2 * warp + slot) * rows + r] = make_float2(m[nt][e], l[nt][e]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int x = 0; x < E; x += 4) {
                            const int d = (8 * q + g) * E + x;
                            auto at = [&](int y) {
                                return y < E / 2 ? o[q * (E / 2) + y][nt][e] : o[q * (E / 2) + y - E / 2][nt][2 + e];
                            };
                            const float4 v = make_float4(at(x), at(x + 1), at(x + 2), at(x + 3));
                            if (!whole) *reinterpret_cast<float4 *>(keep + r * DP + d) = v;
                            else if (d < D) store_out4(a, ref.head * D + d, v, f);
                        }
                }
            fresh = true;
        }
        advance(p);
    }

    // ---- join the block's open pieces, in order: a segment has at most one per warp ----
    __syncthreads();
    const int2 piece = lane < 2 * W ? s_piece[lane] : make_int2(-1, 0);
    const uint32_t before = __ballot_sync(~0u, piece.x >= 0) & ((1u << lane) - 1u);
    const int prior = __shfl_sync(~0u, piece.x, before ? 31 - __clz(before) : lane);
    uint32_t leaders = __ballot_sync(~0u, piece.x >= 0 && (before == 0u || prior != piece.x));
    const uint32_t in_work = __ballot_sync(~0u, piece.y & 2);
    for (; leaders; leaders &= leaders - 1u) {
        const int first = __ffs(leaders) - 1, seg = __shfl_sync(~0u, piece.x, first);
        const uint32_t members = __ballot_sync(~0u, piece.x == seg);
        const bool starts = first & 1, ends = __shfl_sync(~0u, piece.y, 31 - __clz(members)) & 1, whole = starts && ends;
        const int b = quotient(seg, w.tiles_div), sg = seg - b * tiles;
        const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
        const float vs = TYPE == kE4m3 ? __ldg(a.c.v_scale + kh) : 1.f;
        const size_t out = ((size_t)blockIdx.x * 2 + (starts ? 1 : 0)) * rows;
        for (int i = tid; i < rows * (DP / 4); i += C::threads) {
            const int r = i / (DP / 4), d = 4 * (i - r * (DP / 4));
            const RowRef ref = row_ref(a, w, b, kh, tile * rows + r);
            if (!ref.real) continue;
            float2 ml[W];
            float mm = kNoRef, ll = 0.f;
#pragma unroll
            for (int x = 0; x < W; ++x) {
                const uint32_t has = members >> (2 * x) & 3u;
                ml[x] = has ? s_ml[(2 * x + (has >> 1)) * rows + r] : make_float2(kNoRef, 0.f);
                mm = fmaxf(mm, ml[x].x);
            }
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < W; ++x) {
                if (!(members >> (2 * x) & 3u)) continue;
                const float f = ex2(ml[x].x - mm);
                ll += ml[x].y * f;
                const float *src = in_work & members & 3u << (2 * x)
                                       ? w.head_o + ((size_t)blockIdx.x * W + x) * rows * DP
                                       : reinterpret_cast<const float *>(smem + x * C::ring);
                const float4 v = *reinterpret_cast<const float4 *>(src + r * DP + d);
                sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
            }
            if (whole) {
                if (d < D) store_out4(a, ref.head * D + d, sum, row_factor(ll, vs));
                if (d == 0 && a.lse) a.lse[ref.head] = row_lse(mm, ll);
            } else {
                *reinterpret_cast<float4 *>(w.part_o + (out + r) * DP + d) = sum;
                if (d == 0) w.part_ml[out + r] = make_float2(mm, ll);
            }
        }
    }
}

}  // namespace qg
