// attn_paged.cu -- attention over a paged cache: workspace, launches, and the
// second kernel: the join of segments that several blocks share, and the
// accumulation of attention weights.  The streaming kernel is in attn_paged.cuh.
#include <cudaTypedefs.h>

#include "attn_launch.cuh"

namespace qg {

extern template int launch_attn_stream<kBf16, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2],
                                                     cudaStream_t);
extern template int launch_attn_stream<kBf16, true>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2],
                                                    cudaStream_t);
extern template int launch_attn_stream<kF16, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2],
                                                    cudaStream_t);
extern template int launch_attn_stream<kE4m3, false>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2],
                                                     cudaStream_t);
extern template int launch_attn_stream<kE4m3, true>(const AttnArgs &, const AttnWork &, const CUtensorMap (&)[2],
                                                    cudaStream_t);
extern template AttnPlan attn_plan<kBf16>(int, int);
extern template AttnPlan attn_plan<kF16>(int, int);
extern template AttnPlan attn_plan<kE4m3>(int, int);

namespace {

constexpr long long kEnoughBytes = 128 << 10, kWholeBytes = 384 << 10;
constexpr size_t kScoreBytes = (size_t)1 << 30;
// Slots a thread adds weights for: its chain of dependent reads, not bytes,
// bounds the second kernel (9 sequences of 500 to 8192 slots, 8 heads, 40 query
// heads: 42.4 us a call with one, 39.8 with two, 41.0 with four; 40 sequences
// of 2000 and more: 178, 165, 168).
constexpr int kFinishThreads = 256, kFinishSlots = 2;

// The second kernel of a call.  Its first blocks join segments that several
// blocks of the streaming kernel share: block (x, y) does `per` rows of the
// segment that the streaming kernel's block x left open at its end (its last
// piece, then the first pieces of the blocks after it).  A thread takes four
// elements of a row of every so many pieces, four loads in flight.  The
// further blocks add up attention weights from the scores that the streaming
// kernel left, a thread two slots:
//   weight[t] += sum over the rows of a key-value head of 2^(z_t - lse).
__global__ void __launch_bounds__(kFinishThreads)
    attn_finish_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnWork w, int rows, int dp,
                       int per, int join_blocks) {
    __shared__ float4 s_acc[kFinishThreads];
    __shared__ float s_lse[64];
    const int tid = threadIdx.x, R = a.S * a.group;
    griddep_launch_dependents();

    if ((int)blockIdx.x < join_blocks) {
        griddep_wait();
        const int groups = rows / per, x = blockIdx.x / groups;
        const int2 open = w.open[x];
        if (open.x < 0) return;
        const int pieces = open.y, b = quotient(open.x, w.tiles_div), sg = open.x - b * w.tiles;
        const int kh = quotient(sg, w.row_tiles_div), tile = sg - kh * w.row_tiles;
        const int quads = dp / 4, sets = kFinishThreads / (quads * per);
        const int set = tid / (quads * per), item = tid - set * quads * per, local = item / quads;
        const int r = (blockIdx.x - x * groups) * per + local, d = 4 * (item - local * quads);
        const RowRef ref = row_ref(a, w, b, kh, tile * rows + r);
        auto at = [&](int i) { return ((size_t)(x + i) * 2 + (i == 0 ? 1 : 0)) * rows + r; };
        float m = kNoRef, l = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ref.real) {
            constexpr int kAhead = 4;
            float4 v[kAhead];
            float f[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = set + k * sets;
                f[k] = kNoRef;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < pieces) v[k] = *reinterpret_cast<const float4 *>(w.part_o + at(i) * dp + d), f[k] = w.part_ml[at(i)].x;
            }
#pragma unroll 8
            for (int i = 0; i < pieces; ++i) m = fmaxf(m, w.part_ml[at(i)].x);
#pragma unroll 8
            for (int i = 0; i < pieces; ++i) {
                const float2 y = w.part_ml[at(i)];
                l += y.y * ex2(y.x - m);
            }
            auto add = [&](float4 y, float g) {
                sum.x += y.x * g, sum.y += y.y * g, sum.z += y.z * g, sum.w += y.w * g;
            };
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (set + k * sets < pieces) add(v[k], ex2(f[k] - m));
#pragma unroll 4
            for (int i = set + kAhead * sets; i < pieces; i += sets)
                add(*reinterpret_cast<const float4 *>(w.part_o + at(i) * dp + d), ex2(w.part_ml[at(i)].x - m));
        }
        if (sets > 1) {
            s_acc[tid] = sum;
            __syncthreads();
            if (set > 0) return;
            for (int k = 1; k < sets; ++k) {
                const float4 y = s_acc[k * quads * per + tid];
                sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
            }
        }
        if (!ref.real || set >= sets) return;
        const float vs = a.c.type == kE4m3 ? a.c.v_scale[kh] : 1.f;
        if (d < a.c.dim) {
            if (a.c.type != kE4m3) sum = with_infinities(a, ref, b, kh, d, sum, l);
            store_out4(a, ref.head * a.c.dim + d, sum, row_factor(l, vs));
        }
        if (d == 0 && a.lse) a.lse[ref.head] = row_lse(m, l);
        return;
    }

    const int at = blockIdx.x - join_blocks, heads = a.n_seq * a.c.n_heads;
    const int part = at / heads, bh = at - part * heads, b = bh / a.c.n_heads, kh = bh - b * a.c.n_heads;
    // before the wait, past L1: lengths and tables; then all loads that depend on no other
    int len = __ldcg(a.lens + b);
    len = len < 0 ? 0 : len < a.max_len ? len : a.max_len;
    const int t0 = part * kFinishThreads * kFinishSlots + tid;
    if (t0 - tid >= len) {
        if (blockIdx.x == 0) griddep_wait();          // this kernel must not be complete before the streaming kernel is
        return;
    }
    SlotRef ref[kFinishSlots];
    float sum[kFinishSlots], had[kFinishSlots];
#pragma unroll
    for (int x = 0; x < kFinishSlots; ++x) {
        const int t = t0 + x * kFinishThreads;
        ref[x].page = -1, sum[x] = had[x] = 0.f;
        if (t < len) {
            int index;
            split_slot(a.c, t, &index, &ref[x].off);
            ref[x].page = __ldcg(a.table + (size_t)b * a.table_stride + index);
        }
    }
    griddep_wait();
    for (int tile = 0; tile < w.row_tiles; ++tile) {
        const int seg = b * w.tiles + kh * w.row_tiles + tile;
        const float *z = w.scores + ((size_t)seg * w.score_slots + t0) * w.score_rows;
        const size_t next = (size_t)kFinishThreads * w.score_rows;
        const int2 span = tid < rows ? w.span[seg] : make_int2(0, 0);
        float4 z0[kFinishSlots], z1[kFinishSlots];    // the first rows' scores, while lse comes
#pragma unroll
        for (int x = 0; x < kFinishSlots; ++x)
            if (t0 + x * kFinishThreads < len) {
                z0[x] = reinterpret_cast<const float4 *>(z + x * next)[0];
                if (w.score_rows > 4) z1[x] = reinterpret_cast<const float4 *>(z + x * next)[1];
            }
        if (tile == 0) {
#pragma unroll
            for (int x = 0; x < kFinishSlots; ++x) {
                if ((unsigned)ref[x].page >= (unsigned)a.c.n_pages) ref[x].page = -1;
                if (ref[x].page >= 0) had[x] = a.c.weight[slot_weight(a.c, ref[x], kh)];
            }
        }
        __syncthreads();
        float lse = -INFINITY;                        // of row tid, in log2 units
        if (tid < rows) {
            const RowRef r = row_ref(a, w, b, kh, tile * rows + tid);
            if (r.real) {
                if (span.y == 1) {
                    lse = a.lse[r.head] * 1.44269504088896340736f;
                } else {                              // its pieces' statistics: the join may not have run yet
                    auto stat = [&](int i) {
                        return w.part_ml[((size_t)(span.x + i) * 2 + (i == 0 ? 1 : 0)) * rows + tid];
                    };
                    float m = kNoRef, l = 0.f;
#pragma unroll 8
                    for (int i = 0; i < span.y; ++i) m = fmaxf(m, stat(i).x);
#pragma unroll 8
                    for (int i = 0; i < span.y; ++i) l += stat(i).y * ex2(stat(i).x - m);
                    lse = l == 0.f ? -INFINITY : m + log2f(l);
                }
            }
            s_lse[tid] = lse;
        }
        const bool odd = __syncthreads_or(lse != lse);
#pragma unroll
        for (int x = 0; x < kFinishSlots; ++x) {
            if (ref[x].page < 0) continue;
            auto add = [&](float y, int r) {
                if (s_lse[r] != -INFINITY) sum[x] += ex2(y - s_lse[r]);
            };
            if (__builtin_expect(odd, 0)) {
                // a row is NaN, and so would be its share of a slot that it does not see
                const int t = t0 + x * kFinishThreads;
#pragma unroll 1
                for (int r = 0; r < rows && tile * rows + r < R; ++r)
                    if (t < len - a.S + 1 + quotient(tile * rows + r, w.group_div)) add(z[x * next + r], r);
                continue;
            }
            add(z0[x].x, 0), add(z0[x].y, 1), add(z0[x].z, 2), add(z0[x].w, 3);
            if (w.score_rows > 4) add(z1[x].x, 4), add(z1[x].y, 5), add(z1[x].z, 6), add(z1[x].w, 7);
#pragma unroll 2
            for (int r = 8; r < rows && tile * rows + r < R; r += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(z + x * next + r);
                add(y.x, r), add(y.y, r + 1), add(y.z, r + 2), add(y.w, r + 3);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < kFinishSlots; ++x)
        if (ref[x].page >= 0) a.c.weight[slot_weight(a.c, ref[x], kh)] = had[x] + sum[x];
}

int page_steps(int page) { return page / 16 + (page % 16 != 0); }   // page + 15 may pass 2^31 - 1

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

AttnPlan plan_of(int type, int rows, int dim) {
    return type == kBf16 ? attn_plan<kBf16>(rows, dim)
           : type == kF16 ? attn_plan<kF16>(rows, dim) : attn_plan<kE4m3>(rows, dim);
}

// Sequences per launch: their lengths sit in shared memory, their cost units
// are counted in 31 bits, and the scores kept for the weights stay within 1 GiB
// where one sequence's do.
struct Layout {
    AttnPlan pl;
    int rows, row_tiles, seqs, score_slots, score_rows;
    int ctas, ranks;
    size_t part_o, part_ml, head_o, open, span, lse, scores, bytes;
};
Layout layout(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate) {
    Layout y;
    const int R = S * (n_q_heads / c.n_heads);
    y.pl = plan_of(c.type, R, c.dim);
    y.rows = y.pl.rows;
    y.row_tiles = (R + y.rows - 1) / y.rows;
    y.score_slots = max_len;
    // whole 16 bytes a slot: 32 query heads over 8 (9 sequences as above) 37.1 us, 39.9 with all 8 rows
    y.score_rows = y.row_tiles == 1 ? (R + 3) & ~3 : y.rows;
    const int count = (int)fmin(kAttnMaxSeq, kAttnMaxUnits / attn_units(c, max_len, S, n_q_heads));
    y.seqs = n_seq < count ? n_seq : count;
    // One block, or a cluster of two, four or eight, per segment, where all
    // run at once: the fewest blocks of at most kEnoughBytes of K and V each,
    // else the most of at most kWholeBytes (an SM streams that in less than the
    // second kernel takes).  Clusters of one-block SMs that run at once: 76 of
    // two, 36 of four, 15 of eight.  8 heads of 128 bf16, by blocks a segment:
    //   520 slots: 10.2 us with one, 10.3 with two, 9.7 with four; equal ranges 12.3
    //   1000: 13.2 with one, 11.2 with two, 9.7 with four; 12.7
    //   2000: 11.2 with four, 9.8 with eight; 12.6
    //   4000: 11.3 with eight; 14.2
    const long long segments = (long long)y.seqs * c.n_heads * y.row_tiles;
    const long long bytes = (long long)max_len * c.dim * (c.type == kE4m3 ? 1 : 2) * 2;
    const int sms = num_sms(), at_once[4] = {sms, sms / 2, sms * 36 / 152, sms * 15 / 152};
    y.ranks = 0;
    for (int k = 0; k < 4 && !y.ranks; ++k)
        if (segments <= at_once[k] && bytes <= kEnoughBytes << k) y.ranks = 1 << k;
    for (int k = 3; k >= 0 && !y.ranks; --k)
        if (segments <= at_once[k] && bytes <= kWholeBytes << k) y.ranks = 1 << k;
    y.ctas = y.ranks ? (int)segments * y.ranks : sms;
    const size_t ctas = y.ctas;
    const size_t tile_f = (size_t)y.rows * y.pl.dp * 4;
    const size_t seq_scores = (size_t)c.n_heads * y.row_tiles * y.score_slots * y.score_rows * 4;
    if (accumulate && seq_scores * y.seqs > kScoreBytes) {
        const size_t fit = kScoreBytes / seq_scores;
        y.seqs = fit < 1 ? 1 : (int)fit;
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += up256(n);
        return here;
    };
    y.part_o = take(y.ranks == 1 ? 0 : 2 * ctas * tile_f);
    y.part_ml = take(y.ranks == 1 ? 0 : 2 * ctas * y.rows * sizeof(float2));
    y.head_o = take(y.ranks ? 0 : ctas * y.pl.piece_rows * y.pl.dp * 4);
    y.open = take(y.ranks ? 0 : ctas * sizeof(int2));
    y.span = take(accumulate ? (size_t)segments * sizeof(int2) : 0);
    y.lse = take(accumulate ? (size_t)y.seqs * S * n_q_heads * 4 : 0);
    y.scores = take(accumulate ? seq_scores * y.seqs : 0);
    y.bytes = at;
    return y;
}

// Tensor map of the k or v pool: [page][head][slot][dim] in boxes of a step's
// slots by `box_bytes`, zeros where a box passes the end of a page or a row.
int cache_map(CUtensorMap *map, const KvView &c, const char *base, int box_bytes, int box_rows) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) QG_REFUSE(kECuda, "qattn_paged: cuTensorMapEncodeTiled is not available from the driver");
    const int esz = c.type == kE4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page, (cuuint64_t)c.n_heads, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_b, (cuuint64_t)c.head_b, (cuuint64_t)c.page_b};
    const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / esz), (cuuint32_t)box_rows, 1, 1}, steps[4] = {1, 1, 1, 1};
    const CUresult r = encode(
        map, c.type == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
             : c.type == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
        4, const_cast<char *>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
        box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) QG_REFUSE(kECuda, "qattn_paged: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return kOk;
}

}  // namespace

double attn_units(const KvView &c, int max_len, int S, int n_q_heads) {
    const int R = S * (n_q_heads / c.n_heads), rows = plan_of(c.type, R, c.dim).rows, full = max_len / c.page;
    const double steps = (double)full * page_steps(c.page) + (max_len - full * c.page + 15) / 16;
    return (double)c.n_heads * ((R + rows - 1) / rows) * (steps + kSegmentCost);
}

size_t ws_attn_paged(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate) {
    return layout(c, n_seq, max_len, S, n_q_heads, accumulate).bytes;
}

// Fewer sequences or a smaller max_len may take a plan that needs more: every
// part at its most over all of them, and over fewer new tokens.  No plan has
// more blocks than SMs.
size_t ws_attn_paged_most(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate) {
    const size_t ctas = num_sms(), seqs = n_seq < kAttnMaxSeq ? n_seq : kAttnMaxSeq;
    size_t most = 0;
    for (int s = 1; s <= S; ++s) {
        const Layout y = layout(c, n_seq, max_len, s, n_q_heads, accumulate);
        const size_t row = (size_t)y.pl.dp * 4, segments = (size_t)c.n_heads * y.row_tiles;
        size_t n = up256(2 * ctas * y.rows * row) + up256(2 * ctas * y.rows * sizeof(float2)) +
                   up256(ctas * y.pl.piece_rows * row) + up256(ctas * sizeof(int2));
        if (accumulate) {
            const size_t one = segments * y.score_slots * y.score_rows * 4;
            const size_t all = one > kScoreBytes ? one : one * seqs < kScoreBytes ? one * seqs : kScoreBytes;
            n += up256(seqs * segments * sizeof(int2)) + up256(seqs * s * n_q_heads * 4) + up256(all);
        }
        if (n > most) most = n;
    }
    return most;
}

int run_attn_paged(const AttnArgs &args, void *ws, cudaStream_t st) {
    const Layout y = layout(args.c, args.n_seq, args.max_len, args.S, args.n_q_heads, args.accumulate);
    char *base = static_cast<char *>(ws);
    AttnWork w;
    w.part_o = reinterpret_cast<float *>(base + y.part_o);
    w.part_ml = reinterpret_cast<float2 *>(base + y.part_ml);
    w.head_o = reinterpret_cast<float *>(base + y.head_o);
    w.open = reinterpret_cast<int2 *>(base + y.open);
    w.span = reinterpret_cast<int2 *>(base + y.span);
    w.scores = reinterpret_cast<float *>(base + y.scores);
    w.score_slots = y.score_slots;
    w.score_rows = y.score_rows;
    w.row_tiles = y.row_tiles;
    w.tiles = args.c.n_heads * y.row_tiles;
    w.ranks = y.ranks;
    w.tiles_div = fast_div(w.tiles);
    w.row_tiles_div = fast_div(w.row_tiles);
    w.group_div = fast_div(args.group);
    w.page_steps = page_steps(args.c.page);
    w.page_steps_div = fast_div(w.page_steps);
    w.box_rows = args.c.page < 16 ? args.c.page : 16;
    CUtensorMap maps[2];
    int rc = cache_map(&maps[0], args.c, args.c.k, y.pl.box_bytes, w.box_rows);
    if (rc == kOk) rc = cache_map(&maps[1], args.c, args.c.v, y.pl.box_bytes, w.box_rows);
    if (rc != kOk) return rc;
    for (int b0 = 0; b0 < args.n_seq; b0 += y.seqs) {
        AttnArgs a = args;
        a.n_seq = args.n_seq - b0 < y.seqs ? args.n_seq - b0 : y.seqs;
        const size_t rows = (size_t)b0 * a.S;
        a.table += (size_t)b0 * a.table_stride;
        a.lens += b0;
        a.q = static_cast<const uint16_t *>(a.q) + rows * a.q_stride;
        a.o = static_cast<char *>(a.o) + rows * a.n_q_heads * a.c.dim * (a.o_type == kF32 ? 4 : 2);
        if (a.lse) a.lse += rows * a.n_q_heads;
        else if (a.accumulate) a.lse = reinterpret_cast<float *>(base + y.lse);
        w.ctas = y.ranks ? a.n_seq * w.tiles * y.ranks : y.ctas;
        rc = a.c.type == kF16    ? launch_attn_stream<kF16, false>(a, w, maps, st)
             : a.c.type == kE4m3 ? (a.o_type == kBf16 ? launch_attn_stream<kE4m3, false>(a, w, maps, st)
                                                      : launch_attn_stream<kE4m3, true>(a, w, maps, st))
             : a.o_type != kBf16 ? launch_attn_stream<kBf16, true>(a, w, maps, st)
                                 : launch_attn_stream<kBf16, false>(a, w, maps, st);
        // a segment's pieces: few where there are many segments, and a block then does
        // several rows; else one, its threads sharing the pieces
        const int most = kFinishThreads / (y.pl.dp / 4), per = (long long)a.n_seq * w.tiles * 8 < w.ctas ? 1 : most < 8 ? most : 8;
        const int joins = y.ranks ? 0 : w.ctas * (y.rows / per);
        const long long adds = a.accumulate ? (long long)a.n_seq * a.c.n_heads *
                                                  ((a.max_len - 1) / (kFinishThreads * kFinishSlots) + 1)
                                            : 0;
        if (rc == kOk && joins + adds > 0)
            rc = launch_pdl("qattn_paged", attn_finish_kernel, dim3((unsigned)(joins + adds)), kFinishThreads,
                            0, st, a, w, y.rows, y.pl.dp, per, joins);
        if (rc != kOk) return rc;
    }
    return kOk;
}

}  // namespace qg
