// attn_paged.cu -- attention over a paged cache: workspace, launches, the join
// of segments that several blocks share, and the accumulation of attention
// weights.  The streaming kernel is in attn_paged.cuh.
#include "attn_launch.cuh"

namespace qg {

extern template int launch_attn_stream<kBf16>(const AttnArgs &, const AttnWork &, const AttnPlan &, cudaStream_t);
extern template int launch_attn_stream<kF16>(const AttnArgs &, const AttnWork &, const AttnPlan &, cudaStream_t);
extern template int launch_attn_stream<kE4m3>(const AttnArgs &, const AttnWork &, const AttnPlan &, cudaStream_t);
extern template AttnPlan attn_plan<kBf16>(int, int);
extern template AttnPlan attn_plan<kF16>(int, int);
extern template AttnPlan attn_plan<kE4m3>(int, int);

namespace {

constexpr int kJoinThreads = 256;

// Joins the pieces of the segment that block x of the streaming kernel left
// open at its end: that block's last piece, then the first pieces of the
// blocks after it.  Block (x, y) does rows 8y .. 8y + 7.
template <int TYPE>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs a,
                                                                 const __grid_constant__ AttnWork w, int rows,
                                                                 int dp) {
    extern __shared__ float2 s_ml[];                  // [pieces][8]: factor, sum
    __shared__ float s_l[8];
    griddep_launch_dependents();
    griddep_wait();
    const int2 open = w.tail[blockIdx.x];
    const int seg = open.x, pieces = open.y, r0 = 8 * blockIdx.y;
    if (seg < 0) return;
    const int tiles = a.c.n_heads * w.row_tiles;
    const int b = seg / tiles, sg = seg - b * tiles, kh = sg / w.row_tiles, tile = sg - kh * w.row_tiles;
    if (tile * rows + r0 >= a.S * a.group) return;
    auto base = [&](int i) { return ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * rows + r0; };
    for (int i = threadIdx.x; i < 8 * pieces; i += kJoinThreads) s_ml[i] = w.part_ml[base(i >> 3) + (i & 7)];
    __syncthreads();
    // one warp a row: largest maximum, then factors and the sum
    const int r = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool real = tile * rows + r0 + r < a.S * a.group;
    float m = kNoRef, l = 0.f;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, s_ml[8 * i + r].x);
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    for (int i = lane; i < pieces; i += 32) {
        const float2 x = s_ml[8 * i + r];
        const float f = ex2(x.x - m);
        s_ml[8 * i + r].x = f;
        l += x.y * f;
    }
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    if (lane == 0) {
        s_l[r] = l;
        if (real && a.lse) a.lse[row_ref(a, b, kh, tile * rows + r0 + r).head] = row_lse(m, l);
    }
    __syncthreads();
    const float vs = TYPE == kE4m3 ? __ldg(a.c.v_scale + kh) : 1.f;
    for (int i = threadIdx.x; i < 8 * (dp / 4); i += kJoinThreads) {
        const int row = i / (dp / 4), d = 4 * (i - row * (dp / 4));
        const RowRef ref = row_ref(a, b, kh, tile * rows + r0 + row);
        if (!ref.real || d >= a.c.dim) continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int x = 0; x < pieces; ++x) {
            const float f = s_ml[8 * x + row].x;
            const float4 v = *reinterpret_cast<const float4 *>(w.part_o + (base(x) + row) * dp + d);
            sum.x += v.x * f, sum.y += v.y * f, sum.z += v.z * f, sum.w += v.w * f;
        }
        store_out4(a, ref.head * a.c.dim + d, sum, row_factor(s_l[row], vs));
    }
}

// weight[t] += sum over the rows of a key-value head of exp(z_t - lse), from
// the scores that the streaming kernel left; a thread a slot.
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) attn_weight_kernel(const __grid_constant__ AttnArgs a,
                                                                     const __grid_constant__ AttnWork w, int rows) {
    __shared__ float s_lse[64];
    griddep_launch_dependents();
    griddep_wait();
    const int kh = blockIdx.x % a.c.n_heads, b = blockIdx.x / a.c.n_heads;
    const int len = seq_len(a.lens, b, a.max_len, nullptr);
    if ((int)blockIdx.y * kWeightThreads >= len) return;
    const int t = blockIdx.y * kWeightThreads + threadIdx.x, R = a.S * a.group;
    SlotRef ref{-1, 0};
    if (t < len) ref = find_slot(a.c, a.table + (size_t)b * a.table_stride, t);
    float sum = 0.f;
    for (int tile = 0; tile < w.row_tiles; ++tile) {
        __syncthreads();
        if (threadIdx.x < rows) {
            const RowRef r = row_ref(a, b, kh, tile * rows + threadIdx.x);
            s_lse[threadIdx.x] = r.real ? a.lse[r.head] * 1.44269504088896340736f : -INFINITY;
        }
        __syncthreads();
        if (ref.page < 0) continue;
        const size_t seg = ((size_t)b * a.c.n_heads + kh) * w.row_tiles + tile;
        const float *z = w.scores + (seg * w.score_slots + t) * rows;
        for (int r = 0; r < rows && tile * rows + r < R; r += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(z + r);
            if (s_lse[r] != -INFINITY) sum += ex2(x.x - s_lse[r]);
            if (s_lse[r + 1] != -INFINITY) sum += ex2(x.y - s_lse[r + 1]);
        }
    }
    if (ref.page >= 0) a.c.weight[slot_weight(a.c, ref, kh)] += sum;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

AttnPlan plan_of(int type, int rows, int dim) {
    return type == kBf16 ? attn_plan<kBf16>(rows, dim)
           : type == kF16 ? attn_plan<kF16>(rows, dim) : attn_plan<kE4m3>(rows, dim);
}

// Sequences per launch: their lengths sit in shared memory, and the scores
// kept for the weights stay within 1 GiB where one sequence's do.
struct Layout {
    AttnPlan pl;
    int rows, row_tiles, seqs, score_slots;
    size_t part_o, part_ml, head_o, tail, lse, scores, bytes;
};
Layout layout(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate) {
    Layout y;
    const int R = S * (n_q_heads / c.n_heads), ctas = num_sms();
    y.pl = plan_of(c.type, R, c.dim);
    y.rows = 8 * y.pl.nt;
    y.row_tiles = (R + y.rows - 1) / y.rows;
    y.score_slots = (max_len + 15) / 16 * 16;
    y.seqs = n_seq < kAttnMaxSeq ? n_seq : kAttnMaxSeq;
    const size_t tile_f = (size_t)y.rows * y.pl.dp * 4;
    const size_t seq_scores = (size_t)c.n_heads * y.row_tiles * y.score_slots * y.rows * 4;
    if (accumulate && seq_scores * y.seqs > ((size_t)1 << 30)) {
        const size_t fit = ((size_t)1 << 30) / seq_scores;
        y.seqs = fit < 1 ? 1 : (int)fit;
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += up256(n);
        return here;
    };
    y.part_o = take(2 * ctas * tile_f);
    y.part_ml = take((size_t)2 * ctas * y.rows * sizeof(float2));
    y.head_o = take((size_t)ctas * y.pl.warps * tile_f);
    y.tail = take((size_t)ctas * sizeof(int2));
    y.lse = take(accumulate ? (size_t)y.seqs * S * n_q_heads * 4 : 0);
    y.scores = take(accumulate ? seq_scores * y.seqs : 0);
    y.bytes = at;
    return y;
}

template <int TYPE>
int run(const AttnArgs &a, const AttnWork &w, const Layout &y, cudaStream_t st) {
    int rc = launch_attn_stream<TYPE>(a, w, y.pl, st);
    if (rc != kOk) return rc;
    const int ctas = num_sms();
    return launch_pdl("qattn_paged", attn_join_kernel<TYPE>, dim3(ctas, y.pl.nt), kJoinThreads,
                      (size_t)8 * ctas * sizeof(float2), st, a, w, y.rows, y.pl.dp);
}

}  // namespace

size_t ws_attn_paged(const KvView &c, int n_seq, int max_len, int S, int n_q_heads, int accumulate) {
    return layout(c, n_seq, max_len, S, n_q_heads, accumulate).bytes;
}

int run_attn_paged(const AttnArgs &args, void *ws, cudaStream_t st) {
    const Layout y = layout(args.c, args.n_seq, args.max_len, args.S, args.n_q_heads, args.accumulate);
    char *base = static_cast<char *>(ws);
    AttnWork w;
    w.part_o = reinterpret_cast<float *>(base + y.part_o);
    w.part_ml = reinterpret_cast<float2 *>(base + y.part_ml);
    w.head_o = reinterpret_cast<float *>(base + y.head_o);
    w.tail = reinterpret_cast<int2 *>(base + y.tail);
    w.scores = reinterpret_cast<float *>(base + y.scores);
    w.score_slots = y.score_slots;
    w.row_tiles = y.row_tiles;
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
        int rc = a.c.type == kBf16 ? run<kBf16>(a, w, y, st)
                 : a.c.type == kF16 ? run<kF16>(a, w, y, st) : run<kE4m3>(a, w, y, st);
        if (rc == kOk && a.accumulate && a.max_len > 0)
            rc = launch_pdl("qattn_paged", attn_weight_kernel,
                            dim3(a.n_seq * a.c.n_heads, (a.max_len + kWeightThreads - 1) / kWeightThreads),
                            kWeightThreads, 0, st, a, w, y.rows);
        if (rc != kOk) return rc;
    }
    return kOk;
}

}  // namespace qg
