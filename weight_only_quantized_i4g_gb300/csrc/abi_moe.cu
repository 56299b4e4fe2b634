// abi_moe.cu -- the extern "C" entry points of the expert layer (declared in
// include/qgemv.h): every argument the host can see is checked before any
// kernel is enqueued.
#include <limits.h>
#include <stdint.h>

#include "../../include/qgemv.h"
#include "moe.cuh"

using namespace qg;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool is_wide(int type) { return type == QG_F32 || type == QG_BF16 || type == QG_F16; }
size_t size_of(int type) { return type == QG_F32 ? 4 : type == QG_E4M3 ? 1 : 2; }

// Tokens, their slots and rows of `width` elements.
int check_slots(const char *fn, int n_tokens, int k, int width, int n_rows) {
    if (n_tokens < 0 || n_rows < 0)
        QG_REFUSE(kEInval, "%s: n_tokens = %d and n_rows = %d must be >= 0", fn, n_tokens, n_rows);
    if (width > INT_MAX - 65536) QG_REFUSE(kEInval, "%s: a row of %d elements overflows", fn, width);
    if (k < 1 || width < 1) QG_REFUSE(kEInval, "%s: k = %d and the row's width %d must be >= 1", fn, k, width);
    if ((long long)n_tokens * k > INT_MAX)
        QG_REFUSE(kEInval, "%s: n_tokens * k = %lld slots, must be below 2^31", fn, (long long)n_tokens * k);
    // a kernel's blocks are counted along one axis
    if ((long long)n_tokens * (((long long)width + 127) / 128) > INT_MAX)
        QG_REFUSE(kEInval, "%s: n_tokens * ceil(width / 128) must be below 2^31", fn);
    return kOk;
}

// Of the calls that move rows.
int check_places(const char *fn, const void *place, int n_tokens, int k, int n_rows) {
    if (k > INT_MAX - kTogether) QG_REFUSE(kEInval, "%s: k = %d slots a token overflow", fn, k);
    if (!place && (long long)n_tokens * k > n_rows)
        QG_REFUSE(kEInval, "%s: without place a row is a slot: n_rows = %d is below n_tokens * k = %lld", fn, n_rows,
                  (long long)n_tokens * k);
    return kOk;
}

int check_product(const char *fn, int fmt, const void *Y, int y_type, const void *X, const void *x_scales,
                  const void *w, const void *w_scales, int n_experts, int M, int I, int O, const void *ws) {
    if (fmt != QG_FMT_FP8B128 && fmt != QG_FMT_FP8UE8M0)
        QG_REFUSE(kEInval, "%s: format id %d is not QG_FMT_FP8B128 or QG_FMT_FP8UE8M0", fn, fmt);
    if (!is_wide(y_type)) QG_REFUSE(kEInval, "%s: y_type %d is not QG_F32, QG_BF16 or QG_F16", fn, y_type);
    if (M < 0 || I < 1 || O < 1) QG_REFUSE(kEInval, "%s: M = %d must be >= 0, I = %d and O = %d >= 1", fn, M, I, O);
    if (n_experts < 1 || n_experts > kMaxSortExperts)
        QG_REFUSE(kEInval, "%s: n_experts = %d, must be in [1, %d]", fn, n_experts, kMaxSortExperts);
    if (M > INT_MAX - 256 || I > INT_MAX - 256 || O > INT_MAX - 256) QG_REFUSE(kEInval, "%s: sizes overflow", fn);
    if ((M + 63) / 64 > 65535) QG_REFUSE(kEInval, "%s: M = %d rows, must be at most %d", fn, M, 65535 * 64);
    if (M == 0) return kOk;
    if (!Y || !X || !x_scales || !w || !w_scales)
        QG_REFUSE(kEInval, "%s: Y, X, x_scales, w and w_scales must be non-NULL", fn);
    if (!aligned(Y, size_of(y_type)) || !aligned(x_scales, 4) || (fmt == QG_FMT_FP8B128 && !aligned(w_scales, 4)))
        QG_REFUSE(kEAlign, "%s: Y must be aligned to its type, x_scales and f32 w_scales to 4 bytes", fn);
    if (ws && !aligned(ws, 256)) QG_REFUSE(kEAlign, "%s: workspace must be 256-byte aligned", fn);
    return kOk;
}

int product(const char *fn, int fmt, void *Y, int y_type, const uint8_t *X, const float *x_scales, const uint8_t *w,
            const void *w_scales, const int *offsets, int n_experts, int M, int I, int O, const void *ws,
            qg_stream_t stream) {
    const int rc = check_product(fn, fmt, Y, y_type, X, x_scales, w, w_scales, n_experts, M, I, O, ws);
    if (rc || M == 0) return rc;
    cudaGetLastError();
    E4m3Args a{};
    a.Y = Y;
    a.y_type = y_type;
    a.X = X;
    a.x_scale = x_scales;
    a.w = w;
    a.w_scale = w_scales;
    a.w_power = fmt == QG_FMT_FP8UE8M0;
    a.offsets = offsets;
    a.experts = n_experts;
    a.M = M;
    a.I = I;
    a.O = O;
    a.err = device_error_word();
    return run_gemm_e4m3(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t qg_moe_sort_workspace_bytes(int n_tokens, int k, int n_experts) {
    if (n_tokens < 1 || k < 1 || (long long)n_tokens * k > INT_MAX || n_experts < 1 || n_experts > kMaxSortExperts)
        return 0;
    return ws_moe_sort(n_tokens * k, n_experts);
}

int qg_moe_sort(int *offsets, int *order, int *place, const int *ids, int n_tokens, int k, int n_experts, void *ws,
                size_t ws_bytes, qg_stream_t stream) {
    const char *fn = "qg_moe_sort";
    int rc = check_slots(fn, n_tokens, k, 1, 0);
    if (rc) return rc;
    if (n_experts < 1 || n_experts > kMaxSortExperts)
        QG_REFUSE(kEInval, "%s: n_experts = %d, must be in [1, %d]", fn, n_experts, kMaxSortExperts);
    if (!offsets) QG_REFUSE(kEInval, "%s: offsets must be non-NULL", fn);
    if (n_tokens > 0 && (!place || !ids)) QG_REFUSE(kEInval, "%s: place and ids must be non-NULL", fn);
    if (!aligned(offsets, 4) || !aligned(order, 4) || !aligned(place, 4) || !aligned(ids, 4))
        QG_REFUSE(kEAlign, "%s: offsets, order, place and ids must be 4-byte aligned", fn);
    const size_t need = qg_moe_sort_workspace_bytes(n_tokens, k, n_experts);
    if (need > 0 && (ws == nullptr || ws_bytes < need))
        QG_REFUSE(kEWorkspace, "%s: needs a workspace of %zu bytes (qg_moe_sort_workspace_bytes; got %zu)", fn, need,
                  ws == nullptr ? (size_t)0 : ws_bytes);
    if (ws && !aligned(ws, 256)) QG_REFUSE(kEAlign, "%s: workspace must be 256-byte aligned", fn);
    cudaGetLastError();
    const SortArgs a{offsets, order, place, ids, n_tokens * k, n_experts, 0};
    return run_moe_sort(a, ws, reinterpret_cast<cudaStream_t>(stream));
}

int qg_moe_dispatch(void *rows, int rows_type, float *row_scales, const void *x, int x_type, size_t x_stride,
                    const int *place, int n_tokens, int k, int I, int n_rows, qg_stream_t stream) {
    const char *fn = "qg_moe_dispatch";
    int rc = check_slots(fn, n_tokens, k, I, n_rows);
    if (rc) return rc;
    if (!is_wide(x_type)) QG_REFUSE(kEInval, "%s: x_type %d is not QG_F32, QG_BF16 or QG_F16", fn, x_type);
    const bool codes = rows_type == QG_E4M3;
    if (!codes && rows_type != x_type)
        QG_REFUSE(kEInval, "%s: rows_type %d must be x_type %d or QG_E4M3", fn, rows_type, x_type);
    if ((rc = check_places(fn, place, n_tokens, k, n_rows))) return rc;
    if (n_tokens > 1 && x_stride < (size_t)I)
        QG_REFUSE(kEInval, "%s: x_stride = %zu is below I = %d", fn, x_stride, I);
    if (x_stride > (size_t)1 << 40) QG_REFUSE(kEInval, "%s: x_stride = %zu overflows", fn, x_stride);
    if (n_tokens == 0 || n_rows == 0) return kOk;
    if (!rows || !x || (codes && !row_scales))
        QG_REFUSE(kEInval, "%s: rows, x and (e4m3 rows) row_scales must be non-NULL", fn);
    if (!aligned(rows, size_of(rows_type)) || !aligned(x, size_of(x_type)) || !aligned(place, 4) ||
        !aligned(row_scales, 4))
        QG_REFUSE(kEAlign, "%s: rows and x must be aligned to their types, place and row_scales to 4 bytes", fn);
    cudaGetLastError();
    const DispatchArgs a{rows, row_scales, x, x_stride, place, n_tokens, k, I, n_rows};
    return run_moe_dispatch(a, x_type, codes, reinterpret_cast<cudaStream_t>(stream));
}

int qg_moe_combine(void *out, int out_type, const void *y, int y_type, const float *weights, const int *place,
                   int n_tokens, int k, int O, int n_rows, qg_stream_t stream) {
    const char *fn = "qg_moe_combine";
    int rc = check_slots(fn, n_tokens, k, O, n_rows);
    if (rc) return rc;
    if (!is_wide(out_type) || !is_wide(y_type))
        QG_REFUSE(kEInval, "%s: out_type %d and y_type %d must be QG_F32, QG_BF16 or QG_F16", fn, out_type, y_type);
    if ((rc = check_places(fn, place, n_tokens, k, n_rows))) return rc;
    if (n_tokens == 0) return kOk;
    if (!out || (n_rows > 0 && !y)) QG_REFUSE(kEInval, "%s: out and y must be non-NULL", fn);
    if (!aligned(out, size_of(out_type)) || !aligned(y, size_of(y_type)) || !aligned(weights, 4) || !aligned(place, 4))
        QG_REFUSE(kEAlign, "%s: out and y must be aligned to their types, weights and place to 4 bytes", fn);
    cudaGetLastError();
    const CombineArgs a{out, y, weights, place, n_tokens, k, O, n_rows};
    return run_moe_combine(a, out_type, y_type, reinterpret_cast<cudaStream_t>(stream));
}

int qg_moe_combine_grad(void *dy, float *dweights, const void *dout, int dout_type, const void *y, int y_type,
                        const float *weights, const int *place, int n_tokens, int k, int O, int n_rows,
                        qg_stream_t stream) {
    const char *fn = "qg_moe_combine_grad";
    int rc = check_slots(fn, n_tokens, k, O, n_rows);
    if (rc) return rc;
    if (!is_wide(dout_type) || !is_wide(y_type))
        QG_REFUSE(kEInval, "%s: dout_type %d and y_type %d must be QG_F32, QG_BF16 or QG_F16", fn, dout_type, y_type);
    if ((rc = check_places(fn, place, n_tokens, k, n_rows))) return rc;
    if (n_tokens == 0) return kOk;
    if (!dy && !dweights) QG_REFUSE(kEInval, "%s: dy and dweights are both NULL", fn);
    if (!dout || (dweights && n_rows > 0 && !y))
        QG_REFUSE(kEInval, "%s: dout and (with dweights) y must be non-NULL", fn);
    if (!aligned(dy, size_of(y_type)) || !aligned(y, size_of(y_type)) || !aligned(dout, size_of(dout_type)) ||
        !aligned(dweights, 4) || !aligned(weights, 4) || !aligned(place, 4))
        QG_REFUSE(kEAlign, "%s: dy, y and dout must be aligned to their types, the rest to 4 bytes", fn);
    cudaGetLastError();
    const CombineGradArgs a{dy, dweights, dout, y, weights, place, n_tokens, k, O, n_rows};
    return run_moe_combine_grad(a, dout_type, y_type, reinterpret_cast<cudaStream_t>(stream));
}

size_t qgemm_e4m3_workspace_bytes(int, int, int, int) { return 0; }   // a split K is added up over clusters

int qgemm_e4m3(int fmt, void *Y, int y_type, const uint8_t *X, const float *x_scales, const uint8_t *w,
               const void *w_scales, int M, int I, int O, void *ws, size_t, qg_stream_t stream) {
    return product("qgemm_e4m3", fmt, Y, y_type, X, x_scales, w, w_scales, nullptr, 1, M, I, O, ws, stream);
}

int qgemm_e4m3_moe(int fmt, void *Y, int y_type, const uint8_t *X, const float *x_scales, const uint8_t *w,
                   const void *w_scales, const int *offsets, int n_experts, int M, int I, int O, void *ws, size_t,
                   qg_stream_t stream) {
    const char *fn = "qgemm_e4m3_moe";
    if (!offsets) QG_REFUSE(kEInval, "%s: offsets must be non-NULL", fn);
    if (!aligned(offsets, 4)) QG_REFUSE(kEAlign, "%s: offsets must be 4-byte aligned", fn);
    return product(fn, fmt, Y, y_type, X, x_scales, w, w_scales, offsets, n_experts, M, I, O, ws, stream);
}

}  // extern "C"
