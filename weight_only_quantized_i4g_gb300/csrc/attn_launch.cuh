// attn_launch.cuh -- which instantiation of the attention kernel a call takes,
// and its launch.
#pragma once

#include "attn_paged.cuh"

namespace qg {

struct AttnPlan {
    int dp, rows;       // padded head size, rows of a segment
    int box_bytes;      // bytes of a row that one copy moves
    size_t piece_rows;  // rows of O that all warps of a block hold, at most
};

// The smallest padded head size (the padding is not read from memory); then as
// many tiles of 8 rows a warp as its registers take (two, or four at 64
// dimensions, one at 256: four at 128 spill), and groups of two or four warps
// for more rows (64 dimensions: 32 rows of 16 f16 sequences to 4099 slots, four
// new tokens, 26.9 us with two warps of two tiles, 33.9 with one of four, though
// 48 to 8190 take 147 and 136; 64 rows of 48 bf16 sequences 256 us with two of
// four, 251 with four of two, of e4m3 264 and 295).  More than a group's rows are
// further segments.  48 ragged bf16 sequences, 128 dimensions, 8 cache heads, 12,
// 32 and 64 rows: 139, 222 and 420 us (before Q moved to shared memory 264 and 507
// with groups, 272 and 543 with segments of 16 rows, 321 and 632 with four tiles a
// warp).
template <int TYPE, bool FINE, class Fn>
auto attn_dispatch(int rows, int dim, Fn fn) {
    if (dim <= 64)
        return rows <= 8    ? fn(AttnCfg<TYPE, 64, 1, 1, FINE>())
               : rows <= 16 ? fn(AttnCfg<TYPE, 64, 2, 1, FINE>())
               : rows <= 32 ? fn(AttnCfg<TYPE, 64, 2, 2, FINE>()) : fn(AttnCfg<TYPE, 64, 4, 2, FINE>());
    if (dim <= 128)
        return rows <= 8    ? fn(AttnCfg<TYPE, 128, 1, 1, FINE>())
               : rows <= 16 ? fn(AttnCfg<TYPE, 128, 2, 1, FINE>())
               : rows <= 32 ? fn(AttnCfg<TYPE, 128, 2, 2, FINE>()) : fn(AttnCfg<TYPE, 128, 2, 4, FINE>());
    return rows <= 8    ? fn(AttnCfg<TYPE, 256, 1, 1, FINE>())
           : rows <= 16 ? fn(AttnCfg<TYPE, 256, 1, 2, FINE>()) : fn(AttnCfg<TYPE, 256, 1, 4, FINE>());
}

// The same for both forms of FINE, but for the warps of a block.
template <int TYPE>
AttnPlan attn_plan(int rows, int dim) {
    return attn_dispatch<TYPE, false>(rows, dim, [](auto cfg) {
        using C = decltype(cfg);
        return AttnPlan{C::DP, C::rows, C::BB, (size_t)(C::GW > 1 ? 16 : C::W) * C::warp_rows};
    });
}

template <int TYPE, bool FINE>
int launch_attn_stream(const AttnArgs &a, const AttnWork &w, const CUtensorMap (&maps)[2], cudaStream_t st) {
    return attn_dispatch<TYPE, FINE>(a.S * a.group, a.c.dim, [&](auto cfg) {
        using C = decltype(cfg);
        static_assert(C::W <= 16, "the plan's piece_rows");
        const size_t smem = attn_fixed_smem<C>() + (2 * (size_t)a.n_seq + 1) * sizeof(int);
        auto *kernel = attn_stream_kernel<TYPE, C::DP, C::NT, C::GW, FINE, true>;
        if constexpr (C::GW == 1)
            if (a.S == 1) kernel = attn_stream_kernel<TYPE, C::DP, C::NT, C::GW, FINE, false>;
        set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), 232448);
        return launch_clusters("qattn_paged", kernel, dim3(w.ctas), dim3(C::threads), w.ranks > 1 ? w.ranks : 1, smem, st, a, w,
                               maps[0], maps[1]);
    });
}

}  // namespace qg
