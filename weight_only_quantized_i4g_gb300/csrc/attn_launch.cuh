// attn_launch.cuh -- which instantiation of the attention kernel a call takes,
// and its launch.
#pragma once

#include "attn_paged.cuh"

namespace qg {

struct AttnPlan {
    int dp, nt;         // padded head size, tiles of 8 rows per segment
    int warps;
    int box_bytes;      // bytes of a row that one copy moves
    size_t smem;        // without the lengths
};

// The smallest padded head size (the padding is not read from memory), and
// one, two or (64 dimensions) four tiles of 8 rows a warp.  More rows make
// several segments that read K and V each: at 128 dimensions four tiles spill
// (48 bf16 sequences, 32 rows: 321 us against 272 with two segments of two
// tiles; 64 rows: 632 against 543; e4m3, 32 rows: 367 against 263).
template <int TYPE, class Fn>
auto attn_dispatch(int rows, int dim, Fn fn) {
    const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    if (dim <= 64)
        return nt == 1 ? fn(AttnCfg<TYPE, 64, 1>()) : nt == 2 ? fn(AttnCfg<TYPE, 64, 2>()) : fn(AttnCfg<TYPE, 64, 4>());
    if (dim <= 128) return nt == 1 ? fn(AttnCfg<TYPE, 128, 1>()) : fn(AttnCfg<TYPE, 128, 2>());
    return nt == 1 ? fn(AttnCfg<TYPE, 256, 1>()) : fn(AttnCfg<TYPE, 256, 2>());
}

template <int TYPE>
AttnPlan attn_plan(int rows, int dim) {
    return attn_dispatch<TYPE>(rows, dim, [](auto cfg) {
        using C = decltype(cfg);
        return AttnPlan{C::DP, C::NT, C::W, C::BB, attn_fixed_smem<C>()};
    });
}

template <int TYPE>
int launch_attn_stream(const AttnArgs &a, const AttnWork &w, const AttnPlan &pl, const CUtensorMap (&maps)[2],
                       cudaStream_t st) {
    return attn_dispatch<TYPE>(a.S * a.group, a.c.dim, [&](auto cfg) {
        using C = decltype(cfg);
        const size_t smem = pl.smem + (2 * (size_t)a.n_seq + 1) * sizeof(int);
        auto *kernel = attn_stream_kernel<TYPE, C::DP, C::NT>;
        set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), 232448);
        return launch_pdl("qattn_paged", kernel, dim3(w.ctas), dim3(C::threads), smem, st, a, w, maps[0], maps[1]);
    });
}

}  // namespace qg
