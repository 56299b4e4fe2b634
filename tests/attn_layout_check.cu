// attn_layout_check.cu -- the attention kernels' index arithmetic on the CPU
// (host code only, from the kernels' own headers): division by multiplication,
// where the copies' swizzle puts a step's chunks and which banks the fragment
// reads touch, shared memory, and how steps are shared out over blocks and
// groups of warps.  Prints "ok" or what is wrong.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "attn_launch.cuh"

using namespace qg;

static int bad = 0;
#define CHECK(c, ...)                                       \
    do {                                                    \
        if (!(c) && bad++ < 20) printf(__VA_ARGS__), printf("\n"); \
    } while (0)

static void divisions() {
    std::vector<int> ds;
    for (int d = 1; d < 5000; ++d) ds.push_back(d);
    for (int k = 12; k < 31; ++k)
        for (int e = -1; e <= 1; ++e) ds.push_back((1 << k) + e);
    ds.push_back(0x7FFFFFFF);
    for (int d : ds) {
        const FastDiv f = fast_div(d);
        unsigned x = 12345u;
        for (int i = 0; i < 200; ++i) {
            x = x * 1664525u + 1013904223u;
            const long long m = (long long)((x >> 1) / (unsigned)d) * d;
            for (long long y : {(long long)(x >> 1), m - 1, m, m + d - 1, m + d, 0x7FFFFFFFLL, 0LL})
                if (y >= 0 && y <= 0x7FFFFFFFLL) CHECK(quotient((int)y, f) == y / d, "division %lld / %d", y, d);
        }
    }
}

// A read of `size` bytes by 32 lanes goes in phases of 128 bytes; every phase
// must touch each bank at most once.
static int conflicts(const std::vector<int> &at, int size) {
    int worst = 1;
    const int lanes = 128 / size;
    for (int p = 0; p < 32; p += lanes) {
        int bank[32] = {};
        std::set<int> seen;
        for (int l = p; l < p + lanes; ++l)
            if (seen.insert(at[l]).second)
                for (int b = 0; b < size; b += 4) ++bank[(at[l] + b) / 4 % 32];
        for (int b : bank) worst = b > worst ? b : worst;
    }
    return worst;
}

template <int TYPE, int DP, int NT, int GW, bool THIRD>
static void layout() {
    using C = AttnCfg<TYPE, DP, NT, GW, THIRD>;
    const char *what = "layout";
    printf("type %d dp %d nt %d gw %d: W %d G %d NS %d stage %d smem %zu\n", TYPE, DP, NT, GW, C::W, C::G, C::NS, C::stage,
           attn_fixed_smem<C>());
    CHECK(attn_fixed_smem<C>() + (2 * kAttnMaxSeq + 1) * 4 <= 232448, "%s: shared memory", what);
    CHECK(C::NS >= 1 && C::stage == 32 * DP * C::ESZ && C::stage % 1024 == 0, "%s: stage", what);
    CHECK(C::stage >= 32 * DP || GW > 1, "%s: a slab fits the stage", what);
    // every chunk of 16 slots has a place of its own, as the hardware swizzle has it
    std::set<int> places;
    const int chunks = DP * C::ESZ / 16, per = C::BB / 16;
    for (int row = 0; row < 16; ++row)
        for (int x = 0; x < chunks; ++x) {
            const int at = chunk_place<C>(row, x), box = x / per;
            places.insert(at);
            const int linear = box * C::box + row * C::BB + x % per * 16;
            const int swz = C::BB == 128 ? linear ^ ((linear >> 7 & 7) << 4) : linear ^ ((linear >> 7 & 3) << 4);
            CHECK(at == swz && at % 16 == 0 && at < 16 * DP * C::ESZ, "%s: place of %d, %d", what, row, x);
        }
    CHECK((int)places.size() == 16 * chunks, "%s: places collide", what);
    // K: 4 threads a slot hold each chunk once; V: 8 threads
    std::set<int> k;
    for (int i = 0; i < C::NI; ++i)
        for (int c = 0; c < 4; ++c) k.insert(k_chunk<C>(i, c));
    CHECK((int)k.size() == chunks && *k.rbegin() == chunks - 1, "%s: K chunks", what);
    for (int i = 0; i < C::NI; ++i)
        for (int half = 0; half < 2; ++half) {
            std::vector<int> at;
            for (int l = 0; l < 32; ++l) at.push_back(chunk_place<C>((l >> 2) + 8 * half, k_chunk<C>(i, l & 3)));
            CHECK(conflicts(at, 16) == 1, "%s: K read %d", what, i);
        }
    for (int q = 0; q < C::NQ; ++q)
        for (int j = 0; j < 4; ++j) {
            std::vector<int> at;
            for (int l = 0; l < 32; ++l) {
                const int g = l >> 2, row = 2 * (l & 3) + (j & 1) + 8 * (j >> 1);
                at.push_back(C::VB == 16 ? chunk_place<C>(row, 8 * q + g) : chunk_place<C>(row, g >> 1) + 8 * (g & 1));
            }
            CHECK(conflicts(at, C::VB) <= (C::VB == 16 ? 1 : 2), "%s: V read %d", what, q);
        }
    std::set<int> slab;
    for (int r = 0; r < 8; ++r)
        for (int x = 0; x < DP / 4; ++x) slab.insert(slab_place<C>(r, x));
    CHECK((int)slab.size() == 2 * DP && *slab.rbegin() == 2 * DP - 1, "%s: slab", what);
    for (int e = 0; e < 2; ++e)
        for (int x = 0; x < C::E; x += 4) {
            std::vector<int> at;
            for (int l = 0; l < 32; ++l) at.push_back(16 * slab_place<C>(2 * (l & 3) + e, ((l >> 2) * C::E + x) / 4));
            CHECK(conflicts(at, 16) <= 2, "%s: slab store", what);
        }
}

template <int TYPE, bool THIRD>
static void layouts() {
    std::set<int> done;
    for (int dim : {64, 128, 256})
        for (int rows : {1, 9, 17, 33}) {
            attn_dispatch<TYPE, THIRD>(rows, dim, [&](auto cfg) {
                using C = decltype(cfg);
                if (done.insert(C::DP * 100 + C::NT * 10 + C::GW).second) layout<TYPE, C::DP, C::NT, C::GW, THIRD>();
                CHECK(C::rows >= (rows < 33 ? rows : 32), "rows %d at %d", rows, dim);
                return 0;
            });
        }
}

// Shares out the steps of sequences of the given lengths as the kernels do and
// checks that every step is done once, in order, by one group, and that the
// spans of shared segments are what the second kernel is told.
static void share(const std::vector<int> &lens, int tiles, int page, int ctas, int groups) {
    KvView c = {};
    c.page = page;
    c.page_div = fast_div(page);
    AttnWork w = {};
    w.tiles = tiles;
    w.tiles_div = fast_div(tiles);
    w.page_steps = (page + 15) / 16;
    w.page_steps_div = fast_div(w.page_steps);
    const int n = (int)lens.size();
    std::vector<int> prefix(n + 1, 0), steps(n);
    for (int b = 0; b < n; ++b) {
        steps[b] = seq_steps(c, w, lens[b]);
        int slots = 0;      // slots of the steps of a sequence, page by page
        for (int i = 0; i < steps[b]; ++i) {
            const int pg = i / w.page_steps, slot = 16 * (i % w.page_steps), before = pg * page;
            int count = (lens[b] - before < page ? lens[b] - before : page) - slot;
            count = count > 16 ? 16 : count;
            CHECK(count >= 1, "empty step %d of %d slots, page %d", i, lens[b], page);
            slots += count;
        }
        CHECK(slots == lens[b], "%d slots in steps of %d, page %d", slots, lens[b], page);
        prefix[b + 1] = prefix[b] + (lens[b] > 0 ? steps[b] + kSegmentCost : 0);
    }
    const int total = prefix[n] * tiles, chunk = units_per_block(total, ctas, groups);
    std::vector<std::vector<int>> first(n * tiles, std::vector<int>()), last(n * tiles, std::vector<int>());
    std::vector<int> next(n * tiles, 0), from(n * tiles, -1), to(n * tiles, -1);
    Place at = locate(0, prefix.data(), n, w);
    for (int x = 0; x < ctas; ++x) {
        const int c0 = x * chunk < total ? x * chunk : total, c1 = c0 + chunk < total ? c0 + chunk : total;
        if (c0 >= c1) continue;
        for (int g = 0; g < groups; ++g) {
            Place p = locate(part_of(c0, c1, g, groups), prefix.data(), n, w);
            const Place e = locate(part_of(c0, c1, g + 1, groups), prefix.data(), n, w);
            for (int left = steps_between(p, e, prefix.data(), tiles); left > 0; --left) {
                CHECK(p.b == at.b && p.seg == at.seg && p.i == at.i, "out of order at block %d", x);
                CHECK(p.b < n && p.n == steps[p.b] && p.page == p.i / w.page_steps && p.sub == p.i % w.page_steps,
                      "place at block %d", x);
                if (p.b >= n) return;
                const int s = p.b * tiles + p.seg;
                CHECK(next[s] == p.i, "segment %d: step %d after %d", s, p.i, next[s]);
                ++next[s];
                if (from[s] < 0) from[s] = x;
                to[s] = x;
                advance(p, prefix.data(), n, w);
                advance(at, prefix.data(), n, w);
            }
            CHECK(p.b == e.b && p.seg == e.seg && p.i == e.i, "range of block %d ends elsewhere", x);
        }
    }
    for (int b = 0; b < n; ++b)
        for (int sg = 0; sg < tiles; ++sg) {
            const int s = b * tiles + sg;
            CHECK(next[s] == steps[b], "segment %d: %d steps of %d", s, next[s], steps[b]);
            if (steps[b])
                CHECK(blocks_spanned(b, sg, from[s], chunk, prefix.data(), tiles) == to[s] - from[s] + 1, "span of segment %d", s);
        }
}

int main() {
    divisions();
    layouts<kBf16, false>();
    layouts<kBf16, true>();
    layouts<kF16, false>();
    layouts<kE4m3, false>();
    layouts<kE4m3, true>();
    unsigned x = 7u;
    auto rnd = [&](int m) {
        x = x * 1664525u + 1013904223u;
        return (int)((unsigned long long)(x >> 8) * m >> 24);
    };
    for (int it = 0; it < 3000; ++it) {
        const int n = 1 + rnd(it % 7 == 0 ? 300 : 12), most = 1 << (1 + rnd(14));
        std::vector<int> lens(n);
        for (int &v : lens) v = rnd(4) ? rnd(most) : rnd(3);
        const int pages[] = {1, 3, 7, 16, 20, 24, 32, 64, 100, 128};
        const int parts[] = {2, 4, 8, 12, 16};
        share(lens, 1 + rnd(9), pages[rnd(10)], 152, parts[rnd(5)]);
    }
    share({}, 1, 16, 152, 8);
    printf(bad ? "%d wrong\n" : "ok\n", bad);
    return bad != 0;
}
