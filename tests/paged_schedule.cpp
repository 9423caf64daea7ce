// The sharing out of attention over a paged cache, run on the host: every tile of every unit has to
// be taken by exactly one worker, in pieces whose partials have a place of their own.
//   paged_schedule SEED CASES
// A thread of one lane stands for a warp; what the schedule needs of CUDA is defined here.
#include <cuda_runtime.h>

#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <type_traits>
#include <vector>

template <class A, class B>
static std::common_type_t<A, B> min(A a, B b) { return b < a ? b : a; }
template <class A, class B>
static std::common_type_t<A, B> max(A a, B b) { return a < b ? b : a; }
static const struct { int x; } threadIdx = {0};
template <class T>
static T __shfl_sync(unsigned, T v, int) { return v; }
template <class T>
static T __shfl_up_sync(unsigned, T v, int) { return v; }
template <class T>
static T __shfl_xor_sync(unsigned, T v, int) { return v; }
static void __syncthreads() {}
static void __syncwarp() {}
static unsigned __funnelshift_r(unsigned lo, unsigned hi, unsigned s) { return (unsigned)((((uint64_t)hi << 32) | lo) >> (s & 31)); }
static unsigned atomicCAS(unsigned *p, unsigned want, unsigned v) { const unsigned was = *p; *p = was == want ? v : was; return was; }
static unsigned atomicOr(unsigned *p, unsigned v) { const unsigned was = *p; *p |= v; return was; }

#include "../context_attention_rsa_gb300/csrc/paged_sched.cuh"

using namespace rsa;
using namespace rsa::paged;

static std::mt19937 rng;
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

// What one worker takes: false where something is wrong with it.
template <bool kSide>
static bool take(const PrefixAttnParams &p, int worker, std::map<std::tuple<int, int, int, int>, int> &taken)
{
    int64_t singles = 0, pairs = 0;
    for (int s = 0; s <= p.R; ++s) {
        const Segment g = segment<kSide>(p, s);
        singles += g.line;
        pairs += g.pair_line;
    }
    Stretch st;
    st.left = 0;
    int64_t single0 = 0, pair0 = 0;
    for (int s = 0; s <= p.R; ++s) {
        const Segment g = segment<kSide>(p, s);
        place(p, Line(p, pairs, singles), pairs, singles, worker, g, s, single0, pair0, kSide, &st);
        single0 += g.line;
        pair0 += g.pair_line;
    }
    Walk<kSide> walk;
    walk.begin(p, st, worker);
    int slots = 0;
    for (Piece x; walk.next(p, x);) {
        const Segment g = segment<kSide>(p, x.seg);
        if (x.t0 < 0 || x.t1 <= x.t0 || x.t1 > g.tiles || x.head < 0 || x.head >= p.Hkv || x.tok < g.tok0 || x.ntok < 1 ||
            x.ntok > p.unit_tokens || x.tok + x.ntok > g.tok0 + g.ntok || (x.tok - g.tok0) % p.unit_tokens)
            return false;
        if (x.first != (x.t0 == 0) || x.whole != (x.t0 == 0 && x.t1 == g.tiles))
            return false;
        slots += !x.first;
        for (int t = x.t0; t < x.t1; ++t)
            ++taken[{x.seg, x.head, (x.tok - g.tok0) / p.unit_tokens, t}];
    }
    return slots <= 1;  // (a worker has one slot for a unit that another began)
}

template <bool kSide>
static bool all(const PrefixAttnParams &p)
{
    std::map<std::tuple<int, int, int, int>, int> taken;
    for (int w = 0; w < p.workers; ++w)
        if (!take<kSide>(p, w, taken))
            return false;
    size_t want = 0;
    for (int s = 0; s <= p.R; ++s) {
        const Segment g = segment<kSide>(p, s);
        want += (size_t)g.groups * p.Hkv * g.tiles;
    }
    for (const auto &t : taken)
        if (t.second != 1)
            return false;
    return taken.size() == want;
}

int main(int argc, char **argv)
{
    rng.seed(argc > 1 ? atoi(argv[1]) : 0);
    const int cases = argc > 2 ? atoi(argv[2]) : 100;
    for (int i = 0; i < cases; ++i) {
        PrefixAttnParams p = {};
        const int workers[] = {1, 2, 3, 8, 152, 160}, groups[] = {1, 2, 5, 8, 40, 64, 128};
        p.workers = workers[pick(0, 5)];
        p.G = groups[pick(0, 6)];
        p.Hkv = pick(1, 5);
        p.R = pick(1, 12);
        const bool side = pick(0, 1), light = pick(0, 1);
        p.unit_tokens = side || light ? max(1, 128 / p.G) * (side ? 2 : 1) : 2 * max(1, 128 / p.G);
        p.light_tokens = max(1, p.unit_tokens / 2);
        p.light_tile = light ? 1 : 2;
        p.heavy_tile = light ? 2 : 3;
        p.tile_shift = light ? 5 : 7;
        p.unit = light ? 4 : 6;
        p.unit_shift = pick(0, 1) ? 5 : 31;
        p.side_by_side = side ? side_by_side(p.workers) : 0;
        p.page_shift = 4;
        p.max_pages = 400;
        p.prefix_len = pick(0, 2) ? 0 : pick(1, 3000);
        std::vector<int32_t> cu(1, pick(0, 3) ? 0 : pick(0, 5)), kv;
        for (int r = 0; r < p.R; ++r) {
            const int n = pick(0, 4) ? pick(0, 20) : pick(0, 300);
            cu.push_back(cu.back() + n);
            kv.push_back(pick(0, 5) ? n + pick(0, 3000) : pick(0, n + 1));
        }
        p.T = max(1, cu.back() + pick(0, 3));
        std::vector<int32_t> table(p.R * p.max_pages), pages(300);
        p.cu_q = cu.data();
        p.kv_len = kv.data();
        p.block_table = table.data();
        p.table_stride = p.max_pages;
        p.prefix_pages = pages.data();
        if (!(side ? all<true>(p) : all<false>(p))) {
            printf("case %d: workers %d G %d Hkv %d R %d side %d prefix %lld\n", i, p.workers, p.G, p.Hkv, p.R, (int)side,
                   (long long)p.prefix_len);
            return 1;
        }
    }
    return 0;
}
