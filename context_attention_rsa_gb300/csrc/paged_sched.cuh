// How the work of attention over a paged cache is cut and shared out, for a
// batch whose lengths only the device knows.
//
//   segment   one set of keys and the query tokens that see it: segment 0 is
//             the shared prefix with every token of the batch, segment 1 + r
//             request r's own keys with its own tokens
//   unit      up to `unit_tokens` consecutive tokens of a segment with all
//             G query heads of one key head: the rows that share a key tile
//   tile      128 keys of a unit (of few drafted tokens in fp32: fewer)
// All tiles of all units lie on one line: segments in order, in a segment the
// key heads, in a head the token groups, in a unit its tiles.  A tile takes
// light_tile places, or heavy_tile where its unit has many rows, and a unit
// some places before its first tile, for what it costs to begin and to end one,
// so that a place takes about the same time everywhere.  The line is cut into
// `workers` equal stretches, one for each CTA, so that one long request, many
// short ones and a prefix all fill the GPU alike.  The tiles of a unit that
// begin in a stretch are a piece; it leaves a partial (o, lse) for its rows: in
// the rows' own place (home) if the piece begins the unit, else in the worker's
// slot, as only a worker's first piece can begin inside a unit.  Workspace:
// two homes for every row and 256 rows for every worker, whatever the lengths.
// Every place is written once and joined in a fixed order by the next launch:
// results do not depend on timing.
//
// Side by side (drafted tokens on the tensor cores): units of one key head against the same
// keys are taken at the same time by different workers, so that its tiles come from L2 for
// all but one of them; at other times they come from HBM again.
//   - where the prefix has a unit for every worker or more, each first takes a whole
//     one, or several, and only the rest is on the line;
//   - two token groups of a request are a pair.  The line begins with the even groups of
//     all pairs, then the odd ones in the same order, then the units of no pair; the even
//     ones are padded to whole stretches, so that the two of a pair lie a whole number
//     of stretches apart.
//
// Every CTA scans the R lengths itself (8 bytes a request, from L2), which
// takes 1.8 us and saves a launch.
#pragma once

#include "rsa_internal.h"

namespace rsa {
namespace paged {

constexpr int kTileShift = 7, kTileKeys = 1 << kTileShift;

// PrefixAttnParams::side_by_side of a call that wants it: there have to be two workers for two units,
// and with one the odd groups would lie behind its stretch.
inline int side_by_side(int workers) { return workers > 1 ? -1 : 0; }

struct Segment {
    int tok0, ntok;        // its query tokens
    int keys;              // its keys
    const int32_t *pages;  // their pages
    int groups, tiles;     // token groups; key tiles of a unit
    int see0;              // token i of the segment sees keys [0, min(keys, see0 + i)): all of the prefix
    int cost, unit;        // places of a tile; of a unit before its first one
    int pairs, singles;    // pairs of token groups, groups of no pair
    int skip;              // its first units (of no pair) that are not on the line
    int64_t line;          // places on the line of its units of no pair
    int64_t pair_line;     // ... of the even ones of its pairs

    // (below 2^28: fewer than 2^26 tiles of 32 keys or 2^24 of 128)
    __device__ __forceinline__ int unit_line() const { return tiles * cost + unit; }
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Segment s, its lengths forced into the buffers (`report`: and recorded).  kSide false: units
// are taken in order, whatever p says.
template <bool kSide>
__device__ __forceinline__ Segment segment(const PrefixAttnParams &p, int s, bool report = false)
{
    Segment g;
    const int T = (int)p.T;
    if (s == 0) {
        g.tok0 = 0;
        g.keys = (int)p.prefix_len;
        g.ntok = p.prefix_len > 0 ? clamp_int(p.cu_q[p.R], 0, T) : 0;
        g.pages = p.prefix_pages;
        g.see0 = g.keys;
    } else {
        const int r = s - 1, a = p.cu_q[r], b = p.cu_q[r + 1], n = p.kv_len[r];
        g.tok0 = clamp_int(a, 0, T);
        g.ntok = clamp_int(b, g.tok0, T) - g.tok0;
        g.keys = clamp_int(n, 0, p.max_pages << p.page_shift);
        g.pages = p.block_table + r * p.table_stride;
        g.see0 = g.keys - g.ntok + 1;
        if (report) {
            if (g.tok0 != a)
                record_bad_index(p.err, kSiteQueryRows, a);
            else if (g.tok0 + g.ntok != b)
                record_bad_index(p.err, kSiteQueryRows, b);
            if (g.keys != n)
                record_bad_index(p.err, kSiteKvLen, n);
        }
    }
    g.groups = (int)(((int64_t)g.ntok + p.unit_tokens - 1) / p.unit_tokens);
    g.tiles = (int)(((int64_t)g.keys + (1 << p.tile_shift) - 1) >> p.tile_shift);
    g.cost = g.ntok > p.light_tokens ? p.heavy_tile : p.light_tile;
    g.unit = p.unit + (min(g.ntok, p.unit_tokens) * p.G >> p.unit_shift);
    g.pairs = kSide && s > 0 ? (g.groups & p.side_by_side) >> 1 : 0;
    g.singles = g.groups - 2 * g.pairs;
    const int64_t units = (int64_t)g.singles * p.Hkv;
    g.skip = kSide && s == 0 && g.tiles > 0 ? (int)(units / p.workers) * p.workers & p.side_by_side : 0;
    g.line = g.tiles > 0 ? (units - g.skip) * g.unit_line() : 0;
    g.pair_line = g.tiles > 0 ? (int64_t)g.pairs * p.Hkv * g.unit_line() : 0;
    return g;
}

// The line: its parts, and a worker's places on it: never less than a tile takes, so that
// every stretch inside a unit has a piece of it.
struct Line {
    int64_t share;
    int64_t odd, rest;  // where the odd groups and the units of no pair begin

    __device__ __forceinline__ Line(const PrefixAttnParams &p, int64_t pairs, int64_t singles)
    {
        // (the even groups' padding takes a part of one stretch)
        const int64_t total = 2 * pairs + singles, over = p.workers - (pairs > 0 && p.workers > 1);
        share = max((total + over - 1) / over, (int64_t)(p.T > p.light_tokens ? p.heavy_tile : p.light_tile));
        odd = pairs > 0 ? (pairs + share - 1) / share * share : 0;
        rest = odd + pairs;
    }
};

// A worker's stretch of the line, and where it begins.
struct Stretch {
    Segment g;     // its first segment
    int64_t off;   // its first place on that segment's part of the line
    int64_t left;  // its places
    int seg;
    int part;      // of the line: even groups, odd groups, units of no pair
};

// Writes down the worker's stretch if it begins in segment s, before which lie `single0` and
// `pair0` places.
__device__ __forceinline__ void place(const PrefixAttnParams &p, const Line &line, int64_t pairs, int64_t singles, int worker,
                                      const Segment &g, int s, int64_t single0, int64_t pair0, bool side, Stretch *s_out)
{
    const int64_t at = worker * line.share, end = line.rest + singles, single = at - line.rest;
    if (g.line > 0 && single >= single0 && single < single0 + g.line)
        *s_out = Stretch{g, single - single0, min(line.share, end - at), s, 2};
    if (side && g.pair_line > 0 && single < 0) {
        const int part = at >= line.odd;
        const int64_t pair = part ? at - line.odd : at;
        if (pair >= pair0 && pair < pair0 + g.pair_line)
            *s_out = Stretch{g, pair - pair0, min(line.share, (part ? end : pairs) - at), s, part};
    }
}

// Every thread of the block (NT of them) calls this with a word of shared
// memory a warp (kSide: two).  Worker 0 leaves the sums for the joining launch: plan[s] =
// the places before segment s's units of no pair, plan[R + 1] = all of them; pair_plan for the
// even groups.
template <int NT, bool kSide>
__device__ __forceinline__ Stretch find_stretch(const PrefixAttnParams &p, int worker, int64_t *s_sum,
                                                Stretch *s_out)
{
    constexpr int NW = NT / 32, kSums = kSide ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nseg = p.R + 1;
    // The line's length: with up to NT segments it falls out of the scan below.
    int64_t total[2] = {0, 0};
    if (nseg > NT) {
        for (int s = threadIdx.x; s < nseg; s += NT) {
            const Segment g = segment<kSide>(p, s);
            total[0] += g.line;
            total[1] += g.pair_line;
        }
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                total[k] += __shfl_xor_sync(0xffffffffu, total[k], o);
            if (lane == 0)
                s_sum[k * NW + warp] = total[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            total[k] = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                total[k] += s_sum[k * NW + w];
        }
    }
    if (threadIdx.x == 0)
        s_out->left = 0;
    int64_t before[2] = {0, 0};
    for (int s0 = 0; s0 < nseg; s0 += NT) {
        const int s = s0 + threadIdx.x;
        Segment g;
        g.line = g.pair_line = 0;
        if (s < nseg)
            g = segment<kSide>(p, s, worker == 0);
        int64_t x[2] = {g.line, g.pair_line};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
            for (int k = 0; k < kSums; ++k) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
                if (lane >= o)
                    x[k] += y;
            }
        }
        __syncthreads();  // s_sum is free
        if (lane == 31) {
#pragma unroll
            for (int k = 0; k < kSums; ++k)
                s_sum[k * NW + warp] = x[k];
        }
        __syncthreads();
        int64_t first[2] = {before[0] + x[0] - g.line, before[1] + x[1] - g.pair_line};
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < warp)
                    first[k] += s_sum[k * NW + w];
                before[k] += s_sum[k * NW + w];
            }
            if (nseg <= NT)
                total[k] = before[k];
        }
        const Line line(p, kSide ? total[1] : 0, total[0]);
        if (worker == 0) {
            if (s < nseg)
                p.plan[s] = first[0];
            if (s == p.R)
                p.plan[p.R + 1] = total[0];
            if (kSide && s < nseg)
                p.pair_plan[s] = first[1];
            if (kSide && s == p.R)
                p.pair_plan[p.R + 1] = total[1];
        }
        place(p, line, kSide ? total[1] : 0, total[0], worker, g, s, first[0], first[1], kSide, s_out);
    }
    __syncthreads();
    return *s_out;
}

// The same for fewer than 32 requests, by a warp that needs it: a lane each, no barrier (one
// request of 1000 keys 11.8 -> 11.3 us, now 10.6).  The joining launch then asks for no sums.
template <bool kSide>
__device__ __forceinline__ Stretch few_stretch(const PrefixAttnParams &p, int worker, Stretch *s_out, bool report)
{
    const int lane = threadIdx.x & 31;
    Segment g;
    g.line = g.pair_line = 0;
    if (lane <= p.R)
        g = segment<kSide>(p, lane, report && worker == 0);
    int64_t x[2] = {g.line, g.pair_line};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < (kSide ? 2 : 1); ++k) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o)
                x[k] += y;
        }
    }
    const int64_t singles = __shfl_sync(0xffffffffu, x[0], 31), pairs = kSide ? __shfl_sync(0xffffffffu, x[1], 31) : 0;
    if (lane == 0)
        s_out->left = 0;
    __syncwarp();
    place(p, Line(p, pairs, singles), pairs, singles, worker, g, lane, x[0] - g.line, x[1] - g.pair_line, kSide, s_out);
    __syncwarp();
    return *s_out;
}

// One piece: tiles [t0, t1) of a unit.
struct Piece {
    int seg;
    int tok, ntok;         // the unit's tokens
    int head;              // its key head
    int keys;              // the segment's keys
    const int32_t *pages;
    int64_t see0;          // unit token i sees keys [0, min(keys, see0 + i))
    int drafted;           // the segment's keys from here on are its tokens' own (the prefix: none); may be negative
    int t0, t1;
    bool first, whole;     // it begins the unit; it is all of it
};

// Segments in ascending order for a warp that walks them: a lane each, 32 at a time,
// so that a batch of short ones does not wait for its lengths request by request.
template <bool kSide>
struct Batch {
    Segment mine;
    int base = -64;

    __device__ __forceinline__ Segment get(const PrefixAttnParams &p, int s)
    {
        const int lane = threadIdx.x & 31;
        if ((kSide && s < base) || s - base >= 32) {
            base = s;
            mine = segment<kSide>(p, min(s + lane, p.R));
        }
        const int from = s - base;
        Segment g;
        g.tok0 = __shfl_sync(0xffffffffu, mine.tok0, from);
        g.ntok = __shfl_sync(0xffffffffu, mine.ntok, from);
        g.keys = __shfl_sync(0xffffffffu, mine.keys, from);
        g.pages = reinterpret_cast<const int32_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.pages), from));
        g.singles = __shfl_sync(0xffffffffu, mine.singles, from);
        g.pairs = kSide ? __shfl_sync(0xffffffffu, mine.pairs, from) : 0;
        g.skip = kSide ? __shfl_sync(0xffffffffu, mine.skip, from) : 0;
        g.tiles = __shfl_sync(0xffffffffu, mine.tiles, from);
        g.see0 = __shfl_sync(0xffffffffu, mine.see0, from);
        g.cost = __shfl_sync(0xffffffffu, mine.cost, from);
        g.unit = __shfl_sync(0xffffffffu, mine.unit, from);
        return g;
    }
};

// Walks a worker's pieces.  Roles of a CTA that walk by themselves see the same pieces.
template <bool kSide>
struct Walk {
    Segment g;
    int seg, part, head;
    int k;         // the unit of the key head's in this part of the line
    int at;        // the next place in the unit
    int64_t left;  // places left
    int whole, skip;  // the next of the prefix' units that are not on the line, and their number

    __device__ __forceinline__ void begin(const PrefixAttnParams &p, const Stretch &st, int worker)
    {
        whole = worker;
        skip = kSide ? segment<kSide>(p, 0).skip : 0;
        left = st.left;
        if (left <= 0)
            return;
        seg = st.seg;
        part = kSide ? st.part : 2;
        g = st.g;
        const int len = g.unit_line();
        const int64_t unit = st.off / len;
        at = (int)(st.off - unit * len);
        enter(unit + (kSide && part == 2 ? g.skip : 0));
    }
    __device__ __forceinline__ int of_head() const { return !kSide || part == 2 ? g.singles : g.pairs; }
    __device__ __forceinline__ void enter(int64_t unit)
    {
        head = (int)(unit / of_head());
        k = (int)(unit - (int64_t)head * of_head());
    }
    // The first tile that begins at place `u` of the unit or later.
    __device__ __forceinline__ int first_tile(int u) const
    {
        return u <= g.unit ? 0 : (u - g.unit + g.cost - 1) / g.cost;
    }
    __device__ __forceinline__ bool next(const PrefixAttnParams &p, Piece &x)
    {
        return next(p, x, [&](int s) { return segment<kSide>(p, s); });
    }
    // With `segment_of` to say what a segment is.
    template <class F>
    __device__ __forceinline__ bool next(const PrefixAttnParams &p, Piece &x, F segment_of)
    {
        if (kSide && whole < skip) {
            const Segment f = segment<kSide>(p, 0);
            const int h = whole / f.groups, i0 = (whole - h * f.groups) * p.unit_tokens;
            x.seg = 0;
            x.tok = f.tok0 + i0;
            x.ntok = min(p.unit_tokens, f.ntok - i0);
            x.head = h;
            x.keys = x.drafted = f.keys;
            x.pages = f.pages;
            x.see0 = f.keys;
            x.t0 = 0;
            x.t1 = f.tiles;
            x.first = x.whole = true;
            whole += p.workers;
            return true;
        }
        while (left > 0) {
            if (head >= p.Hkv || of_head() == 0 || g.tiles == 0) {
                if (++seg > p.R) {
                    if (!kSide || part != 1)
                        return false;  // (only if the lengths changed meanwhile)
                    part = 2;          // after the odd groups
                    seg = 0;
                }
                g = segment_of(seg);
                head = k = at = 0;
                if (kSide && seg == 0 && of_head() > 0)
                    enter(g.skip);
                continue;
            }
            const int len = g.unit_line(), end = (int)min((int64_t)len, at + left);
            const int i0 = (!kSide ? k : (part == 2 ? 2 * g.pairs + k : 2 * k + part)) * p.unit_tokens;
            x.seg = seg;
            x.tok = g.tok0 + i0;
            x.ntok = min(p.unit_tokens, g.ntok - i0);
            x.head = head;
            x.keys = g.keys;
            x.pages = g.pages;
            x.see0 = seg == 0 ? g.keys : (int64_t)g.see0 + i0;
            x.drafted = seg == 0 ? g.keys : g.see0 - 1;
            x.t0 = first_tile(at);
            x.t1 = first_tile(end);
            x.first = x.t0 == 0;
            x.whole = x.first && x.t1 == g.tiles;
            left -= end - at;
            at = end;
            if (at == len) {
                at = 0;
                if (++k == of_head()) {
                    k = 0;
                    ++head;
                }
            }
            if (x.t1 > x.t0)
                return true;  // (else no tile begins in this part)
        }
        return false;
    }
};

// 32 bits of a row's mask from drafted token j on; tokens before the first count as set.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *row, int words, int j)
{
    auto word = [&](int w) { return w < 0 ? 0xffffffffu : (w < words ? row[w] : 0u); };
    return __funnelshift_r(word(j >> 5), word((j >> 5) + 1), j & 31);
}

// The piece is all there is for its rows: its (o, lse) is the result.
__device__ __forceinline__ bool is_result(const PrefixAttnParams &p, const Piece &x)
{
    return x.seg > 0 && x.whole && p.prefix_len == 0;
}

}  // namespace paged
}  // namespace rsa
