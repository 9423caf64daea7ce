// How the work of attention over a paged cache is cut and shared out, for a
// batch whose lengths only the device knows.
//
//   segment   one set of keys and the query tokens that see it: segment 0 is
//             the shared prefix with every token of the batch, segment 1 + r
//             request r's own keys with its own tokens
//   unit      up to `unit_tokens` consecutive tokens of a segment with all
//             G query heads of one key head: the rows that share a key tile
//   tile      128 keys of a unit
// All tiles of all units lie on one line: segments in order, in a segment the
// key heads, in a head the token groups, in a unit its tiles.  A tile takes
// light_tile places, or heavy_tile where its unit has many rows, and a unit
// some places before its first tile, for what it costs to begin and to end one, so that a place takes about the same time everywhere.  The line is cut
// into `workers` equal stretches, one for each CTA, so that one long request,
// many short ones and a prefix all fill the GPU alike.  The tiles of a unit that
// begin in a stretch are a piece; it leaves a partial (o, lse) for its rows: in
// the rows' own place (home) if the piece begins the unit, else in the worker's
// slot, as only a worker's first piece can begin inside a unit.  Workspace:
// two homes for every row and 256 rows for every worker, whatever the lengths.
// Every place is written once and joined in a fixed order by the next launch:
// results do not depend on timing.
//
// Every CTA scans the R lengths itself (8 bytes a request, from L2), which
// takes 1.8 us and saves a launch.
#pragma once

#include "rsa_internal.h"

namespace rsa {
namespace paged {

constexpr int kTileKeys = 128;
struct Segment {
    int tok0, ntok;        // its query tokens
    int keys;              // its keys
    const int32_t *pages;  // their pages
    int groups, tiles;     // token groups; key tiles of a unit
    int see0;              // token i of the segment sees keys [0, min(keys, see0 + i)): all of the prefix
    int cost, unit;        // places of a tile; of a unit before its first one
    int64_t line;          // places on the line

    // (below 2^26: fewer than 2^24 tiles of 128 keys)
    __device__ __forceinline__ int unit_line() const { return tiles * cost + unit; }
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Segment s, its lengths forced into the buffers (`report`: and recorded).
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
    g.tiles = (int)(((int64_t)g.keys + kTileKeys - 1) / kTileKeys);
    g.cost = g.ntok > p.light_tokens ? p.heavy_tile : p.light_tile;
    g.unit = p.unit + (min(g.ntok, p.unit_tokens) * p.G >> p.unit_shift);
    g.line = g.tiles > 0 ? (int64_t)g.groups * p.Hkv * g.unit_line() : 0;
    return g;
}

// Places of a worker on a line of `total`: never less than a tile takes, so that
// every stretch inside a unit has a piece of it.
__device__ __forceinline__ int64_t share_of(const PrefixAttnParams &p, int64_t total)
{
    return max((total + p.workers - 1) / p.workers, (int64_t)(p.T > p.light_tokens ? p.heavy_tile : p.light_tile));
}

// A worker's stretch of the line, and where it begins.
struct Stretch {
    Segment g;     // its first segment
    int64_t off;   // its first place on that segment's line
    int64_t left;  // its places
    int seg;
};

// Every thread of the block (NT of them) calls this with a word of shared
// memory a warp.  Worker 0 leaves the sums for the joining launch: plan[s] = the
// line's places before segment s, plan[R + 1] = all of them.
template <int NT>
__device__ __forceinline__ Stretch find_stretch(const PrefixAttnParams &p, int worker, int64_t *s_sum,
                                                Stretch *s_out)
{
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nseg = p.R + 1;
    // The line's length: with up to NT segments it falls out of the scan below.
    int64_t total = 0;
    if (nseg > NT) {
        for (int s = threadIdx.x; s < nseg; s += NT)
            total += segment(p, s).line;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0)
            s_sum[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            total += s_sum[w];
    }
    if (threadIdx.x == 0)
        s_out->left = 0;
    int64_t before = 0;
    for (int s0 = 0; s0 < nseg; s0 += NT) {
        const int s = s0 + threadIdx.x;
        Segment g;
        g.line = 0;
        if (s < nseg)
            g = segment(p, s, worker == 0);
        int64_t x = g.line;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        __syncthreads();  // s_sum is free
        if (lane == 31)
            s_sum[warp] = x;
        __syncthreads();
        int64_t first = before + x - g.line;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp)
                first += s_sum[w];
            before += s_sum[w];
        }
        if (nseg <= NT)
            total = before;
        const int64_t share = share_of(p, total);
        const int64_t at = worker * share;
        if (worker == 0) {
            if (s < nseg)
                p.plan[s] = first;
            if (s == p.R)
                p.plan[p.R + 1] = total;
        }
        if (g.line > 0 && at >= first && at < first + g.line)
            *s_out = Stretch{g, at - first, min(share, total - at), s};
    }
    __syncthreads();
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
struct Batch {
    Segment mine;
    int base = -64;

    __device__ __forceinline__ Segment get(const PrefixAttnParams &p, int s)
    {
        const int lane = threadIdx.x & 31;
        if (s - base >= 32) {
            base = s;
            mine = segment(p, min(s + lane, p.R));
        }
        const int from = s - base;
        Segment g;
        g.tok0 = __shfl_sync(0xffffffffu, mine.tok0, from);
        g.ntok = __shfl_sync(0xffffffffu, mine.ntok, from);
        g.keys = __shfl_sync(0xffffffffu, mine.keys, from);
        g.pages = reinterpret_cast<const int32_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.pages), from));
        g.groups = __shfl_sync(0xffffffffu, mine.groups, from);
        g.tiles = __shfl_sync(0xffffffffu, mine.tiles, from);
        g.see0 = __shfl_sync(0xffffffffu, mine.see0, from);
        g.cost = __shfl_sync(0xffffffffu, mine.cost, from);
        g.unit = __shfl_sync(0xffffffffu, mine.unit, from);
        g.line = __shfl_sync(0xffffffffu, mine.line, from);
        return g;
    }
};

// Walks a worker's pieces.  Roles of a CTA that walk by themselves see the same pieces.
struct Walk {
    Segment g;
    int seg, head, group;
    int at;        // the next place in the unit
    int64_t left;  // places left

    __device__ __forceinline__ void begin(const Stretch &st)
    {
        left = st.left;
        if (left <= 0)
            return;
        seg = st.seg;
        g = st.g;
        const int len = g.unit_line();
        const int64_t unit = st.off / len;
        at = (int)(st.off - unit * len);
        head = (int)(unit / g.groups);
        group = (int)(unit - (int64_t)head * g.groups);
    }
    // The first tile that begins at place `u` of the unit or later.
    __device__ __forceinline__ int first_tile(int u) const
    {
        return u <= g.unit ? 0 : (u - g.unit + g.cost - 1) / g.cost;
    }
    __device__ __forceinline__ bool next(const PrefixAttnParams &p, Piece &x)
    {
        return next(p, x, [&](int s) { return segment(p, s); });
    }
    // With `segment_of` to say what a segment is.
    template <class F>
    __device__ __forceinline__ bool next(const PrefixAttnParams &p, Piece &x, F segment_of)
    {
        while (left > 0) {
            if (head >= p.Hkv || g.line == 0) {
                if (++seg > p.R)
                    return false;  // (only if the lengths changed meanwhile)
                g = segment_of(seg);
                head = group = at = 0;
                continue;
            }
            const int len = g.unit_line(), end = (int)min((int64_t)len, at + left);
            const int i0 = group * p.unit_tokens;
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
                if (++group == g.groups) {
                    group = 0;
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
