// Kept rows of a paged cache moved together, in place, in all layers.
//
//   row(base + i) <- row(base + keep_i),  i < m,  keep strictly ascending
//
// keep_i >= i, so a row's new place is never behind its old one, and never at or behind
// the old place of a row that comes later: if the rows go in ascending order, each is
// read before it is written over.  The 16-byte columns of a row do not meet, and
// neither do layers, heads, keys and values.  So a block takes the columns of some of
// them and goes through the list in batches: every thread reads its rows of the batch, a
// barrier, then it writes them; no batch reads what an earlier one has written.  Rows that
// stay where they are (an accepted path's first tokens) are not touched.
// A block checks all of its request's list, and the pages in it, before it moves
// anything, so that all blocks of a request agree.
#include "ptx_sm103.cuh"
#include "rsa_internal.h"

namespace rsa {
namespace {

struct Cut {
    int cols;        // 16-byte columns of a row that a block takes
    int parts;       // blocks that share a row
    int row_lanes;   // threads that share a column, each with kDepth rows of a batch
    int slabs;       // (layer, head, keys or values) of a block
};

// A kept row: where it lies and where it goes, in rows of key head 0 of a layer; -1: stays.
struct Move {
    int64_t from, to;
};

__device__ __forceinline__ int64_t row_of(const CompactParams &p, int page, int token)
{
    return (((int64_t)page * p.c.Hkv) << p.c.page_shift) + (token & ((1 << p.c.page_shift) - 1));
}

// kDepth: rows that a thread has in flight.  kOnce: no list is longer than a batch.
template <int kThreads, int kDepth, bool kOnce>
__global__ void __launch_bounds__(kThreads) cache_compact_kernel(const __grid_constant__ CompactParams p, const Cut cut)
{
    extern __shared__ Move s_move[];  // of a batch (of three, in turn)
    const int r = blockIdx.x, tid = threadIdx.x, batch = cut.row_lanes * kDepth;
    ptx::wait_for_launch_before();
    const int base = p.cached_len[r], all = p.kv_len[r], m = p.keep_len[r];
    const int32_t *keep = p.keep + r * p.keep_stride;

    // ---- can the list be followed? -------------------------------------------------
    const int64_t room = (int64_t)p.max_pages << p.c.page_shift;
    bool ok = base >= 0 && all >= base && all <= room && m >= 0 && m <= p.max_keep;
    const bool tell = blockIdx.y == 0;
    if (!ok && tell && tid == 0)
        record_bad_index(p.err, kSiteCompactLen, base < 0 ? base : (all < base || all > room ? all : m));
    int bad = 0;
    if (ok)
        for (int i = tid; i < m; i += kThreads) {
            const int k = keep[i], before = i > 0 ? keep[i - 1] : -1;
            if (k <= before || k < 0 || k >= all - base) {
                if (tell)
                    record_bad_index(p.err, kSiteKeep, k);
                bad = 1;
                continue;
            }
            if (k == i) {
                if (i < batch)
                    s_move[i] = Move{-1, -1};
                continue;
            }
            const int32_t *table = p.block_table + r * p.table_stride;
            const int from = table[(base + k) >> p.c.page_shift];
            const int to = i < all - base ? table[(base + i) >> p.c.page_shift] : -1;  // (i >= all - base: the list does not ascend)
            if (from < 0 || from >= p.c.n_pages || to < 0 || to >= p.c.n_pages) {
                if (tell)
                    record_bad_index(p.err, kSiteCompactPage, from < 0 || from >= p.c.n_pages ? from : to);
                bad = 1;
            } else if (i < batch) {
                s_move[i] = Move{row_of(p, from, base + k), row_of(p, to, base + i)};
            }
        }
    ok = !__syncthreads_or(bad) && ok;
    if (tell && tid == 0)
        p.new_len[r] = ok ? base + m : base;
    if (!ok)
        return;

    // ---- the moves -----------------------------------------------------------------
    const int col = tid % cut.cols, lane = tid / cut.cols % cut.row_lanes, slab0 = tid / (cut.cols * cut.row_lanes);
    const int group = blockIdx.y / cut.parts, part = blockIdx.y - group * cut.parts;
    const int slab = group * cut.slabs + slab0;
    const bool works = slab < 2 * p.c.layers * p.c.Hkv;
    const int head = slab % p.c.Hkv, kv = slab / p.c.Hkv & 1, layer = works ? slab / (2 * p.c.Hkv) : 0;
    char *at = p.c.data[kv] + layer * p.c.layer_bytes + (((int64_t)head << p.c.page_shift) * p.c.row) +
               (part * cut.cols + col) * 16;
    uint4 x[kDepth];
    auto read = [&](const Move *list, int n) {
#pragma unroll
        for (int e = 0; e < kDepth; ++e) {
            const int i = e * cut.row_lanes + lane;
            if (works && i < n && list[i].from >= 0)
                x[e] = *reinterpret_cast<const uint4 *>(at + list[i].from * p.c.row);
        }
    };
    auto write = [&](const Move *list, int n) {
#pragma unroll
        for (int e = 0; e < kDepth; ++e) {
            const int i = e * cut.row_lanes + lane;
            if (works && i < n && list[i].from >= 0)
                *reinterpret_cast<uint4 *>(at + list[i].to * p.c.row) = x[e];
        }
    };
    if constexpr (kOnce) {
        read(s_move, m);
        __syncthreads();  // all has been read
        write(s_move, m);
        return;
    }
    // Three lists in turn: one is written while the batch before it is read, and the one before
    // that may still be being written back.
    const int32_t *table = p.block_table + r * p.table_stride;
    Move *list = s_move, *next = s_move + batch, *after = next + batch;
    for (int i0 = 0; i0 < m; i0 += batch) {
        read(list, m - i0);
        for (int i = tid; i < batch && i0 + batch + i < m; i += kThreads) {
            const int to = i0 + batch + i, k = keep[to];
            next[i] = Move{-1, -1};
            if (k != to)
                next[i] = Move{row_of(p, table[(base + k) >> p.c.page_shift], base + k),
                               row_of(p, table[(base + to) >> p.c.page_shift], base + to)};
        }
        __syncthreads();  // the batch has been read, the next one's list is there
        write(list, m - i0);
        Move *const done = list;
        list = next;
        next = after;
        after = done;
    }
}

template <int kThreads, int kDepth, bool kOnce>
cudaError_t launch(const CompactParams &p, cudaStream_t s)
{
    Cut cut;
    const int64_t slabs = 2ll * p.c.layers * p.c.Hkv;
    cut.cols = p.c.row / 16;
    cut.parts = 1;
    // (where blocks are few, several share a row, down to 64 bytes each, for longer batches)
    for (; !kOnce && cut.cols > 4 && p.R * slabs * cut.parts * 2 <= 152; cut.cols /= 2)
        cut.parts *= 2;
    cut.row_lanes = 1;
    while (cut.row_lanes * kDepth < p.max_keep && cut.row_lanes * cut.cols < kThreads)
        cut.row_lanes *= 2;
    cut.slabs = kThreads / (cut.cols * cut.row_lanes);
    const int64_t groups = (slabs + cut.slabs - 1) / cut.slabs * cut.parts;  // (below 2^16)
    const size_t smem = (kOnce ? 1 : 3) * sizeof(Move) * cut.row_lanes * kDepth;  // (at most 24 KB)
    return launch_early(cache_compact_kernel<kThreads, kDepth, kOnce>, dim3((unsigned)p.R, (unsigned)groups), kThreads, smem, s, 1, p, cut);
}

}  // namespace

// Short lists fit a batch of 256 threads (64 requests with up to 6 rows in 16 layers 6.0 us;
// by the loop, when launches cost 2 us more, 10.2 against 8.2).  Long ones go through
// batches of 128 rows of a head at least: whole rows of whole pages (4 caches of 8192 rows
// in 4 layers 178 us, 6.0 TB/s, 0.88 of a copy; with
// 256 threads of 8 rows 194, with blocks that share rows by columns 191 to 330).
cudaError_t launch_cache_compact(const CompactParams &p, cudaStream_t s)
{
    return p.max_keep <= 8 * 256 / (p.c.row / 16) ? launch<256, 8, true>(p, s) : launch<512, 4, false>(p, s);
}

}  // namespace rsa
