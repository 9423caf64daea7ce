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
#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 256;
constexpr int kDepth = 8;  // rows that a thread has in flight

struct Cut {
    int cols;        // 16-byte columns of a row
    int row_lanes;   // threads that share a column, each with kDepth rows of a batch
    int slabs;       // (layer, head, keys or values) of a block
};

// A kept row: where it lies and where it goes, in rows of key head 0 of a layer; -1: stays.
struct Move {
    int64_t from, to;
};

__device__ __forceinline__ int64_t row_of(const CompactParams &p, int r, int token)
{
    const int page = p.block_table[r * p.table_stride + (token >> p.c.page_shift)];
    return (((int64_t)page * p.c.Hkv) << p.c.page_shift) + (token & ((1 << p.c.page_shift) - 1));
}

__global__ void __launch_bounds__(kThreads) cache_compact_kernel(const __grid_constant__ CompactParams p, const Cut cut)
{
    extern __shared__ Move s_move[];  // of a batch
    const int r = blockIdx.x, tid = threadIdx.x, batch = cut.row_lanes * kDepth;
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
            if (k == i)
                continue;
            const int32_t *table = p.block_table + r * p.table_stride;
            const int from = table[(base + k) >> p.c.page_shift];
            const int to = i < all - base ? table[(base + i) >> p.c.page_shift] : -1;  // (i >= all - base: the list does not ascend)
            if (from < 0 || from >= p.c.n_pages || to < 0 || to >= p.c.n_pages) {
                if (tell)
                    record_bad_index(p.err, kSiteCompactPage, from < 0 || from >= p.c.n_pages ? from : to);
                bad = 1;
            }
        }
    ok = !__syncthreads_or(bad) && ok;
    if (tell && tid == 0)
        p.new_len[r] = ok ? base + m : base;
    if (!ok)
        return;

    // ---- the moves -----------------------------------------------------------------
    const int col = tid % cut.cols, lane = tid / cut.cols % cut.row_lanes, slab0 = tid / (cut.cols * cut.row_lanes);
    const int slab = blockIdx.y * cut.slabs + slab0;
    const bool works = slab < 2 * p.c.layers * p.c.Hkv;
    const int head = slab % p.c.Hkv, kv = slab / p.c.Hkv & 1, layer = works ? slab / (2 * p.c.Hkv) : 0;
    char *at = p.c.data[kv] + layer * p.c.layer_bytes + (((int64_t)head << p.c.page_shift) * p.c.row) + col * 16;
    for (int i0 = 0; i0 < m; i0 += batch) {
        for (int i = tid; i < batch && i0 + i < m; i += kThreads) {
            const int k = keep[i0 + i];
            s_move[i] = k == i0 + i ? Move{-1, -1} : Move{row_of(p, r, base + k), row_of(p, r, base + i0 + i)};
        }
        __syncthreads();
        uint4 x[kDepth];
#pragma unroll
        for (int e = 0; e < kDepth; ++e) {
            const int i = e * cut.row_lanes + lane;
            if (works && i0 + i < m && s_move[i].from >= 0)
                x[e] = *reinterpret_cast<const uint4 *>(at + s_move[i].from * p.c.row);
        }
        __syncthreads();  // the batch has been read
#pragma unroll
        for (int e = 0; e < kDepth; ++e) {
            const int i = e * cut.row_lanes + lane;
            if (works && i0 + i < m && s_move[i].from >= 0)
                *reinterpret_cast<uint4 *>(at + s_move[i].to * p.c.row) = x[e];
        }
        __syncthreads();  // s_move is written again
    }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactParams &p, cudaStream_t s)
{
    Cut cut;
    cut.cols = p.c.row / 16;
    cut.row_lanes = 1;
    while (cut.row_lanes * kDepth < p.max_keep && cut.row_lanes * cut.cols < kThreads)
        cut.row_lanes *= 2;
    cut.slabs = kThreads / (cut.cols * cut.row_lanes);
    const int64_t slabs = 2ll * p.c.layers * p.c.Hkv, groups = (slabs + cut.slabs - 1) / cut.slabs;
    const size_t smem = sizeof(Move) * cut.row_lanes * kDepth;  // (at most 4 KB)
    cache_compact_kernel<<<dim3((unsigned)p.R, (unsigned)groups), kThreads, smem, s>>>(p, cut);
    return cudaGetLastError();
}

}  // namespace rsa
