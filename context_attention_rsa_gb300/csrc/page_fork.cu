// Forks of requests over a paged cache: full pages are shared and counted, a partial
// last page (without counts: every page) is copied to a fresh one, in all layers.
//
// One launch and no traffic between blocks, as for the step's plan: every block reads the
// forks and their lengths, checks them and sums up the fresh pages before each, and then
// does its share of the table entries and of the rows.  Nothing that any block reads
// is written by another: sources and destinations are different rows, and a copy's
// destination comes from free_pages.
// A page's rows of one key head lie side by side: a warp reads 4 KB of them, 16 bytes a lane,
// and writes them for every fork of the request: HBM's rate of writes bounds it (240 forks
// of 16 requests in 24 layers of 5 heads, 0.98 GB written, 210 us, 4.7 TB/s; a fill of 1 GB
// takes 267).  Without counts every page is copied (as many forks 18.8 GB, 3155 us, 6.0 TB/s, 0.88 of
// a copy).
#include <climits>

#include "ptx_sm103.cuh"
#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kDepth = 8;             // 16-byte loads that a lane has in flight
constexpr int kPiece = kDepth * 512;  // bytes that a warp copies at once

// Largest i in [0, n) with a[i] <= x, for ascending a with a[0] <= x.
__device__ __forceinline__ int last_not_above(const int *a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// What is counted of a fork.
struct Counts {
    int entries, fresh, copies;  // table entries; fresh pages; pages copied, where it is the first fork of its source

    __device__ __forceinline__ void add(const Counts &x) { entries += x.entries, fresh += x.fresh, copies += x.copies; }
};

// Exclusive sums of the three lists in place, with the totals behind them, by the whole block.
// (They stay below 2^31.)
__device__ __forceinline__ Counts exclusive_sums(int *entries, int *fresh, int *copies, int n, Counts *s_warp)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (n + kThreads - 1) / kThreads | 1;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    Counts mine{0, 0, 0};
    for (int i = i0; i < i1; ++i)
        mine.add(Counts{entries[i], fresh[i], copies[i]});
    Counts x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Counts y{__shfl_up_sync(0xffffffffu, x.entries, o), __shfl_up_sync(0xffffffffu, x.fresh, o),
                       __shfl_up_sync(0xffffffffu, x.copies, o)};
        if (lane >= o)
            x.add(y);
    }
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    Counts before{x.entries - mine.entries, x.fresh - mine.fresh, x.copies - mine.copies}, total{0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp)
            before.add(s_warp[w]);
        total.add(s_warp[w]);
    }
    for (int i = i0; i < i1; ++i) {
        const Counts v{entries[i], fresh[i], copies[i]};
        entries[i] = before.entries, fresh[i] = before.fresh, copies[i] = before.copies;
        before.add(v);
    }
    if (tid == 0)
        entries[n] = total.entries, fresh[n] = total.fresh, copies[n] = total.copies;
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kThreads) page_fork_kernel(const __grid_constant__ PageForkParams p)
{
    extern __shared__ int smem[];
    int *s_pages = smem;                // [F + 1] table entries before each fork
    int *s_fresh = s_pages + p.F + 1;   // [F + 1] fresh pages before each fork
    int *s_copies = s_fresh + p.F + 1;  // [F + 1] pages to copy before each fork, the forks of one source counted once
    int *s_first = s_copies + p.F + 1;  // [R] the first fork of each source
    int *s_forks = s_first + p.R;       // [R] its forks
    unsigned *s_used = reinterpret_cast<unsigned *>(s_forks + p.R);  // a bit for each request: it is in dst
    __shared__ Counts s_warp[kWarps];
    __shared__ int s_list[kWarps][32];
    const int tid = threadIdx.x, P = 1 << p.c.page_shift, F = p.F;
    const bool shared = p.shares != nullptr;

    // ---- the forks, and what makes them impossible ---------------------------------------
    for (int i = tid; i < p.R; i += kThreads) {
        s_first[i] = INT_MAX;
        s_forks[i] = 0;
    }
    for (int i = tid; i < (p.R + 31) / 32; i += kThreads)
        s_used[i] = 0;
    ptx::wait_for_launch_before();
    const long long start = p.free_start ? *p.free_start : 0;
    __syncthreads();
    // (what is wrong is told at barriers, so that all threads take the same ways)
    int bad = 0, bad_len = 0;
    for (int f = tid; f < F; f += kThreads) {
        const int a = p.src[f], b = p.dst[f];
        if (a == -1 && b == -1)
            continue;  // no fork
        if (a < 0 || a >= p.R || b < 0 || b >= p.R || (atomicOr(&s_used[b >> 5], 1u << (b & 31)) >> (b & 31) & 1)) {
            bad = 1;
            continue;
        }
        s_pages[f] = p.kv_len[a];
        atomicMin(&s_first[a], f);
        atomicAdd(&s_forks[a], 1);
    }
    bad = __syncthreads_or(bad);
    if (!bad)
        for (int f = tid; f < F; f += kThreads) {
            const int a = p.src[f];
            if (a < 0) {
                s_pages[f] = s_fresh[f] = s_copies[f] = 0;
                continue;
            }
            const int n = s_pages[f];
            if (s_used[a >> 5] >> (a & 31) & 1)
                bad = 1;
            const bool fits = n >= 0 && n <= (int64_t)p.max_pages << p.c.page_shift;
            if (!fits)
                bad_len = 1;
            const int pages = fits ? (int)(((int64_t)n + P - 1) >> p.c.page_shift) : 0;
            s_pages[f] = pages;
            s_fresh[f] = shared ? (n & (P - 1)) != 0 : pages;
            s_copies[f] = s_first[a] == f ? s_fresh[f] : 0;
        }
    bad = __syncthreads_or(bad);
    bad_len = __syncthreads_or(bad_len);
    Counts all{0, 0, 0};
    if (!bad && !bad_len)
        all = exclusive_sums(s_pages, s_fresh, s_copies, F, s_warp);
    const int entries = all.entries, fresh = all.fresh, pages = all.copies;
    int code = 0;
    if (bad)
        code = RSA_PLAN_BAD_REQUEST;
    else if (bad_len)
        code = RSA_PLAN_BAD_LENGTH;
    else if (start < 0 || start > p.n_free || fresh > p.n_free - start)
        code = RSA_PLAN_NO_PAGES;
    const long long g0 = (long long)blockIdx.x * kThreads + tid, gn = (long long)gridDim.x * kThreads;
    if (g0 == 0) {
        p.info[0] = code;
        p.info[1] = code || !shared ? 0 : entries - fresh;
        p.info[2] = code ? 0 : fresh;
        p.info[3] = start + (code ? 0 : fresh);
    }
    if (code)
        return;
    // (dst's lengths and rows of the table are written, src's are read: no request is in both)
    for (long long f = g0; f < F; f += gn)
        if (p.src[f] >= 0)
            p.kv_len[p.dst[f]] = p.kv_len[p.src[f]];

    // ---- table entries -------------------------------------------------------------------
    for (long long i = g0; i < entries; i += gn) {
        const int f = last_not_above(s_pages, F, (int)i), j = (int)i - s_pages[f], a = p.src[f];
        int id;
        if (shared && j < p.kv_len[a] >> p.c.page_shift) {
            id = p.block_table[a * p.table_stride + j];
            if (id >= 0 && id < p.c.n_pages)
                atomicAdd(&p.shares[id], 1);
            else
                record_bad_index(p.err, kSiteForkPage, id);
        } else {
            id = p.free_pages[start + s_fresh[f] + (shared ? 0 : j)];
        }
        p.block_table[p.dst[f] * p.table_stride + j] = id;
    }

    // ---- rows ------------------------------------------------------------------------------
    // The forks of one source copy the same pages: the first of them stands for all.
    // A warp takes up to kPiece bytes of such a page's rows of one key head, of keys or values, in
    // a layer, reads them once and writes them for every fork.
    const int lane = tid & 31, warp = tid >> 5, heads = 2 * p.c.Hkv, page_bytes = p.c.row << p.c.page_shift;
    const int pieces = (page_bytes + kPiece - 1) / kPiece;
    const long long items = (long long)pages * heads * pieces * p.c.layers;
    for (long long i = (long long)blockIdx.x * kWarps + warp; i < items; i += (long long)gridDim.x * kWarps) {
        // (layer, piece, page, head), the head fastest
        int c, slab, piece, layer;
        if (items <= UINT_MAX) {
            const unsigned q = (unsigned)i / (unsigned)heads, u = q / (unsigned)pages;
            slab = (int)((unsigned)i - q * heads), c = (int)(q - u * (unsigned)pages), layer = (int)(u / (unsigned)pieces);
            piece = (int)(u - (unsigned)layer * pieces);
        } else {
            const long long q = i / heads, u = q / pages;
            slab = (int)(i - q * heads), c = (int)(q - u * pages), layer = (int)(u / pieces);
            piece = (int)(u - (long long)layer * pieces);
        }
        const int f = last_not_above(s_copies, F, c), a = p.src[f], len = p.kv_len[a];
        const int j = shared ? len >> p.c.page_shift : c - s_copies[f];
        const int first = piece * kPiece / 16, n = min((piece + 1) * kPiece, min(P, len - (j << p.c.page_shift)) * p.c.row) / 16;
        if (first >= n)
            continue;
        const int from = p.block_table[a * p.table_stride + j];
        if (from < 0 || from >= p.c.n_pages) {
            if (lane == 0)
                record_bad_index(p.err, kSiteForkPage, from);
            continue;
        }
        char *data = p.c.data[slab & 1] + layer * p.c.layer_bytes + (int64_t)(slab >> 1) * page_bytes;
        const int64_t stride = (int64_t)p.c.Hkv * page_bytes;
        const uint4 *x = reinterpret_cast<const uint4 *>(data + from * stride);
        uint4 v[kDepth];
#pragma unroll
        for (int e = 0; e < kDepth; ++e)
            if (first + lane + 32 * e < n)
                v[e] = x[first + lane + 32 * e];
        // 32 forks at a time: each lane finds the fresh page of one
        for (int next = f, left = s_forks[a]; left > 0;) {
            int found = 0;
            __syncwarp();
            for (; found < min(left, 32); next += 32) {
                const bool mine = next + lane < F && p.src[next + lane] == a;
                const unsigned who = __ballot_sync(0xffffffffu, mine);
                const int at = found + __popc(who & ((1u << lane) - 1));
                if (mine && at < 32)
                    s_list[warp][at] = next + lane;
                found += __popc(who);
                if (found > 32) {  // the others of these 32 in the next turn
                    next = __shfl_sync(0xffffffffu, next + lane, __ffs(__ballot_sync(0xffffffffu, mine && at == 32)) - 1) - 32;
                    found = 32;
                }
            }
            __syncwarp();
            int to = -1;
            if (lane < found) {
                to = p.free_pages[start + s_fresh[s_list[warp][lane]] + (shared ? 0 : j)];
                if (to < 0 || to >= p.c.n_pages) {
                    record_bad_index(p.err, kSiteForkPage, to);
                    to = -1;
                }
            }
            for (int k = 0; k < found; ++k) {
                const int page = __shfl_sync(0xffffffffu, to, k);
                if (page < 0)
                    continue;
                uint4 *y = reinterpret_cast<uint4 *>(data + page * stride);
#pragma unroll
                for (int e = 0; e < kDepth; ++e)
                    if (first + lane + 32 * e < n)
                        y[first + lane + 32 * e] = v[e];
            }
            left -= found;
        }
    }
}

}  // namespace

cudaError_t launch_page_fork(const PageForkParams &p, cudaStream_t s)
{
    auto smem_of = [](int64_t F, int64_t R) constexpr { return (size_t)(3 * F + 3 + 2 * R + (R + 31) / 32) * 4; };
    constexpr size_t kMost = smem_of(kPageForkMost, kPagePlanMaxRequests);  // 224 KB
    const size_t smem = smem_of(p.F, p.R);
    // (always the most: the limit is the kernel's, not the call's, and another thread may launch it
    // between this one's two calls)
    if (smem > 48 * 1024 - 2048) {
        cudaError_t e = cudaFuncSetAttribute(page_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess)
            return e;
    }
    // As many warps as there may be pieces to copy, at most what the SMs hold.
    const int64_t pieces = (((int64_t)p.c.row << p.c.page_shift) + kPiece - 1) / kPiece;
    const int64_t items = (int64_t)p.F * (p.shares ? 1 : p.max_pages) * 2 * p.c.Hkv * pieces * p.c.layers;
    int64_t blocks = (items + kWarps - 1) / kWarps;
    const int64_t entries = ((int64_t)p.F * p.max_pages + kThreads - 1) / kThreads;
    blocks = blocks > entries ? blocks : entries;
    blocks = blocks < 1 ? 1 : (blocks > 304 ? 304 : blocks);
    return launch_early(page_fork_kernel, dim3((unsigned)blocks), kThreads, smem, s, 1, p);
}

}  // namespace rsa
