// Pages that requests give back, onto the list of free pages.
//
// Which pages become free is a set, and the set does not depend on the order in which
// entries are looked at: a bitmap of all pages in shared memory takes it, and reading
// the bitmap in order gives the pages ascending.  Users of a page are counted down by
// atomics; of those that count one down in the same call exactly one finds 0.
// One launch of one cluster.  Every CTA sums up all requests' entries (8 bytes a request, from L2) and marks the pages of its share of the
// entries; then each reads a part of the bitmap.  Where a bitmap of all pages fits a CTA's
// shared memory (780000 pages), each marks one of its own, and the parts are put
// together through distributed shared memory; else each CTA holds a part and the others
// mark in it, which the network between the SMs takes one by one (84000 entries 13 us
// instead of 1).  A thread takes consecutive entries, so that it searches their request
// once (each by itself: 9 us more).  Latency bounds it: lengths, table entries, counts and
// the cluster's barriers one after the other.
#include <cooperative_groups.h>

#include "ptx_sm103.cuh"
#include "rsa_internal.h"

namespace rsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;  // of the cluster

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

// The sum of `mine` over the threads before this one, and over all.
template <int kThreads>
__device__ __forceinline__ int block_sum(int mine, int *s_warp, int *total)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto scan = [&](int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        return x;
    };
    const int x = scan(mine);
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    const int w = scan(lane < kWarps ? s_warp[lane] : 0);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
    __syncthreads();  // s_warp is written again
    return (warp ? before : 0) + x - mine;
}

// Consecutive entries, each the id of a page given back.
struct Entries {
    const PageFreeParams &p;
    const int *before;  // [R + 1] entries before each request's
    const int *kept;    // [R] the first entry that each request gives back, or NULL: worked out again
    int r, end;         // the request of the entry last asked for, and where its entries end
    const int32_t *row;

    __device__ __forceinline__ Entries(const PageFreeParams &p_, const int *before_, const int *kept_, int i)
        : p(p_), before(before_), kept(kept_)
    {
        r = last_not_above(before, p.R, i);
        enter();
    }
    __device__ __forceinline__ void enter()
    {
        const int first = kept ? kept[r] : (int)(((int64_t)p.keep_len[r] + (1 << p.page_shift) - 1) >> p.page_shift);
        row = p.block_table + r * p.table_stride + first - before[r];
        end = before[r + 1];
    }
    // Where entry i is, not before the last one and less than all.
    __device__ __forceinline__ const int32_t *at(int i)
    {
        if (i >= end) {
            do
                ++r;
            while (i >= before[r + 1]);
            enter();
        }
        return row + i;
    }
};

// kWhole: every CTA has a bitmap of all pages (kCtas parts of `words` words), else its part.
// kBatch: lengths or entries that a thread has in flight.  spare: words of shared memory behind
// all else.
template <int kThreads, bool kWhole, int kBatch>
__global__ void __launch_bounds__(kThreads) page_free_kernel(const __grid_constant__ PageFreeParams p, const int words, const int spare)
{
    extern __shared__ int smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank();
    const int held = kWhole ? words * kCtas : words;
    unsigned *s_bits = reinterpret_cast<unsigned *>(smem);  // [held]
    int *s_before = smem + held;                            // [R + 1]
    int *s_kept = kWhole ? s_before + p.R + 1 : nullptr;    // [R]
    __shared__ int s_warp[32];
    __shared__ int s_freed[kCtas], s_marked[kCtas];  // pages in each CTA's part; entries that each has marked
    const int R = p.R, P = 1 << p.page_shift;

    if (kWhole)
        ptx::cluster_begin_arrive();
    for (int i = tid; i < held; i += kThreads)
        s_bits[i] = 0;
    // ---- the requests' entries -----------------------------------------------------------
    ptx::wait_for_launch_before();
    const long long start = *p.free_start;
    int bad = 0;
    for (int rb = tid; rb < R; rb += kThreads * kBatch) {
        int ns[kBatch], ks[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int r = rb + e * kThreads;
            ns[e] = r < R ? p.kv_len[r] : 0;
            ks[e] = r < R ? p.keep_len[r] : 0;
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int r = rb + e * kThreads;
            const int64_t n = ns[e], k = ks[e];
            const bool fits = k >= 0 && k <= n && n <= (int64_t)p.max_pages << p.page_shift;
            bad |= !fits;
            const int kept = (int)((k + P - 1) >> p.page_shift);
            if (r < R)
                s_before[r] = fits ? (int)((n + P - 1) >> p.page_shift) - kept : 0;
            if (kWhole && r < R)
                s_kept[r] = kept;
        }
    }
    bad = __syncthreads_or(bad);
    // (a row has at most max_pages entries, and all rows 2^30)
    const int per = (R + kThreads - 1) / kThreads | 1, r0 = min(R, tid * per), r1 = min(R, r0 + per);
    int mine = 0, entries;
    for (int r = r0; r < r1; ++r)
        mine += s_before[r];
    int sum = block_sum<kThreads>(mine, s_warp, &entries);
    for (int r = r0; r < r1; ++r) {
        const int n = s_before[r];
        s_before[r] = sum;
        sum += n;
    }
    if (tid == 0)
        s_before[R] = entries;
    if (kWhole)
        ptx::cluster_begin_wait();
    if (bad) {  // (the same in every CTA)
        if (rank == 0 && tid == 0) {
            p.info[0] = RSA_PLAN_BAD_LENGTH;
            p.info[1] = p.info[2] = 0;
            p.info[3] = start;
        }
        return;
    }
    if (kWhole)
        __syncthreads();
    else
        cluster.sync();  // every part of the bitmap is empty

    // ---- what becomes free ---------------------------------------------------------------
    const int run = (entries + kCtas * kThreads - 1) / (kCtas * kThreads);
    const int first = min((int64_t)entries, (int64_t)(rank * kThreads + tid) * run), last = min(entries - first, run) + first;
    int marked = 0;
    if (first < last) {
        Entries list(p, s_before, s_kept, first);
        for (int i0 = first; i0 < last; i0 += kBatch) {
            const int32_t *at[kBatch];
            int id[kBatch], left[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                at[e] = i0 + e < last ? list.at(i0 + e) : nullptr;
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                id[e] = at[e] ? *at[e] : 0;
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                left[e] = 1;
                if (!at[e])
                    continue;
                if (id[e] < 0 || id[e] >= p.n_pages)
                    record_bad_index(p.err, kSiteFreePage, id[e]);
                else
                    left[e] = p.shares ? atomicSub(&p.shares[id[e]], 1) : 0;
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                if (left[e] == 0) {
                    const int w = id[e] >> 5, owner = kWhole ? rank : w / words;
                    unsigned *bits = kWhole ? s_bits : cluster.map_shared_rank(s_bits, owner) - owner * words;
                    atomicOr(bits + w, 1u << (id[e] & 31));
                    ++marked;
                } else if (left[e] < 0) {
                    record_bad_index(p.err, kSiteFreeTwice, id[e]);
                }
            }
        }
    }
    int in_cta;
    block_sum<kThreads>(marked, s_warp, &in_cta);
    if (tid < kCtas)
        *cluster.map_shared_rank(&s_marked[rank], tid) = in_cta;
    cluster.sync();  // the bitmap is complete

    // ---- where they go -------------------------------------------------------------------
    unsigned *part = kWhole ? s_bits + rank * words : s_bits;  // (word w of it is word rank * words + w of all)
    const int wper = (words + kThreads - 1) / kThreads, w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
    int count = 0;
    for (int w = w0; w < w1; ++w) {
        if (kWhole) {
            unsigned x = 0;
#pragma unroll
            for (int c = 0; c < kCtas; ++c)
                x |= cluster.map_shared_rank(part, c)[w];
            part[w] = x;  // (no other CTA reads this part)
        }
        count += __popc(part[w]);
    }
    const int mine0 = block_sum<kThreads>(count, s_warp, &in_cta);  // this thread's first page among the CTA's
    if (tid < kCtas)
        *cluster.map_shared_rank(&s_freed[rank], tid) = in_cta;
    cluster.sync();
    int freed = 0, marks = 0, before = 0;
    for (int c = 0; c < kCtas; ++c) {
        if (c < rank)
            before += s_freed[c];
        freed += s_freed[c];
        marks += s_marked[c];
    }
    const bool ok = start >= freed && start <= p.n_free;
    if (rank == 0 && tid == 0) {
        p.info[0] = ok ? RSA_PLAN_OK : RSA_PLAN_NO_ROOM;
        p.info[1] = ok ? freed : 0;
        p.info[2] = ok ? entries : 0;
        p.info[3] = ok ? start - freed : start;
    }
    if (!ok) {
        // users are counted up again
        if (p.shares && first < last) {
            Entries list(p, s_before, s_kept, first);
            for (int i = first; i < last; ++i) {
                const int id = *list.at(i);
                if (id >= 0 && id < p.n_pages)
                    atomicAdd(&p.shares[id], 1);
            }
        }
        return;
    }
    int32_t *to = p.free_pages + (start - freed) + before;
    // Each thread lists its words' pages; in shared memory first, where they fit what is no longer
    // needed, so that they are written side by side (61000 pages 15.0 -> 12.2 us, now 11.3): the other parts
    // of the bitmap, the sums and what lies behind them.
    const bool staged = kWhole && marks == freed && in_cta <= held - words + 2 * R + 1 + spare;
    auto stage = [&](int i) -> int & { return smem[i < rank * words ? i : i + words]; };
    for (int w = w0, at = mine0; w < w1; ++w)
        for (unsigned left = part[w]; left; left &= left - 1, ++at) {
            const int id = ((rank * words + w) << 5) + __ffs(left) - 1;
            if (staged)
                stage(at) = id;
            else
                to[at] = id;
            if (p.shares)
                p.shares[id] = 0;
        }
    if (staged) {
        __syncthreads();
        for (int i = tid; i < in_cta; i += kThreads)
            to[i] = stage(i);
    }
    if (marks == freed)
        return;
    // (only without shares) Some page was marked twice: the entries take their marks back, and
    // one that finds none is an entry too many.
    cluster.sync();
    if (first < last) {
        Entries list(p, s_before, s_kept, first);
        for (int i = first; i < last; ++i) {
            const int id = *list.at(i);
            if (id < 0 || id >= p.n_pages)
                continue;
            const int w = id >> 5, owner = w / words;
            unsigned *bits = cluster.map_shared_rank(s_bits, owner) - (kWhole ? 0 : owner * words);
            if (!(atomicAnd(bits + w, ~(1u << (id & 31))) >> (id & 31) & 1))
                record_bad_index(p.err, kSiteFreeTwice, id);
        }
    }
    cluster.sync();  // no CTA ends while others look at its part
}

constexpr int64_t kMostWhole = 780000;  // pages: 98 KB of bitmap beside 128 KB of sums and kept pages

// Words of a part of the bitmap, and bytes of shared memory without the spare ones.
constexpr int64_t words_of(int64_t n_pages) { return ((n_pages + 31) / 32 + kCtas - 1) / kCtas; }
template <bool kWhole>
constexpr size_t smem_of(int64_t n_pages, int64_t R)
{
    return (size_t)(kWhole ? words_of(n_pages) * kCtas + 2 * R + 1 : words_of(n_pages) + R + 1) * 4;
}

template <int kThreads, bool kWhole, int kBatch>
cudaError_t launch(const PageFreeParams &p, cudaStream_t s)
{
    constexpr size_t kMost = smem_of<kWhole>(kWhole ? kMostWhole : kPageFreeMaxPages, kPagePlanMaxRequests);
    constexpr size_t kSpare = 8 * 1024, kSpareUpTo = 200 * 1024;
    static_assert(kMost <= 226 * 1024 && (!kWhole || kSpareUpTo + kSpare <= kMost), "shared memory");
    const size_t used = smem_of<kWhole>(p.n_pages, p.R);
    const size_t spare = kWhole && used <= kSpareUpTo ? kSpare : 0, smem = used + spare;
    // (always the most: the limit is the kernel's, not the call's, and another thread may launch it
    // between this one's two calls)
    if (smem > 48 * 1024 - 1024) {
        cudaError_t e =
            cudaFuncSetAttribute(page_free_kernel<kThreads, kWhole, kBatch>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
        if (e != cudaSuccess)
            return e;
    }
    return launch_early(page_free_kernel<kThreads, kWhole, kBatch>, dim3(kCtas), kThreads, smem, s, kCtas, p, (int)words_of(p.n_pages),
                        (int)spare / 4);
}

}  // namespace

cudaError_t launch_page_free(const PageFreeParams &p, cudaStream_t s)
{
    if (p.n_pages > kMostWhole)
        return launch<1024, false, 4>(p, s);
    // Fewer threads where there is less to do, for shorter barriers and scans (300 requests of 75000
    // entries in all, a tenth given back, 6.2 us against 6.9; 8 requests 5.0 against 5.9, now 4.2).  One CTA
    // gains 0.1 us where next to nothing is given back and loses 4 where 2000 entries are.
    if ((int64_t)p.R * p.max_pages <= 131072)
        return launch<256, true, 4>(p, s);
    return launch<1024, true, 4>(p, s);
}

}  // namespace rsa
