// Pages that requests give back, onto the list of free pages.
//
// Which pages become free is a set, and the set does not depend on the order in which
// entries are looked at: a bitmap of all pages in shared memory takes it, and reading
// the bitmap in order gives the pages ascending.  Users of a page are counted down by
// atomics; of those that count one down in the same call exactly one finds 0.
// One launch of one cluster: each CTA sums up all requests' entries (8 bytes a request,
// from L2), looks at its share of the entries, and holds its share of the bitmap, into
// which the others write through distributed shared memory.  A bit is one of 2^23 pages
// in 8 CTAs with 128 KB each.  Latency bounds it: lengths, table entries, counts and
// three cluster barriers one after the other.
#include <cooperative_groups.h>

#include "rsa_internal.h"

namespace rsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostCtas = 8;
constexpr int kBatch = 4;  // entries that a thread has in flight

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

// This thread's exclusive sum of `mine` over the block, and the total.
template <int kThreads>
__device__ __forceinline__ long long block_sum(long long mine, long long *s_warp, long long *total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    long long before = x - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp)
            before += s_warp[w];
        all += s_warp[w];
    }
    __syncthreads();
    *total = all;
    return before;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) page_free_kernel(const __grid_constant__ PageFreeParams p, const int words)
{
    extern __shared__ int smem[];
    unsigned *s_bits = reinterpret_cast<unsigned *>(smem);  // [words] this CTA's part of the bitmap
    int *s_before = smem + words;                           // [R + 1] entries before each request's
    __shared__ long long s_warp[kThreads / 32];
    __shared__ int s_freed[kMostCtas];  // pages that each CTA's part holds
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int R = p.R, P = 1 << p.page_shift;

    for (int i = tid; i < words; i += kThreads)
        s_bits[i] = 0;
    // ---- the requests' entries -----------------------------------------------------------
    const long long start = *p.free_start;
    int bad = 0;
    for (int r = tid; r < R; r += kThreads) {
        const int n = p.kv_len[r], k = p.keep_len[r];
        const bool fits = k >= 0 && k <= n && n <= (int64_t)p.max_pages << p.page_shift;
        bad |= !fits;
        s_before[r] = fits ? (int)((((int64_t)n + P - 1) >> p.page_shift) - (((int64_t)k + P - 1) >> p.page_shift)) : 0;
    }
    bad = __syncthreads_or(bad);
    const int per = (R + kThreads - 1) / kThreads | 1, r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long mine = 0, entries;
    for (int r = r0; r < r1; ++r)
        mine += s_before[r];
    long long at = block_sum<kThreads>(mine, s_warp, &entries);
    for (int r = r0; r < r1; ++r) {
        const int n = s_before[r];
        s_before[r] = (int)at;
        at += n;
    }
    if (tid == 0)
        s_before[R] = (int)entries;
    if (bad || entries > 0x7fffffffLL) {  // (the same in every CTA)
        if (rank == 0 && tid == 0) {
            p.info[0] = RSA_PLAN_BAD_LENGTH;
            p.info[1] = p.info[2] = 0;
            p.info[3] = start;
        }
        return;
    }
    cluster.sync();  // every part of the bitmap is empty

    // ---- what becomes free ---------------------------------------------------------------
    const int step = ctas * kThreads;
    auto id_of = [&](long long i) {
        const int r = last_not_above(s_before, R, (int)i);
        const int first = (int)(((int64_t)p.keep_len[r] + P - 1) >> p.page_shift);
        return p.block_table[r * p.table_stride + first + ((int)i - s_before[r])];
    };
    for (long long i0 = rank * kThreads + tid; i0 < entries; i0 += (long long)step * kBatch) {
        int id[kBatch], left[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const long long i = i0 + (long long)e * step;
            id[e] = i < entries ? id_of(i) : -1;
            if (i < entries && (id[e] < 0 || id[e] >= p.n_pages)) {
                record_bad_index(p.err, kSiteFreePage, id[e]);
                id[e] = -1;
            }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            left[e] = id[e] >= 0 && p.shares ? atomicSub(&p.shares[id[e]], 1) : 0;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            if (id[e] < 0)
                continue;
            bool twice = left[e] < 0;
            if (left[e] == 0) {
                const int w = id[e] >> 5, owner = w / words;
                unsigned *bits = cluster.map_shared_rank(s_bits, owner);
                twice = atomicOr(&bits[w - owner * words], 1u << (id[e] & 31)) >> (id[e] & 31) & 1;
            }
            if (twice)
                record_bad_index(p.err, kSiteFreeTwice, id[e]);
        }
    }
    cluster.sync();  // the bitmap is complete

    // ---- where they go -------------------------------------------------------------------
    const int wper = (words + kThreads - 1) / kThreads, w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
    int count = 0;
    for (int w = w0; w < w1; ++w)
        count += __popc(s_bits[w]);
    long long in_cta, before = block_sum<kThreads>(count, s_warp, &in_cta);
    if (tid < ctas)
        *cluster.map_shared_rank(&s_freed[rank], tid) = (int)in_cta;
    cluster.sync();
    long long freed = 0;
    for (int c = 0; c < ctas; ++c) {
        if (c < rank)
            before += s_freed[c];
        freed += s_freed[c];
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
        for (long long i = rank * kThreads + tid; p.shares && i < entries; i += step) {
            const int id = id_of(i);
            if (id >= 0 && id < p.n_pages)
                atomicAdd(&p.shares[id], 1);
        }
        return;
    }
    long long to = start - freed + before;
    for (int w = w0; w < w1; ++w)
        for (unsigned left = s_bits[w]; left; left &= left - 1) {
            const int id = ((rank * words + w) << 5) + __ffs(left) - 1;
            p.free_pages[to++] = id;
            if (p.shares)
                p.shares[id] = 0;
        }
}

template <int kThreads>
cudaError_t launch(const PageFreeParams &p, int ctas, cudaStream_t s)
{
    const int64_t words = ((p.n_pages + 31) / 32 + ctas - 1) / ctas;
    const size_t smem = ((size_t)words + p.R + 1) * 4;
    if (smem > 48 * 1024 - 1024) {
        cudaError_t e = cudaFuncSetAttribute(page_free_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = (unsigned)ctas;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_free_kernel<kThreads>, p, (int)words);
}

}  // namespace

cudaError_t launch_page_free(const PageFreeParams &p, cudaStream_t s)
{
    // One CTA where all its threads have little to do and the bitmap fits; else a cluster.
    if ((int64_t)p.R * p.max_pages <= 4096 && p.n_pages <= 1 << 18)
        return launch<256>(p, 1, s);
    return launch<1024>(p, kMostCtas, s);
}

}  // namespace rsa
