// Forks of requests over a paged cache: full pages are shared and counted, a partial
// last page (without counts: every page) is copied to a fresh one, in all layers.
//
// One launch and no traffic between blocks, as for the step's plan: every block reads the
// forks and their lengths, checks them and sums up the fresh pages before each, and then
// does its share of the table entries and of the rows.  Nothing that any block reads
// is written by another: sources and destinations are different rows, and a copy's
// destination comes from free_pages.
// A page's rows of one key head lie side by side: a warp copies them, 16 bytes a lane.
// The copies go layer by layer, so that the forks of one request read its page
// from L2 after the first.
#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kDepth = 8;  // 16-byte pieces that a lane has in flight

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

// Exclusive sums of a[0..n) in place, a[n] the total (64 bits: also returned), by the whole block.
__device__ __forceinline__ long long exclusive_sums(int *a, int n, long long *s_warp)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (n + kThreads - 1) / kThreads | 1;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    long long mine = 0;
    for (int i = i0; i < i1; ++i)
        mine += a[i];
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
    long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp)
            before += s_warp[w];
        total += s_warp[w];
    }
    for (int i = i0; i < i1; ++i) {
        const int v = a[i];
        a[i] = (int)before;  // (wraps only where the forks are refused)
        before += v;
    }
    if (tid == 0)
        a[n] = (int)total;
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(kThreads) page_fork_kernel(const __grid_constant__ PageForkParams p)
{
    extern __shared__ int smem[];
    int *s_len = smem;                 // [F]
    int *s_pages = s_len + p.F;        // [F + 1] table entries before each fork
    int *s_fresh = s_pages + p.F + 1;  // [F + 1] fresh pages before each fork
    unsigned *s_used = reinterpret_cast<unsigned *>(s_fresh + p.F + 1);  // a bit for each request: it is in dst
    __shared__ long long s_warp[kWarps];
    const int tid = threadIdx.x, P = 1 << p.c.page_shift, F = p.F;
    const bool shared = p.shares != nullptr;

    // ---- the forks, and what makes them impossible ---------------------------------------
    for (int i = tid; i < (p.R + 31) / 32; i += kThreads)
        s_used[i] = 0;
    __syncthreads();
    int bad = 0;
    for (int f = tid; f < F; f += kThreads) {
        const int a = p.src[f], b = p.dst[f];
        if (a < 0 || a >= p.R || b < 0 || b >= p.R || (atomicOr(&s_used[b >> 5], 1u << (b & 31)) >> (b & 31) & 1))
            bad = 1;
    }
    bad = __syncthreads_or(bad);
    int bad_len = 0;
    for (int f = tid; f < F && !bad; f += kThreads) {
        const int a = p.src[f];
        if (s_used[a >> 5] >> (a & 31) & 1) {
            bad = 1;
            break;
        }
        const int n = p.kv_len[a];
        if (n < 0 || n > (int64_t)p.max_pages << p.c.page_shift)
            bad_len = 1;
        const int pages = bad_len ? 0 : (int)(((int64_t)n + P - 1) >> p.c.page_shift);
        s_len[f] = n;
        s_pages[f] = pages;
        s_fresh[f] = shared ? (n & (P - 1)) != 0 : pages;
    }
    bad = __syncthreads_or(bad);
    bad_len = __syncthreads_or(bad_len);
    const long long start = p.free_start ? *p.free_start : 0;
    long long entries = 0, fresh = 0;
    if (!bad && !bad_len) {
        entries = exclusive_sums(s_pages, F, s_warp);
        fresh = exclusive_sums(s_fresh, F, s_warp);
    }
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
    for (long long f = g0; f < F; f += gn)
        p.kv_len[p.dst[f]] = s_len[f];

    // ---- table entries -------------------------------------------------------------------
    for (long long i = g0; i < entries; i += gn) {
        const int f = last_not_above(s_pages, F, (int)i), j = (int)i - s_pages[f], full = s_len[f] >> p.c.page_shift;
        int id;
        if (shared && j < full) {
            id = p.block_table[(int64_t)p.src[f] * p.table_stride + j];
            if (id >= 0 && id < p.c.n_pages)
                atomicAdd(&p.shares[id], 1);
            else
                record_bad_index(p.err, kSiteForkPage, id);
        } else {
            id = p.free_pages[start + s_fresh[f] + (shared ? 0 : j)];
        }
        p.block_table[(int64_t)p.dst[f] * p.table_stride + j] = id;
    }

    // ---- rows ------------------------------------------------------------------------------
    // A warp takes one copied page's rows of one key head, of keys or values, in a layer.
    const int lane = tid & 31;
    const long long heads = 2ll * p.c.Hkv, items = fresh * heads * p.c.layers;
    for (long long i = (long long)blockIdx.x * kWarps + (tid >> 5); i < items; i += (long long)gridDim.x * kWarps) {
        const int layer = (int)(i / (fresh * heads));
        const long long in_layer = i - layer * (fresh * heads);
        const int c = (int)(in_layer / heads), slab = (int)(in_layer - c * heads), head = slab >> 1;
        const int f = last_not_above(s_fresh, F, c);
        const int j = shared ? s_len[f] >> p.c.page_shift : c - s_fresh[f];
        const int rows = min(P, s_len[f] - (j << p.c.page_shift));
        const int from = p.block_table[(int64_t)p.src[f] * p.table_stride + j], to = p.free_pages[start + c];
        if (from < 0 || from >= p.c.n_pages || to < 0 || to >= p.c.n_pages) {
            if (lane == 0)
                record_bad_index(p.err, kSiteForkPage, from < 0 || from >= p.c.n_pages ? from : to);
            continue;
        }
        char *data = p.c.data[slab & 1] + layer * p.c.layer_bytes;
        const int64_t bytes = (int64_t)p.c.row << p.c.page_shift;
        const uint4 *x = reinterpret_cast<const uint4 *>(data + ((int64_t)from * p.c.Hkv + head) * bytes);
        uint4 *y = reinterpret_cast<uint4 *>(data + ((int64_t)to * p.c.Hkv + head) * bytes);
        const int n = rows * (p.c.row / 16);
        for (int k0 = lane; k0 < n; k0 += 32 * kDepth) {
            uint4 v[kDepth];
#pragma unroll
            for (int e = 0; e < kDepth; ++e)
                if (k0 + 32 * e < n)
                    v[e] = x[k0 + 32 * e];
#pragma unroll
            for (int e = 0; e < kDepth; ++e)
                if (k0 + 32 * e < n)
                    y[k0 + 32 * e] = v[e];
        }
    }
}

}  // namespace

cudaError_t launch_page_fork(const PageForkParams &p, cudaStream_t s)
{
    const size_t smem = (3ull * p.F + 2) * 4 + (p.R + 31) / 32 * 4;
    if (smem > 48 * 1024 - 1024) {
        cudaError_t e = cudaFuncSetAttribute(page_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    // As many warps as there are rows to copy for them, at most what the SMs hold.
    const int64_t items = (int64_t)p.F * (p.shares ? 1 : p.max_pages) * 2 * p.c.Hkv * p.c.layers;
    int64_t blocks = (items + kWarps - 1) / kWarps;
    const int64_t entries = ((int64_t)p.F * p.max_pages + kThreads - 1) / kThreads;
    blocks = blocks > entries ? blocks : entries;
    blocks = blocks < 1 ? 1 : (blocks > 608 ? 608 : blocks);
    page_fork_kernel<<<(unsigned)blocks, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rsa
