// The plan of one step over a paged KV cache, made on the GPU from the
// requests' lengths: fresh pages appended to the block tables, and for every
// new token its cache slot and its position.
//
//   have_r = ceil(c_r / P), need_r = ceil((c_r + n_r) / P) - have_r
//   fresh page i of request r = free_pages[start + sum_{s<r} need_s + i]
//   token i of request r (row cu_r + i): pos = c_r + i,
//     slot = page(r, pos / P) * P + pos mod P
//
// One launch and no traffic between blocks: every block reads all lengths
// (8 bytes a request, from L2 after the first block), scans them in shared
// memory and then does its share of the tokens, pages and requests.  A token
// finds its page in the old part of its table or, past that, straight in
// free_pages, so no block reads a table entry that another one writes.  The
// work is a few bytes a token: the launch and the scan's latency bound it at
// any size a server sees (8 requests 6.3 us on the GPU, 4000 requests with 0.42
// million rows 13.1 us, of which the 6.8 MB would take 1).
#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kLoads = 8;            // lengths a thread has in flight (one at a time, 4000 requests took 5 us to read)
constexpr int kTokensPerThread = 4;  // one search of the request serves four consecutive rows

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

template <int kThreads>
__global__ void __launch_bounds__(kThreads) page_plan_kernel(const __grid_constant__ PagePlanParams p)
{
    constexpr int kWarps = kThreads / 32;
    extern __shared__ int smem[];
    int *s_cu = smem;               // [R + 1] first row of each request
    int *s_pg = s_cu + (p.R + 1);   // [R + 1] fresh pages before each request
    int *s_c = s_pg + (p.R + 1);    // [R] cached lengths
    __shared__ long long s_wt[kWarps], s_wp[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = p.R, P = 1 << p.page_shift;

    // ---- lengths, and what makes the whole step impossible --------------------
    const long long start = p.free_start ? *p.free_start : 0;
    int bad_len = 0, bad_row = 0;
    for (int rb = tid; rb < R; rb += kThreads * kLoads) {
        int cs[kLoads], ns[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = rb + i * kThreads;
            cs[i] = r < R ? p.cached_len[r] : 0;
            ns[i] = r < R ? p.new_len[r] : 0;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = rb + i * kThreads;
            const long long c = cs[i], n = ns[i];
            long long need = 0;
            if (c < 0 || n < 0) {
                bad_len = 1;
            } else {
                const long long all = (c + n + P - 1) >> p.page_shift;
                need = all - ((c + P - 1) >> p.page_shift);
                if (all > p.max_pages)
                    bad_row = 1;
            }
            if (r < R) {
                s_cu[r] = (int)max(n, 0ll);
                s_pg[r] = (int)need;
                s_c[r] = cs[i];
            }
        }
    }
    bad_len = __syncthreads_or(bad_len);
    bad_row = __syncthreads_or(bad_row);

    // ---- exclusive sums over the requests: a run per thread, then a block scan --
    // Sums are 64-bit until they are known to fit; runs are of odd length so that
    // the threads of a warp fall into different banks.
    const int per = (R + kThreads - 1) / kThreads | 1;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long t = 0, g = 0;
    for (int r = r0; r < r1; ++r) {
        t += s_cu[r];
        g += s_pg[r];
    }
    long long ti = t, gi = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, ti, o), b = __shfl_up_sync(0xffffffffu, gi, o);
        if (lane >= o) {
            ti += a;
            gi += b;
        }
    }
    if (lane == 31) {
        s_wt[warp] = ti;
        s_wp[warp] = gi;
    }
    __syncthreads();
    long long tokens = 0, pages = 0, tb = ti - t, gb = gi - g;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            tb += s_wt[w];
            gb += s_wp[w];
        }
        tokens += s_wt[w];
        pages += s_wp[w];
    }
    for (int r = r0; r < r1; ++r) {
        const int n = s_cu[r], need = s_pg[r];
        s_cu[r] = (int)tb;  // (wraps only where the step is refused below)
        s_pg[r] = (int)gb;
        tb += n;
        gb += need;
    }
    if (tid == 0) {
        s_cu[R] = (int)tokens;
        s_pg[R] = (int)pages;
    }
    __syncthreads();
    int code = 0;
    if (bad_len)
        code = RSA_PLAN_BAD_LENGTH;
    else if (bad_row)
        code = RSA_PLAN_TABLE_FULL;
    else if (start < 0 || start > p.n_free || pages > p.n_free - start)
        code = RSA_PLAN_NO_PAGES;
    else if (tokens > p.max_tokens)
        code = RSA_PLAN_TOO_MANY_TOKENS;
    const bool ok = code == 0;

    const long long g0 = (long long)blockIdx.x * kThreads + tid, gn = (long long)gridDim.x * kThreads;
    if (g0 == 0) {
        p.info[0] = code;
        p.info[1] = ok ? tokens : 0;
        p.info[2] = ok ? pages : 0;
        p.info[3] = start + (ok ? pages : 0);
    }
    // ---- requests ---------------------------------------------------------------
    for (long long r = g0; r <= R; r += gn) {
        p.cu_new[r] = ok ? s_cu[r] : 0;
        if (r < R)
            p.kv_len[r] = s_c[r] + (ok ? s_cu[r + 1] - s_cu[r] : 0);
    }
    // ---- fresh pages --------------------------------------------------------------
    if (ok)
        for (long long i = g0; i < pages; i += gn) {
            const int r = last_not_above(s_pg, R, (int)i);
            const long long have = ((long long)s_c[r] + P - 1) >> p.page_shift;
            p.block_table[r * p.table_stride + have + (i - s_pg[r])] = p.free_pages[start + i];
        }
    // ---- tokens -------------------------------------------------------------------
    for (long long i0 = g0 * kTokensPerThread; i0 < p.max_tokens; i0 += gn * kTokensPerThread) {
        // First where each row's page id is, then all the ids at once.
        int r = 0;
        long long at[kTokensPerThread], slot[kTokensPerThread], pos[kTokensPerThread];
        const int32_t *from[kTokensPerThread];
#pragma unroll
        for (int k = 0; k < kTokensPerThread; ++k) {
            const long long i = i0 + k;
            from[k] = nullptr;
            at[k] = 0;
            if (!ok || i >= tokens)
                continue;
            // (requests without a new token share their successor's first row: the last
            // of them is the one that owns it)
            if (k == 0)
                r = last_not_above(s_cu, R, (int)i);
            else if (i >= s_cu[r + 1])
                r = i < s_cu[min(r + 2, R)] ? r + 1 : last_not_above(s_cu, R, (int)i);
            at[k] = s_c[r] + (i - s_cu[r]);
            const long long j = at[k] >> p.page_shift, have = ((long long)s_c[r] + P - 1) >> p.page_shift;
            from[k] = j < have ? p.block_table + r * p.table_stride + j : p.free_pages + start + s_pg[r] + (j - have);
        }
        int page[kTokensPerThread];
#pragma unroll
        for (int k = 0; k < kTokensPerThread; ++k)
            page[k] = from[k] ? *from[k] : 0;
#pragma unroll
        for (int k = 0; k < kTokensPerThread; ++k) {
            slot[k] = -1;
            pos[k] = from[k] ? p.pos0 + at[k] : 0;
            if (from[k] && page[k] >= 0 && page[k] < p.n_pages)
                slot[k] = ((long long)page[k] << p.page_shift) + (at[k] & (P - 1));
            else if (from[k])
                record_bad_index(p.err, kSitePlanPage, page[k]);
        }
        if (i0 + kTokensPerThread <= p.max_tokens) {
#pragma unroll
            for (int k = 0; k < kTokensPerThread; k += 2) {
                *reinterpret_cast<longlong2 *>(p.slot_map + i0 + k) = make_longlong2(slot[k], slot[k + 1]);
                *reinterpret_cast<longlong2 *>(p.positions + i0 + k) = make_longlong2(pos[k], pos[k + 1]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTokensPerThread; ++k)
                if (i0 + k < p.max_tokens) {
                    p.slot_map[i0 + k] = slot[k];
                    p.positions[i0 + k] = pos[k];
                }
        }
    }
}

template <int kThreads>
cudaError_t launch(const PagePlanParams &p, int most, cudaStream_t s)
{
    const size_t smem = (size_t)(p.R + 1) * 12;
    if (smem > 48 * 1024 - 1024) {
        cudaError_t e = cudaFuncSetAttribute(page_plan_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)((kPagePlanMaxRequests + 1) * 12));
        if (e != cudaSuccess)
            return e;
    }
    // Enough blocks for one pass over the tokens, at most `most`: every block pays the scan.
    const int64_t work = (p.max_tokens + kTokensPerThread - 1) / kTokensPerThread;
    int64_t blocks = ((work > p.R ? work : p.R) + kThreads - 1) / kThreads;
    blocks = blocks < 1 ? 1 : (blocks > most ? most : blocks);
    page_plan_kernel<kThreads><<<(unsigned)blocks, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Many requests: a block on each of 152 SMs, wide enough to scan them (16000 requests 16.4 us;
// with two on each 22.5, with 256 threads 28.8).  Else narrower blocks, which wait less
// for one another: 1000 requests 8.2 us instead of 10.2.
cudaError_t launch_page_plan(const PagePlanParams &p, cudaStream_t s)
{
    return p.R > 2048 ? launch<512>(p, 152, s) : launch<256>(p, 304, s);
}

}  // namespace rsa
