// Positions and ancestor masks of drafted tokens, from their parents.
//
//   A_i = {i} + A_parent(i),  depth_i = |A_i| - 1,  pos_i = pos0 + cached + depth_i
//
// A thread takes a row and walks up its ancestors, whose indices descend, so that it
// finishes one word of the mask after the other and holds only one.  The parents
// lie in shared memory, those of the block's rows and of as many rows before them as
// a mask has bits.  A row's request comes from a 32-way search of cu_new by its warp.
// The work is a few bytes a token: the launch, two or three dependent reads and one
// shared-memory access for each generation of the deepest tree bound it.
#include <climits>

#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 128;

// The last request whose first row is at most `row` (requests without rows share
// their successor's), for the whole warp; -1 before the first.
__device__ __forceinline__ int request_of(const TreePlanParams &p, int64_t row)
{
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = p.R;
    for (bool first = true; first || n > 1; first = false) {
        const int64_t step = (n + 31) / 32;
        const bool below = lane * step < n && p.cu_new[lo + lane * step] <= row;
        const unsigned vote = __ballot_sync(0xffffffffu, below);
        if (!vote)
            return -1;
        const int k = 31 - __clz(vote);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return (int)lo;
}

__global__ void __launch_bounds__(kThreads) tree_plan_kernel(const __grid_constant__ TreePlanParams p)
{
    extern __shared__ int s_parent[];  // of rows [first, row0 + kThreads)
    const int tid = threadIdx.x, lane = tid & 31, most = 32 * p.words;
    const int64_t row0 = (int64_t)blockIdx.x * kThreads, row = row0 + tid;
    const int64_t first = max((int64_t)0, row0 - (most - 1));
    for (int64_t t = first + tid; t < min(p.T, row0 + kThreads); t += kThreads)
        s_parent[t - first] = p.parent[t];

    // ---- the row's request: the warp's first row's, or one after it --------------------
    const int64_t rows = min((int64_t)max(p.cu_new[p.R], 0), p.T);
    if (row == 0 && p.cu_new[p.R] != rows)
        record_bad_index(p.err, kSiteTreeRows, p.cu_new[p.R]);
    for (int64_t i = row; i < p.R; i += (int64_t)gridDim.x * kThreads)
        if (p.cu_new[i + 1] < p.cu_new[i])
            record_bad_index(p.err, kSiteTreeRows, p.cu_new[i + 1]);
    const int64_t warp_row = row0 + (tid & ~31);
    int r = -1;
    if (warp_row < rows) {
        r = request_of(p, warp_row);
        // (the requests that begin within the warp's rows; more than 31, those of one or
        // no row among them, in several turns)
        for (int from = r + 1;; from += 32) {
            const int begin = from + lane < p.R ? p.cu_new[from + lane] : INT_MAX;
            const unsigned in = __ballot_sync(0xffffffffu, begin < warp_row + 32);
            for (unsigned left = in; left; left &= left - 1) {
                const int k = __ffs(left) - 1;
                if (__shfl_sync(0xffffffffu, begin, k) <= row)
                    r = from + k;
            }
            if (in != 0xffffffffu)
                break;
        }
    }
    __syncthreads();
    if (row >= p.T)
        return;

    // ---- its index, and the way up -----------------------------------------------------
    uint32_t *mask = p.mask + row * p.words;
    int64_t begin = 0, pos = 0;
    bool on = r >= 0 && row < rows;
    if (on) {
        const int64_t a = p.cu_new[r], b = p.cu_new[r + 1];
        begin = max(a, (int64_t)0);
        const int64_t n = b - a, cached = (int64_t)p.kv_len[r] - n;
        on = row < b;
        if (on && row == begin) {
            if (a < 0 || b > p.T)
                record_bad_index(p.err, kSiteTreeRows, a < 0 ? a : b);
            if (cached < 0)
                record_bad_index(p.err, kSiteTreeLen, p.kv_len[r]);
        }
        pos = p.pos0 + max(cached, (int64_t)0);
    }
    int i = on ? (int)(row - begin) : 0;
    if (on && i >= most) {
        if (i == most)
            record_bad_index(p.err, kSiteTreeSize, i);
        on = false;
    }
    int at = p.words - 1;  // the word to be written next
    uint32_t bits = 0;
    if (on) {
        const int base = (int)(begin - first);  // (the row's own index is below `most`: all before it is there)
        for (int depth = 0;; ++depth) {
            for (const int w = i >> 5; at > w; --at) {
                mask[at] = bits;
                bits = 0;
            }
            bits |= 1u << (i & 31);
            int up = s_parent[base + i];
            if (up < -1 || up >= i) {
                if (depth == 0)
                    record_bad_index(p.err, kSiteParent, up);
                up = -1;
            }
            if (up < 0) {
                pos += depth;
                break;
            }
            i = up;
        }
    }
    p.positions[row] = on ? pos : 0;
    for (; at >= 0; --at) {
        mask[at] = bits;
        bits = 0;
    }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams &p, cudaStream_t s)
{
    const size_t smem = (size_t)(kThreads + 32 * p.words) * 4;  // (at most 4.6 KB)
    tree_plan_kernel<<<(unsigned)((p.T + kThreads - 1) / kThreads), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rsa
