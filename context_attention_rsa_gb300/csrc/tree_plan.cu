// Positions and ancestor masks of drafted tokens, from their parents.
//
//   A_i = {i} + A_parent(i),  depth_i = |A_i| - 1,  pos_i = pos0 + cached + depth_i
//
// A thread takes a row and walks up its ancestors, whose indices descend, so that it
// finishes one word of the mask after the other.  Of one or two words it holds both;
// of more only the last, and those done go to shared memory, whence the block writes
// them (lanes end a word at different steps, and a loop that fills words with zeros
// there holds up the whole warp: 17 trees of up to 177, 11.2 us, so 5.0).  Where more than
// half of a block's tokens are children of the one before them, a step goes over up to
// 32 of those (four chains of 1024 36 -> 6.6 us); where few are it would take 1.5 times
// as long, its steps being twice as dear.  The parents
// lie in shared memory, those of the block's rows and of as many rows before them as
// a mask has bits.  A row's request comes from a 32-way search of cu_new by its warp.
// The work is a few bytes a token: the launch, two or three dependent reads and one
// shared-memory access for each generation of the deepest tree bound it (8 trees of 16
// 2.2 us on the GPU; 1000 of up to 64, 33000 rows, 3.3).
#include <climits>

#include "ptx_sm103.cuh"
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

// kShort: masks of one or two words, held whole.
template <bool kShort>
__global__ void __launch_bounds__(kThreads) tree_plan_kernel(const __grid_constant__ TreePlanParams p)
{
    extern __shared__ int s_parent[];  // of rows [first, row0 + kThreads)
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_parent + kThreads + 32 * p.words);  // [kThreads][words + 1] (not kShort)
    uint32_t *s_follow = s_mask + kThreads * (p.words + 1);  // [words + kThreads / 32], from row row0 - 32 words on (not kShort)
    __shared__ int64_t s_begin;  // of the first row's request
    const int tid = threadIdx.x, lane = tid & 31, most = 32 * p.words;
    const int64_t row0 = (int64_t)blockIdx.x * kThreads, row = row0 + tid;
    const int64_t first = max((int64_t)0, row0 - (most - 1));
    if (!kShort)
        for (int k = tid; k < kThreads * (p.words + 1); k += kThreads)
            s_mask[k] = 0;
    ptx::wait_for_launch_before();
    for (int64_t t = first + tid; t < min(p.T, row0 + kThreads); t += kThreads)
        s_parent[t - first] = p.parent[t];

    // (a request for each row to look at: read early, told about late)
    int64_t look = row;
    int look_a = look <= p.R ? p.cu_new[look] : 0, look_b = look <= p.R ? p.cu_new[min(look + 1, (int64_t)p.R)] : 0;

    // ---- the row's request: the warp's first row's, or one after it --------------------
    // Its window of 32 requests comes in one read, with their lengths; more of them begin within
    // the warp's rows only where some have one row or none.
    const int64_t warp_row = row0 + (tid & ~31);
    int64_t begin = 0, end = 0, all = 0;
    for (int from = max(request_of(p, warp_row), 0);; from += 32) {
        const bool there = from + lane < p.R;
        const int a = there ? p.cu_new[from + lane] : INT_MAX, b = there ? p.cu_new[from + lane + 1] : INT_MAX;
        const int n = there ? p.kv_len[from + lane] : 0;
        const unsigned in = __ballot_sync(0xffffffffu, a < warp_row + 32);
        for (unsigned left = in; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const int ak = __shfl_sync(0xffffffffu, a, k), bk = __shfl_sync(0xffffffffu, b, k), nk = __shfl_sync(0xffffffffu, n, k);
            if (ak <= row)  // (requests without rows share their successor's: the last one has them)
                begin = ak, end = bk, all = nk;
        }
        if (in != 0xffffffffu)
            break;
    }
    if (!kShort && tid == 0)
        s_begin = max(begin, (int64_t)0);
    __syncthreads();
    while (look <= p.R) {
        if (look_a < 0 || look_a > p.T || look_b < look_a)
            record_bad_index(p.err, kSiteTreeRows, look_a < 0 || look_a > p.T ? look_a : look_b);
        look += (int64_t)gridDim.x * kThreads;
        if (look <= p.R) {
            look_a = p.cu_new[look];
            look_b = p.cu_new[min(look + 1, (int64_t)p.R)];
        }
    }

    // ---- its index, and the way up -----------------------------------------------------
    bool on = row < end && row < p.T;
    const int64_t cached = all - (end - begin);
    if (on && row == max(begin, (int64_t)0) && cached < 0)
        record_bad_index(p.err, kSiteTreeLen, all);
    begin = max(begin, (int64_t)0);
    const int64_t pos = p.pos0 + max(cached, (int64_t)0);
    int i = on ? (int)(row - begin) : 0;
    if (on && i >= most) {
        if (i == most)
            record_bad_index(p.err, kSiteTreeSize, i);
        on = false;
    }
    const int *parent = s_parent + (begin - first);  // (the row's own index is below `most`: all before it is there)
    int up = on ? parent[i] : -1, depth = 0;
    if (on && (up < -1 || up >= i))
        record_bad_index(p.err, kSiteParent, up);
    // (-1 and what is no earlier token end the walk)
    if constexpr (kShort) {
        uint32_t word[2] = {0, 0};
        auto set = [&] {
            const uint32_t bit = 1u << (i & 31);
            word[0] |= i < 32 ? bit : 0;
            word[1] |= i < 32 ? 0 : bit;
        };
        if (on)
            set();
        while ((unsigned)up < (unsigned)i) {
            i = up;
            up = parent[i];
            ++depth;
            set();
        }
        if (row < p.T) {
            uint32_t *mask = p.mask + row * p.words;
            mask[0] = word[0];
            if (p.words > 1)
                mask[1] = word[1];
        }
    } else {
        // A word of the mask is put away when the next one begins.
        uint32_t *mine = s_mask + tid * (p.words + 1), bits = 0;
        int w = i >> 5;
        const bool follows = on && i > 0 && up == i - 1;  // (the token is the child of the one before it)
        const int rows = __syncthreads_count(on);
        if (2 * __syncthreads_count(follows) > rows) {
            // ---- mostly chains: up to 32 tokens in a row at a time, by a bit for each that follows
            const unsigned vote = __ballot_sync(0xffffffffu, follows);
            if (lane == 0)
                s_follow[p.words + tid / 32] = vote;
            for (int k = tid; k < most; k += kThreads) {  // (whole warps; of the rows before the block's)
                const int64_t t = row0 - most + k;
                const unsigned v = __ballot_sync(0xffffffffu, t >= first && t > s_begin && s_parent[t - first] == t - s_begin - 1);
                if (lane == 0)
                    s_follow[k / 32] = v;
            }
            __syncthreads();
            const int off = on ? (int)(begin - row0) + most : 0;  // of token 0 in s_follow's bits
            for (bool more = on; more;) {
                const int at = off + i, k = at >> 5;
                const uint32_t x = __funnelshift_rc(k > 0 ? s_follow[k - 1] : 0, s_follow[k], (at & 31) + 1);
                // token i is behind `run` others in a row (never more than there are, also where cu_new does not ascend)
                const int run = min(__clz(~x), i), low = i - run;
                depth += run;
                if (i >> 5 != w) {
                    mine[w] = bits;
                    bits = 0;
                    w = i >> 5;
                }
                uint32_t set = ~0u >> (31 - (i & 31));
                if (low >> 5 != w) {
                    mine[w] = bits | set;
                    bits = 0;
                    --w;
                    set = ~0u;
                }
                bits |= set & ~0u << (low & 31);
                up = parent[low];
                more = (unsigned)up < (unsigned)low;
                i = up;
                depth += more;
            }
        } else {
            bits = 1u << (i & 31);
            while ((unsigned)up < (unsigned)i) {
                i = up;
                up = parent[i];
                ++depth;
                if (i >> 5 != w) {
                    mine[w] = bits;
                    bits = 0;
                    w = i >> 5;
                }
                bits |= 1u << (i & 31);
            }
        }
        if (on)
            mine[w] = bits;
        __syncthreads();
        const int n = (int)min((int64_t)kThreads, p.T - row0) * p.words;
        uint32_t *mask = p.mask + row0 * p.words;
        for (int k = tid; k < n; k += kThreads)
            mask[k] = s_mask[k + k / p.words];
    }
    if (row < p.T)
        p.positions[row] = on ? pos + depth : 0;
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams &p, cudaStream_t s)
{
    const int gathered = p.words > 2 ? kThreads * (p.words + 1) + p.words + kThreads / 32 : 0;
    const size_t smem = (size_t)(kThreads + 32 * p.words + gathered) * 4;  // (at most 22 KB)
    auto kernel = p.words <= 2 ? tree_plan_kernel<true> : tree_plan_kernel<false>;
    return launch_early(kernel, dim3((unsigned)((p.T + kThreads - 1) / kThreads)), kThreads, smem, s, 1, p);
}

}  // namespace rsa
