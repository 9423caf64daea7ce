// Attention of packed query rows over a shared prefix and their requests' own
// paged keys, on the CUDA cores (fp32 inputs, whose results tf32 could not
// hold), and the launch that joins the pieces of both types.
//
//   o = softmax([q Kp^T, q Kr^T] / sqrt(d)) [Vp; Vr]
// for the prefix' keys p and the request's own keys r, by pieces of the keys
// whose (o, lse) are joined with
//   M = max_i lse_i, L = M + ln sum e^{lse_i - M}, o = sum e^{lse_i - L} o_i.
//
// A CTA takes its stretch of the work (paged_sched.cuh).  It brings 32 keys and
// values at a time into shared memory; a warp owns up to 16 rows of the unit.
// Lane k scores key k (a dot product along d, its own row of K from shared
// memory, the query broadcast), maximum and sum are shuffles, and for the
// output lane c owns columns c, c + 32, ... with the probabilities broadcast.
// Bound by shared-memory loads and fp32 arithmetic.  Values of masked keys are
// never touched: they may hold anything.
#include <cuda_bf16.h>

#include <cmath>

#include "paged_sched.cuh"

namespace rsa {
namespace {

using namespace paged;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 128;            // rows of a unit
constexpr int kWarpRows = kRows / kWarps;
constexpr int kKeys = 32;             // keys of a block

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void store(float *p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

template <int D>
struct Smem {
    float q[kRows][D];
    float k[kKeys][D + 4];  // (+ 4: the lanes' rows fall into different banks)
    float v[kKeys][D];
    int64_t sum[kWarps];
    Stretch st;
};

template <int D>
__global__ void __launch_bounds__(kThreads) prefix_attn_f32_kernel(const __grid_constant__ PrefixAttnParams p)
{
    constexpr int PER = D / 32;
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G, TU = kRows / G;
    const int worker = blockIdx.x;
    const float scale = 1.0f / sqrtf((float)D);
    const int page_mask = (1 << p.page_shift) - 1;
    const float *kc = static_cast<const float *>(p.k_cache), *vc = static_cast<const float *>(p.v_cache);

    const Stretch st = find_stretch<kThreads>(p, TU, worker, s.sum, &s.st);
    Walk walk;
    walk.begin(p, st, TU);
    Piece x;
    while (walk.next(p, TU, x)) {
        const int rows = (int)x.ntok * G;
        __syncthreads();  // the last piece's rows are done with q
        for (int i = threadIdx.x; i < rows * D; i += kThreads) {
            const int row = i / D, c = i - row * D;
            const int64_t token = x.tok + row / G;
            s.q[row][c] =
                static_cast<const float *>(p.q)[token * p.q_token_stride + (x.head * G + row % G) * p.q_head_stride + c];
        }
        // Row i * kWarps + warp of the unit, and the keys it sees.
        float m[kWarpRows], l[kWarpRows], o[kWarpRows][PER];
        int64_t see[kWarpRows];
        int64_t most = 0;  // the keys that any row sees
#pragma unroll
        for (int i = 0; i < kWarpRows; ++i) {
            const int row = i * kWarps + warp;
            m[i] = -INFINITY;
            l[i] = 0.f;
            see[i] = row < rows ? min(x.keys, x.see0 + row / G) : 0;
#pragma unroll
            for (int c = 0; c < PER; ++c)
                o[i][c] = 0.f;
        }
        most = min(x.keys, x.see0 + (x.ntok - 1));
        const int64_t j1 = min(most, x.t1 * kTileKeys);
        for (int64_t j0 = x.t0 * kTileKeys; j0 < j1; j0 += kKeys) {
            const int nk = (int)min((int64_t)kKeys, j1 - j0);
            __syncthreads();  // the last block of keys is done with
            for (int i = threadIdx.x; i < nk * D; i += kThreads) {
                const int key = i / D, c = i - key * D;
                const int64_t j = j0 + key;
                const int page = x.pages[j >> p.page_shift];
                float a = 0.f, b = 0.f;
                if (page >= 0 && page < p.n_pages) {
                    const int64_t at = ((((int64_t)page * p.Hkv + x.head) << p.page_shift) + (j & page_mask)) * D + c;
                    a = kc[at];
                    b = vc[at];
                } else if (c == 0) {
                    record_bad_index(p.err, 0x55, page);
                }
                s.k[key][c] = a;
                s.v[key][c] = b;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWarpRows; ++i) {
                const int row = i * kWarps + warp;
                const int n = (int)min((int64_t)nk, see[i] - j0);  // keys of the block that the row sees
                if (n <= 0)
                    continue;  // the same for the whole warp
                float sc = -INFINITY;
                if (lane < n) {
                    float dot = 0.f;
                    const float4 *a = reinterpret_cast<const float4 *>(s.q[row]), *b = reinterpret_cast<const float4 *>(s.k[lane]);
#pragma unroll 8
                    for (int c = 0; c < D / 4; ++c) {
                        const float4 u = a[c], w = b[c];
                        dot = fmaf(u.x, w.x, dot);
                        dot = fmaf(u.y, w.y, dot);
                        dot = fmaf(u.z, w.z, dot);
                        dot = fmaf(u.w, w.w, dot);
                    }
                    sc = dot * scale;
                }
                const float mn = fmaxf(m[i], warp_max(sc));
                const float base = mn == -INFINITY ? 0.f : mn;
                const float alpha = expf(m[i] - base), pj = lane < n ? expf(sc - base) : 0.f;
                l[i] = l[i] * alpha + warp_sum(pj);
                m[i] = mn;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    o[i][c] *= alpha;
                for (int k = 0; k < n; ++k) {
                    const float pk = __shfl_sync(0xffffffffu, pj, k);
#pragma unroll
                    for (int c = 0; c < PER; ++c)
                        o[i][c] = fmaf(pk, s.v[k][lane + 32 * c], o[i][c]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kWarpRows; ++i) {
            const int row = i * kWarps + warp;
            if (row >= rows)
                continue;
            const int64_t token = x.tok + row / G;
            const int hq = x.head * G + row % G;
            const Place d = place(p, x, worker, token, hq, row);
            const bool empty = !(l[i] > 0.f) && l[i] == l[i];
            const float inv = empty ? 0.f : 1.f / l[i], lse = empty ? -INFINITY : m[i] + logf(l[i]);
            if (d.final_) {
                float *out = static_cast<float *>(p.out) + (token * p.Hq + hq) * D;
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    out[lane + 32 * c] = o[i][c] * inv;
                if (lane == 0)
                    p.lse[token * p.Hq + hq] = lse;
            } else {
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    d.o[lane + 32 * c] = o[i][c] * inv;
                if (lane == 0)
                    *d.lse = lse;
            }
        }
    }
}

// ---- joining -----------------------------------------------------------------------

// The request of a token: the last r with cu_q[r] <= token (requests without
// tokens share their successor's row), by 32-way search; -1 behind the last one.
__device__ __forceinline__ int64_t request_of(const PrefixAttnParams &p, int64_t token)
{
    const int lane = threadIdx.x & 31;
    if (token >= p.cu_q[p.R])
        return -1;
    int64_t lo = 0, n = p.R;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int64_t step = (n + 31) / 32;
        const int64_t at = lo + lane * step;
        const bool below = lane * step < n && p.cu_q[at] <= token;
        const unsigned vote = __ballot_sync(0xffffffffu, below);
        if (!vote)
            return -1;  // (rows before cu_q[0])
        const int k = 31 - __clz(vote);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

// One warp a row (token, query head): lane c owns columns [c * PER, ...).
template <class E, int D>
__global__ void __launch_bounds__(kThreads) prefix_join_kernel(const __grid_constant__ PrefixAttnParams p, int tokens_per_unit)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= p.T * p.Hq)
        return;
    const int64_t token = row / p.Hq;
    const int hq = (int)(row - token * p.Hq), head = hq / p.G;
    const int64_t r = request_of(p, token);
    if (r < 0)
        return;  // rows behind the last request stay as they are
    const int64_t share = p.plan[p.R + 2];
    float M = -INFINITY, L = 0.f, acc[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c)
        acc[c] = 0.f;
    auto add = [&](const float *o, float lse) {
        if (lse == -INFINITY)
            return;  // an empty piece: its o is not read
        const float mn = fmaxf(M, lse);
        const float a = expf(M - mn), b = expf(lse - mn);
        M = mn;
        L = L * a + b;
#pragma unroll
        for (int c = 0; c < PER; ++c)
            acc[c] = fmaf(o[lane * PER + c], b, acc[c] * a);
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int64_t seg = s == 0 ? 0 : 1 + r;
        const Segment g = segment(p, seg, tokens_per_unit);
        const int64_t i = token - g.tok0;
        if (g.line == 0 || i < 0 || i >= g.ntok)
            continue;  // (outside: only where cu_q does not ascend)
        const int64_t unit = head * g.groups + i / tokens_per_unit;
        const int64_t at = p.plan[seg] + unit * g.tiles;
        const int64_t w0 = at / share, w1 = (at + g.tiles - 1) / share;
        if (s == 1 && w0 == w1 && p.prefix_len == 0)
            return;  // one piece: it went straight to out
        add(p.home_o[s] + row * D, p.home_lse[s][row]);
        const int local = (int)(i % tokens_per_unit) * p.G + (hq - head * p.G);
        for (int64_t w = w0 + 1; w <= w1; ++w) {
            const int64_t slot = w * kPrefixUnitRows + local;
            add(p.slot_o + slot * D, p.slot_lse[slot]);
        }
    }
    const float inv = M == -INFINITY ? 0.f : 1.f / L;
    E *out = static_cast<E *>(p.out) + row * D + lane * PER;
#pragma unroll
    for (int c = 0; c < PER; ++c)
        store(out + c, acc[c] * inv);
    if (lane == 0)
        p.lse[row] = M == -INFINITY ? -INFINITY : M + logf(L);
}

template <int D>
cudaError_t simt(const PrefixAttnParams &p, cudaStream_t s)
{
    cudaError_t e =
        cudaFuncSetAttribute(prefix_attn_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
    if (e != cudaSuccess)
        return e;
    prefix_attn_f32_kernel<D><<<p.workers, kThreads, sizeof(Smem<D>), s>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_prefix_join(p, kRows / p.G, s);
}

template <class E, int D>
cudaError_t join(const PrefixAttnParams &p, int tokens_per_unit, cudaStream_t s)
{
    const int64_t blocks = (p.T * p.Hq + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    prefix_join_kernel<E, D><<<(unsigned)blocks, kThreads, 0, s>>>(p, tokens_per_unit);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_attn_f32(const PrefixAttnParams &p, cudaStream_t s)
{
    if (p.d == 128)
        return simt<128>(p, s);
    if (p.d == 64)
        return simt<64>(p, s);
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefix_join(const PrefixAttnParams &p, int tokens_per_unit, cudaStream_t s)
{
    if (p.d == 128)
        return p.f32 ? join<float, 128>(p, tokens_per_unit, s) : join<__nv_bfloat16, 128>(p, tokens_per_unit, s);
    if (p.d == 64)
        return p.f32 ? join<float, 64>(p, tokens_per_unit, s) : join<__nv_bfloat16, 64>(p, tokens_per_unit, s);
    return cudaErrorInvalidValue;
}

}  // namespace rsa
