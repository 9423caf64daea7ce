// RMS norm of every query and key head with the position rotation in the same
// pass, keys and values written to their slots of the paged cache; and the
// backward pass.
//
//   xhat = x / sqrt(mean(x^2) + eps),  y = R(pos) (w o xhat)
// R turns the pairs (i, i + rot/2), or (2i, 2i+1) when interleaved, of the
// first rot elements by the angle of frequency i at the token's position; the
// cosines and sines come from a table, row pos, [cos_0.. | sin_0..].  With
// several axes each frequency takes the position of its own axis.
// Backward, with g = R(pos)^T dy and c = w o g:
//   dx = (c - xhat mean(c o xhat)) / sqrt(mean(x^2) + eps),  dw = sum g o xhat
// over all tokens and heads.
//
// Bound by HBM: every element is read once and written once, about 10 (20
// backward) operations apart.  So each thread moves 16-byte pieces, a row of d
// elements lies across L = d * size / 16 lanes, its two sums (one per row and
// direction) are shuffles among those lanes, and a group of L lanes takes
// kHeads heads of one token with all their loads in flight at once: the
// token's cosines and sines are read once per group.  The partner of a
// half-turned element is in another lane: one shuffle.  All arithmetic is in
// 32 bits; the result is rounded once, at the store.
#include <cuda_bf16.h>

#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 256;

// 16 bytes of a row as floats.
template <class E>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *x)
    {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *x)
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void two(uint32_t w, float *x)
    {
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t one(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);  // nearest even: the one rounding of the result
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ void unpack(const uint4 &u, float *x)
    {
        two(u.x, x);
        two(u.y, x + 2);
        two(u.z, x + 4);
        two(u.w, x + 6);
    }
    static __device__ __forceinline__ uint4 pack(const float *x)
    {
        return make_uint4(one(x[0], x[1]), one(x[2], x[3]), one(x[4], x[5]), one(x[6], x[7]));
    }
};

template <class E, int D>
struct Shape {
    static constexpr int N = Piece<E>::N;      // elements of a thread
    static constexpr int L = D / N;            // lanes of a row
    static constexpr int kGroups = kThreads / L;
};

// This lane's part of a row's rotation: the factors of its elements (half) or
// pairs (interleaved).  A lane's elements turn all or not at all, and its
// partner's elements are its own pairs' others, as rot/2 is a multiple of 8.
template <int N, bool INTER>
struct Turn {
    static constexpr int M = INTER ? N / 2 : N;
    float c[M], s[M];  // half: s is negated in the pairs' first elements
    bool on;
    int partner;  // lane of the row
};

template <int N, bool INTER>
__device__ __forceinline__ Turn<N, INTER> load_turn(const NormRopeParams &p, int64_t t, int e0)
{
    constexpr int M = Turn<N, INTER>::M;
    Turn<N, INTER> w = {};
    const int half = p.rot >> 1;
    w.on = e0 < p.rot;
    if (!w.on)
        return w;
    const bool second = !INTER && e0 >= half;
    const int f0 = INTER ? e0 >> 1 : (second ? e0 - half : e0);
    w.partner = (second ? e0 - half : e0 + half) / N;
    auto row = [&](int axis) {
        int64_t pos = p.positions[axis * p.T + t];
        if (pos < 0 || pos >= p.max_pos) {
            record_bad_index(p.err, 0x51, pos);
            pos = 0;
        }
        return p.cos_sin + pos * p.rot;
    };
    if (p.n_axes == 1) {
        const float *r = row(0) + f0;
        if constexpr (M % 4 == 0) {
#pragma unroll
            for (int i = 0; i < M; i += 4) {
                const float4 c = *reinterpret_cast<const float4 *>(r + i);
                const float4 n = *reinterpret_cast<const float4 *>(r + half + i);
                w.c[i] = c.x, w.c[i + 1] = c.y, w.c[i + 2] = c.z, w.c[i + 3] = c.w;
                w.s[i] = n.x, w.s[i + 1] = n.y, w.s[i + 2] = n.z, w.s[i + 3] = n.w;
            }
        } else {
            const float2 c = *reinterpret_cast<const float2 *>(r);
            const float2 n = *reinterpret_cast<const float2 *>(r + half);
            w.c[0] = c.x, w.c[1] = c.y;
            w.s[0] = n.x, w.s[1] = n.y;
        }
    } else {
        int axis = 0;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            while (f0 + i >= p.axis_end[axis])
                ++axis;
            const float *r = row(axis);
            w.c[i] = r[f0 + i];
            w.s[i] = r[half + f0 + i];
        }
    }
    if (!INTER && !second) {
#pragma unroll
        for (int i = 0; i < M; ++i)
            w.s[i] = -w.s[i];
    }
    return w;
}

// The lanes of this thread's row: all of them shuffle together, other rows of
// the warp may be elsewhere.
template <int L>
__device__ __forceinline__ unsigned row_mask()
{
    return L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << (threadIdx.x & 31 & ~(L - 1));
}

// y turned by the angles (direction 1) or back (-1), in place.
template <int N, int L, bool INTER>
__device__ __forceinline__ void turn(const NormRopeParams &p, const Turn<N, INTER> &w, float *y, float direction)
{
    if constexpr (INTER) {
        if (w.on) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1], s = w.s[i] * direction;
                y[2 * i] = a * w.c[i] - b * s;
                y[2 * i + 1] = a * s + b * w.c[i];
            }
        }
    } else if (p.rot > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o = __shfl_sync(row_mask<L>(), y[i], w.partner, L);
            if (w.on)
                y[i] = y[i] * w.c[i] + o * (w.s[i] * direction);
        }
    }
}

template <int L>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(row_mask<L>(), x, o, L);
    return x;
}

template <class E, int N>
__device__ __forceinline__ void load_weight(const void *w, int e0, float *x)
{
    if (w) {
        Piece<E>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const E *>(w) + e0), x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = 1.f;
    }
}

template <class E>
__device__ __forceinline__ const uint4 *row_in(const HeadRows &h, int64_t t, int head, int e0)
{
    return reinterpret_cast<const uint4 *>(static_cast<const E *>(h.data) + t * h.token_stride + head * h.head_stride + e0);
}

template <class E>
__device__ __forceinline__ uint4 *row_out(const HeadRows &h, int64_t t, int head, int e0)
{
    return reinterpret_cast<uint4 *>(static_cast<E *>(h.data) + t * h.token_stride + head * h.head_stride + e0);
}

// Forward: a group of L lanes takes up to kHeads heads of one token: of q, of
// k, or (copied to the cache) of v.
template <class E, int D, bool INTER, int kHeads>
__global__ void __launch_bounds__(kThreads)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p, int q_chunks, int kv_chunks)
{
    constexpr int N = Shape<E, D>::N, L = Shape<E, D>::L;
    const int lane = threadIdx.x % L, e0 = lane * N;
    const int chunks = q_chunks + kv_chunks * (p.slot_map ? 2 : 1);
    const int64_t item = (int64_t)blockIdx.x * Shape<E, D>::kGroups + threadIdx.x / L;
    if (item >= p.T * chunks)
        return;  // the whole row of lanes leaves together
    const int64_t t = item / chunks;
    int c = (int)(item - t * chunks);
    const int what = c < q_chunks ? 0 : (c < q_chunks + kv_chunks ? 1 : 2);
    c -= what == 0 ? 0 : (what == 1 ? q_chunks : q_chunks + kv_chunks);
    const HeadRows &in = what == 0 ? p.q : (what == 1 ? p.k : p.v);
    const int heads = what == 0 ? p.Hq : p.Hkv;
    const int h0 = c * kHeads;
    const int n = min(kHeads, heads - h0);

    uint4 raw[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < n)
            raw[i] = *row_in<E>(in, t, h0 + i, e0);
        else
            raw[i] = make_uint4(0u, 0u, 0u, 0u);

    // The token's rows of the cache, if it has a slot.
    E *cache = nullptr;
    int64_t head_step = 0;
    if (what != 0 && p.slot_map) {
        const int64_t slot = p.slot_map[t];
        const int64_t page = slot >> p.page_shift;
        if (slot >= 0 && page < p.n_pages) {
            head_step = (int64_t)D << p.page_shift;
            cache = static_cast<E *>(what == 1 ? p.k_cache : p.v_cache) + (page * p.Hkv + h0) * head_step +
                    (slot & ((1 << p.page_shift) - 1)) * D + e0;
        } else if (slot >= 0) {
            record_bad_index(p.err, 0x52, slot);
        }
    }
    if (what != 2) {
        float w[N];
        load_weight<E, N>(what == 0 ? p.q_weight : p.k_weight, e0, w);
        const Turn<N, INTER> tw = load_turn<N, INTER>(p, t, e0);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            float x[N];
            Piece<E>::unpack(raw[i], x);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e)
                ss = fmaf(x[e], x[e], ss);
            const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < N; ++e)
                x[e] = x[e] * r * w[e];
            turn<N, L>(p, tw, x, 1.f);
            raw[i] = Piece<E>::pack(x);
        }
    }
    const HeadRows &out = what == 0 ? p.q_out : p.k_out;
    const bool keep = what != 2 && out.data;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < n) {
            if (keep)
                *row_out<E>(out, t, h0 + i, e0) = raw[i];
            if (cache)
                *reinterpret_cast<uint4 *>(cache + i * head_step) = raw[i];
        }
}

// Backward: as above, but a group goes through many (token, heads) items and
// keeps its part of the weights' gradients in registers; the block's groups
// are summed in shared memory and leave one row of partial sums, so that the
// result does not depend on any order of atomics.
template <class E, int D, bool INTER, int kHeads>
__global__ void __launch_bounds__(kThreads)
    qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int q_chunks, int kv_chunks)
{
    constexpr int N = Shape<E, D>::N, L = Shape<E, D>::L, G = Shape<E, D>::kGroups;
    __shared__ float part[G][D];
    const int lane = threadIdx.x % L, e0 = lane * N, group = threadIdx.x / L;
    const int chunks = q_chunks + kv_chunks;
    const int64_t items = p.T * chunks;
    float aq[N] = {}, ak[N] = {};
    for (int64_t item = (int64_t)blockIdx.x * G + group; item < items; item += (int64_t)gridDim.x * G) {
        const int64_t t = item / chunks;
        const int c = (int)(item - t * chunks);
        const bool is_q = c < q_chunks;
        const int h0 = (is_q ? c : c - q_chunks) * kHeads;
        const int n = min(kHeads, (is_q ? p.Hq : p.Hkv) - h0);
        const HeadRows &in = is_q ? p.q : p.k, &dy = is_q ? p.dq_out : p.dk_out, &dx = is_q ? p.q_out : p.k_out;
        uint4 xr[kHeads], yr[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < n) {
                xr[i] = *row_in<E>(in, t, h0 + i, e0);
                yr[i] = *row_in<E>(dy, t, h0 + i, e0);
            }
        float w[N];
        load_weight<E, N>(is_q ? p.q_weight : p.k_weight, e0, w);
        const Turn<N, INTER> tw = load_turn<N, INTER>(p, t, e0);
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < n) {  // the same for every lane of the row
                float x[N], g[N];
                Piece<E>::unpack(xr[i], x);
                Piece<E>::unpack(yr[i], g);
                turn<N, L>(p, tw, g, -1.f);
                float ss = 0.f, sd = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    ss = fmaf(x[e], x[e], ss);
                    sd = fmaf(g[e] * w[e], x[e], sd);
                }
                const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + p.eps);
                const float m = row_sum<L>(sd) * (1.f / D) * r;  // mean(c o xhat)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float xh = x[e] * r, dw = g[e] * xh;
                    aq[e] += is_q ? dw : 0.f;
                    ak[e] += is_q ? 0.f : dw;
                    g[e] = r * (g[e] * w[e] - xh * m);
                }
                *row_out<E>(dx, t, h0 + i, e0) = Piece<E>::pack(g);
            }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            part[group][e0 + e] = which ? ak[e] : aq[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < G; ++i)
                a += part[i][threadIdx.x];
            p.partial[((int64_t)blockIdx.x * 2 + which) * D + threadIdx.x] = a;
        }
        __syncthreads();
    }
}

// The blocks' partial sums of one weight's 32 columns, added in a fixed order.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float *partial, int blocks, int d, float *dwq, float *dwk)
{
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
    float a = 0.f;
    for (int b = y; b < blocks; b += 32)
        a += partial[((int64_t)b * 2 + blockIdx.y) * d + col];
    s[y][x] = a;
    __syncthreads();
    if (y == 0) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            a += s[i][x];
        float *dw = blockIdx.y ? dwk : dwq;
        if (dw)
            dw[col] = a;
    }
}

template <class E, int D, bool INTER>
cudaError_t launch_fwd(const NormRopeParams &p, cudaStream_t s)
{
    constexpr int kHeads = 4;
    const int qc = (p.Hq + kHeads - 1) / kHeads, kc = (p.Hkv + kHeads - 1) / kHeads;
    const int64_t items = p.T * (qc + kc * (p.slot_map ? 2 : 1));
    const int64_t blocks = (items + Shape<E, D>::kGroups - 1) / Shape<E, D>::kGroups;
    if (blocks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    qk_norm_rope_kernel<E, D, INTER, kHeads><<<(unsigned)blocks, kThreads, 0, s>>>(p, qc, kc);
    return cudaGetLastError();
}

template <class E, int D, bool INTER>
cudaError_t launch_bwd(const NormRopeParams &p, cudaStream_t s)
{
    constexpr int kHeads = 2;
    const int qc = (p.Hq + kHeads - 1) / kHeads, kc = (p.Hkv + kHeads - 1) / kHeads;
    const int64_t items = p.T * (qc + kc);
    const int64_t want = (items + Shape<E, D>::kGroups - 1) / Shape<E, D>::kGroups;
    const int blocks = (int)(want < kNormRopeBwdBlocks ? want : kNormRopeBwdBlocks);
    qk_norm_rope_bwd_kernel<E, D, INTER, kHeads><<<blocks, kThreads, 0, s>>>(p, qc, kc);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    weight_grad_kernel<<<dim3(D / 32, 2), 1024, 0, s>>>(p.partial, blocks, D, p.dq_weight, p.dk_weight);
    return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch(const NormRopeParams &p, bool backward, cudaStream_t s)
{
    if (p.interleaved)
        return backward ? launch_bwd<E, D, true>(p, s) : launch_fwd<E, D, true>(p, s);
    return backward ? launch_bwd<E, D, false>(p, s) : launch_fwd<E, D, false>(p, s);
}

cudaError_t launch_any(const NormRopeParams &p, bool backward, cudaStream_t s)
{
    if (p.d == 128)
        return p.f32 ? launch<float, 128>(p, backward, s) : launch<__nv_bfloat16, 128>(p, backward, s);
    if (p.d == 64)
        return p.f32 ? launch<float, 64>(p, backward, s) : launch<__nv_bfloat16, 64>(p, backward, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_qk_norm_rope_fwd(const NormRopeParams &p, cudaStream_t s) { return launch_any(p, false, s); }
cudaError_t launch_qk_norm_rope_bwd(const NormRopeParams &p, cudaStream_t s) { return launch_any(p, true, s); }

}  // namespace rsa
