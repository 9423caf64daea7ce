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
// backward) operations apart.  Measured, 64 + 8 heads of 128 in bf16: 32768 tokens
// with their cache rows 224 us, 6.1 TB/s or 0.90 of a plain copy's rate; backward of
// 8192 tokens 84 us, 5.4 TB/s, 0.80, with the sums' launch (the instructions take 0.6
// of the issue slots); 1001 tokens of 8 + 8 heads of 64 in fp32, backward, 9.7 us.  A row of d elements lies across L = d * size / 16
// lanes, its sums are shuffles among those.  A group of L lanes goes through a run
// of items (kHeads heads of one token each): their rows come by 16-byte
// asynchronous copies into a ring of kStages items in shared memory, so that the
// bytes in flight do not sit in registers and do not wait for the arithmetic
// (loaded into registers an item at a time, a 32768-token prompt took 305 us); the
// token's cosines and sines are read when the token changes.  Which elements a lane
// holds depends on the rotation (Layout):
//   whole   halves of the whole row turn (rot = d): 8 bytes of each half, so that a
//           lane has both elements of its pairs and turns them two at a time with
//           packed fp32 arithmetic;
//   pairs   interleaved: 16 bytes in a row, which are whole pairs;
//   part    halves of the first rot < d elements: 16 bytes in a row; the pairs'
//           other elements are in another lane, one shuffle each.
// All arithmetic is in 32 bits; the result is rounded once, at the store.
#include <cuda_bf16.h>

#include "ptx_sm103.cuh"
#include "rsa_internal.h"

namespace rsa {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 4;       // items of a group's ring
constexpr int kBlocksPerSm = 3;  // 64 KB of ring each

enum Layout { kWhole, kPairs, kPart };

// What a lane holds of a row: N elements, 16 bytes, as floats two by two.
template <class E>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float2 *x)
    {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 *x)
    {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float2 two(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t one(const float2 &x)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);  // nearest even: the one rounding of the result
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ void unpack(const uint4 &u, float2 *x)
    {
        x[0] = two(u.x);
        x[1] = two(u.y);
        x[2] = two(u.z);
        x[3] = two(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float2 *x)
    {
        return make_uint4(one(x[0]), one(x[1]), one(x[2]), one(x[3]));
    }
};

template <class E, int D, Layout kLayout>
struct Shape {
    static constexpr int N = Piece<E>::N;      // elements of a lane
    static constexpr int L = D / N;            // lanes of a row
    static constexpr int kGroups = kThreads / L;
    // A lane's first element (kWhole: of its first run of N / 2; the second one is D / 2 on).
    static __device__ __forceinline__ int first(int lane) { return kLayout == kWhole ? lane * (N / 2) : lane * N; }
    // (also of a row in shared memory)
    static __device__ __forceinline__ uint4 load(const E *row, int e0)
    {
        if constexpr (kLayout == kWhole) {
            const uint2 a = *reinterpret_cast<const uint2 *>(row + e0), b = *reinterpret_cast<const uint2 *>(row + e0 + D / 2);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            return *reinterpret_cast<const uint4 *>(row + e0);
        }
    }
    static __device__ __forceinline__ void store(E *row, int e0, const uint4 &u)
    {
        if constexpr (kLayout == kWhole) {
            *reinterpret_cast<uint2 *>(row + e0) = make_uint2(u.x, u.y);
            *reinterpret_cast<uint2 *>(row + e0 + D / 2) = make_uint2(u.z, u.w);
        } else {
            *reinterpret_cast<uint4 *>(row + e0) = u;
        }
    }
};

// This lane's part of a row's rotation: cosines and sines of its pairs (kPart: of
// its elements, the sines negated in the pairs' first ones).  A lane's elements
// turn all or not at all, and its partner's elements are its own pairs' others, as
// rot/2 is a multiple of 8.
template <int N, Layout kLayout>
struct Turn {
    static constexpr int M = kLayout == kPart ? N / 2 : N / 4;
    float2 c[M], s[M];
    bool on;
    int partner;  // kPart: lane of the row
};

template <int N, Layout kLayout>
__device__ __forceinline__ Turn<N, kLayout> load_turn(const NormRopeParams &p, int64_t t, int e0)
{
    constexpr int M = Turn<N, kLayout>::M;
    Turn<N, kLayout> w = {};
    const int half = p.rot >> 1;
    w.on = kLayout == kWhole || e0 < p.rot;
    if (!w.on)
        return w;
    const bool second = kLayout == kPart && e0 >= half;
    const int f0 = kLayout == kPairs ? e0 >> 1 : (second ? e0 - half : e0);
    w.partner = (second ? e0 - half : e0 + half) / N;
    auto row = [&](int axis) {
        int64_t pos = p.positions[axis * p.T + t];
        if (pos < 0 || pos >= p.max_pos) {
            record_bad_index(p.err, kSitePosition, pos);
            pos = 0;
        }
        return p.cos_sin + pos * p.rot;
    };
    if (p.n_axes == 1) {
        const float *r = row(0) + f0;
        if constexpr (M % 2 == 0) {
#pragma unroll
            for (int i = 0; i < M; i += 2) {
                const float4 c = *reinterpret_cast<const float4 *>(r + 2 * i);
                const float4 n = *reinterpret_cast<const float4 *>(r + half + 2 * i);
                w.c[i] = make_float2(c.x, c.y), w.c[i + 1] = make_float2(c.z, c.w);
                w.s[i] = make_float2(n.x, n.y), w.s[i + 1] = make_float2(n.z, n.w);
            }
        } else {
            w.c[0] = *reinterpret_cast<const float2 *>(r);
            w.s[0] = *reinterpret_cast<const float2 *>(r + half);
        }
    } else {
        int axis = 0;
        auto next = [&](int f, float &c, float &n) {
            while (f >= p.axis_end[axis])
                ++axis;
            const float *r = row(axis);
            c = r[f];
            n = r[half + f];
        };
#pragma unroll
        for (int i = 0; i < M; ++i) {
            next(f0 + 2 * i, w.c[i].x, w.s[i].x);
            next(f0 + 2 * i + 1, w.c[i].y, w.s[i].y);
        }
    }
    if (kLayout == kPart && !second) {
#pragma unroll
        for (int i = 0; i < M; ++i)
            w.s[i] = make_float2(-w.s[i].x, -w.s[i].y);
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

__device__ __forceinline__ float2 neg(const float2 &x) { return make_float2(-x.x, -x.y); }

// y turned by the angles (or back), in place.
template <bool kBack, int N, int L, Layout kLayout>
__device__ __forceinline__ void turn(const NormRopeParams &p, const Turn<N, kLayout> &w, float2 *y)
{
    if constexpr (kLayout == kWhole) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float2 a = y[i], b = y[i + N / 4], s = kBack ? neg(w.s[i]) : w.s[i];
            y[i] = __ffma2_rn(a, w.c[i], neg(__fmul2_rn(b, s)));
            y[i + N / 4] = __ffma2_rn(a, s, __fmul2_rn(b, w.c[i]));
        }
    } else if constexpr (kLayout == kPairs) {
        if (w.on) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float a = y[i].x, b = y[i].y, c = i & 1 ? w.c[i / 2].y : w.c[i / 2].x;
                const float s0 = i & 1 ? w.s[i / 2].y : w.s[i / 2].x, s = kBack ? -s0 : s0;
                y[i].x = a * c - b * s;
                y[i].y = a * s + b * c;
            }
        }
    } else if (p.rot > 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float2 o;
            o.x = __shfl_sync(row_mask<L>(), y[i].x, w.partner, L);
            o.y = __shfl_sync(row_mask<L>(), y[i].y, w.partner, L);
            if (w.on)
                y[i] = __ffma2_rn(y[i], w.c[i], __fmul2_rn(o, kBack ? neg(w.s[i]) : w.s[i]));
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

template <class E, int D, Layout kLayout>
__device__ __forceinline__ void load_weight(const void *w, int e0, float2 *x)
{
    using S = Shape<E, D, kLayout>;
    if (w) {
        Piece<E>::unpack(S::load(static_cast<const E *>(w), e0), x);
    } else {
#pragma unroll
        for (int i = 0; i < S::N / 2; ++i)
            x[i] = make_float2(1.f, 1.f);
    }
}

template <class E>
__device__ __forceinline__ E *row_of(const HeadRows &h, int64_t t, int head)
{
    return static_cast<E *>(h.data) + t * h.token_stride + head * h.head_stride;
}

__device__ __forceinline__ float both(const float2 &x) { return x.x + x.y; }

__device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kPending>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// A group's place in the items: chunk c (of kHeads heads) of token t.
struct Item {
    int64_t t;
    int c;
    __device__ __forceinline__ void step(int chunks)
    {
        if (++c == chunks) {
            c = 0;
            ++t;
        }
    }
};

// The group's run of items: equal runs, the same number for every group but the last ones.
struct Run {
    Item first;
    int n;
};
__device__ __forceinline__ Run run_of(int64_t items, int chunks, int groups_per_block)
{
    const int64_t groups = (int64_t)gridDim.x * groups_per_block, each = (items + groups - 1) / groups;
    const int64_t g = (int64_t)blockIdx.x * groups_per_block + threadIdx.x / (kThreads / groups_per_block);
    const int64_t i0 = min(items, g * each);
    return Run{{i0 / chunks, (int)(i0 % chunks)}, (int)(min(items, i0 + each) - i0)};
}

// Forward: an item is up to kHeads heads of q, of k, or (copied to the cache) of v.
template <class E, int D, Layout kLayout, int kHeads>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p, int q_chunks, int kv_chunks)
{
    using S = Shape<E, D, kLayout>;
    constexpr int N = S::N, L = S::L;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x % L, e0 = S::first(lane), group = threadIdx.x / L;
    E *ring = reinterpret_cast<E *>(smem) + group * (kStages * kHeads * D);  // [kStages][kHeads][D]
    const int chunks = q_chunks + kv_chunks * (p.slot_map ? 2 : 1);
    const Run run = run_of(p.T * chunks, chunks, S::kGroups);
    // what an item is of: 0 q, 1 k, 2 v; its first head and their number
    struct Part {
        int what, h0, n;
    };
    auto part = [&](int c) {
        Part x;
        x.what = c < q_chunks ? 0 : (c < q_chunks + kv_chunks ? 1 : 2);
        x.h0 = (c - (x.what == 0 ? 0 : (x.what == 1 ? q_chunks : q_chunks + kv_chunks))) * kHeads;
        x.n = min(kHeads, (x.what == 0 ? p.Hq : p.Hkv) - x.h0);
        return x;
    };
    Item ahead = run.first;
    auto fetch = [&](int k) {
        if (k < run.n) {
            const Part x = part(ahead.c);
            const HeadRows &in = x.what == 0 ? p.q : (x.what == 1 ? p.k : p.v);
            const E *src = row_of<E>(in, ahead.t, x.h0) + lane * N;
            E *dst = ring + (k % kStages) * (kHeads * D) + lane * N;
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (i < x.n)
                    copy_async(dst + i * D, src + i * in.head_stride);
            ahead.step(chunks);
        }
        copies_commit();
    };
    for (int k = 0; k < kStages - 1; ++k)
        fetch(k);
    Item at = run.first;
    int64_t token = -1, slot = -1;
    int weight = -1;
    float2 w[N / 2];
    Turn<N, kLayout> tw;
    for (int k = 0; k < run.n; ++k, at.step(chunks)) {
        fetch(k + kStages - 1);
        if (at.t != token) {
            token = at.t;
            tw = load_turn<N, kLayout>(p, token, e0);
            slot = p.slot_map ? p.slot_map[token] : -1;
        }
        const Part x = part(at.c);
        if (x.what != 2 && x.what != weight) {
            weight = x.what;
            load_weight<E, D, kLayout>(weight == 0 ? p.q_weight : p.k_weight, e0, w);
        }
        // The token's rows of the cache, if it has a slot.
        E *cache = nullptr;
        const int64_t head_step = (int64_t)D << p.page_shift;
        if (x.what != 0 && slot >= 0) {
            const int64_t page = slot >> p.page_shift;
            if (page < p.n_pages)
                cache = static_cast<E *>(x.what == 1 ? p.k_cache : p.v_cache) + (page * p.Hkv + x.h0) * head_step +
                        (slot & ((1 << p.page_shift) - 1)) * D;
            else
                record_bad_index(p.err, kSiteSlot, slot);
        }
        const HeadRows &out = x.what == 0 ? p.q_out : p.k_out;
        const bool keep = x.what != 2 && out.data;
        copies_wait<kStages - 1>();
        __syncwarp(row_mask<L>());  // the other lanes' copies too
        const E *src = ring + (k % kStages) * (kHeads * D);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (i >= x.n)
                break;  // the same for every lane of the row
            uint4 raw = S::load(src + i * D, e0);
            if (x.what != 2) {
                float2 y[N / 2], ss = make_float2(0.f, 0.f);
                Piece<E>::unpack(raw, y);
#pragma unroll
                for (int e = 0; e < N / 2; ++e)
                    ss = __ffma2_rn(y[e], y[e], ss);
                const float r = rsqrtf(row_sum<L>(both(ss)) * (1.f / D) + p.eps);
                const float2 r2 = make_float2(r, r);
#pragma unroll
                for (int e = 0; e < N / 2; ++e)
                    y[e] = __fmul2_rn(__fmul2_rn(y[e], r2), w[e]);
                turn<false, N, L>(p, tw, y);
                raw = Piece<E>::pack(y);
            }
            if (keep)
                S::store(row_of<E>(out, token, x.h0 + i), e0, raw);
            if (cache)
                S::store(cache + i * head_step, e0, raw);
        }
        __syncwarp(row_mask<L>());  // every lane has read the item: its place may be filled again
    }
}

// Backward: as above with two rows a head, of x and of dy; a group keeps its part
// of the weights' gradients in registers; the block's groups are summed in shared
// memory and leave one row of partial sums, so that the result does not depend on
// any order of atomics.
template <class E, int D, Layout kLayout, int kHeads>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int q_chunks, int kv_chunks)
{
    using S = Shape<E, D, kLayout>;
    constexpr int N = S::N, L = S::L, G = S::kGroups;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x % L, e0 = S::first(lane), group = threadIdx.x / L;
    E *ring = reinterpret_cast<E *>(smem) + group * (kStages * 2 * kHeads * D);  // [kStages][x, dy][kHeads][D]
    const int chunks = q_chunks + kv_chunks;
    const Run run = run_of(p.T * chunks, chunks, G);
    ptx::launch_dependents();  // the sums' launch is made ready meanwhile
    float2 aq[N / 2] = {}, ak[N / 2] = {};
    Item ahead = run.first;
    auto fetch = [&](int k) {
        if (k < run.n) {
            const bool is_q = ahead.c < q_chunks;
            const int h0 = (is_q ? ahead.c : ahead.c - q_chunks) * kHeads, n = min(kHeads, (is_q ? p.Hq : p.Hkv) - h0);
            const HeadRows &in = is_q ? p.q : p.k, &dy = is_q ? p.dq_out : p.dk_out;
            const E *xs = row_of<E>(in, ahead.t, h0) + lane * N, *ys = row_of<E>(dy, ahead.t, h0) + lane * N;
            E *dst = ring + (k % kStages) * (2 * kHeads * D) + lane * N;
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (i < n) {
                    copy_async(dst + i * D, xs + i * in.head_stride);
                    copy_async(dst + (kHeads + i) * D, ys + i * dy.head_stride);
                }
            ahead.step(chunks);
        }
        copies_commit();
    };
    for (int k = 0; k < kStages - 1; ++k)
        fetch(k);
    Item at = run.first;
    int64_t token = -1;
    int weight = -1;
    float2 w[N / 2];
    Turn<N, kLayout> tw;
    for (int k = 0; k < run.n; ++k, at.step(chunks)) {
        fetch(k + kStages - 1);
        if (at.t != token) {
            token = at.t;
            tw = load_turn<N, kLayout>(p, token, e0);
        }
        const bool is_q = at.c < q_chunks;
        const int h0 = (is_q ? at.c : at.c - q_chunks) * kHeads, n = min(kHeads, (is_q ? p.Hq : p.Hkv) - h0);
        const HeadRows &dx = is_q ? p.q_out : p.k_out;
        if (weight != is_q) {
            weight = is_q;
            load_weight<E, D, kLayout>(is_q ? p.q_weight : p.k_weight, e0, w);
        }
        copies_wait<kStages - 1>();
        __syncwarp(row_mask<L>());
        const E *src = ring + (k % kStages) * (2 * kHeads * D);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (i >= n)
                break;  // the same for every lane of the row
            float2 x[N / 2], g[N / 2], ss = make_float2(0.f, 0.f), sd = ss;
            Piece<E>::unpack(S::load(src + i * D, e0), x);
            Piece<E>::unpack(S::load(src + (kHeads + i) * D, e0), g);
            turn<true, N, L>(p, tw, g);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                ss = __ffma2_rn(x[e], x[e], ss);
                sd = __ffma2_rn(__fmul2_rn(g[e], w[e]), x[e], sd);
            }
            const float r = rsqrtf(row_sum<L>(both(ss)) * (1.f / D) + p.eps);
            const float m = -row_sum<L>(both(sd)) * (1.f / D) * r;  // -mean(c o xhat)
            const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
            for (int e = 0; e < N / 2; ++e) {
                const float2 xh = __fmul2_rn(x[e], r2);
                if (is_q)
                    aq[e] = __ffma2_rn(g[e], xh, aq[e]);
                else
                    ak[e] = __ffma2_rn(g[e], xh, ak[e]);
                g[e] = __fmul2_rn(r2, __ffma2_rn(g[e], w[e], __fmul2_rn(xh, m2)));
            }
            S::store(row_of<E>(dx, token, h0 + i), e0, Piece<E>::pack(g));
        }
        __syncwarp(row_mask<L>());
    }
    __syncthreads();  // the ring becomes the sums' table
    float(*part)[D] = reinterpret_cast<float(*)[D]>(smem);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            const int at = e0 + (kLayout == kWhole && e >= N / 4 ? D / 2 - N / 2 : 0) + 2 * e;
            *reinterpret_cast<float2 *>(&part[group][at]) = which ? ak[e] : aq[e];
        }
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
    ptx::wait_for_launch_before();
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

// Blocks for `items`, at most `most`; ring bytes of a block: kHeads rows (of `rows` tensors) a stage and group.
template <class E, int D, Layout kLayout>
int blocks_for(int64_t items, int most)
{
    const int64_t want = (items + Shape<E, D, kLayout>::kGroups - 1) / Shape<E, D, kLayout>::kGroups;
    return (int)(want < most ? want : most);
}

template <class E, int D, Layout kLayout>
constexpr int ring_bytes(int kHeads, int rows)
{
    return Shape<E, D, kLayout>::kGroups * kStages * rows * kHeads * D * (int)sizeof(E);
}

template <class E, int D, Layout kLayout>
cudaError_t launch_fwd(const NormRopeParams &p, cudaStream_t s)
{
    constexpr int kHeads = 4, kSmem = ring_bytes<E, D, kLayout>(kHeads, 1);
    auto kernel = qk_norm_rope_kernel<E, D, kLayout, kHeads>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return e;
    const int qc = (p.Hq + kHeads - 1) / kHeads, kc = (p.Hkv + kHeads - 1) / kHeads;
    const int blocks = blocks_for<E, D, kLayout>(p.T * (qc + kc * (p.slot_map ? 2 : 1)), kBlocksPerSm * 152);
    kernel<<<blocks, kThreads, kSmem, s>>>(p, qc, kc);
    return cudaGetLastError();
}

template <class E, int D, Layout kLayout>
cudaError_t launch_bwd(const NormRopeParams &p, cudaStream_t s)
{
    constexpr int kHeads = 2, kSmem = ring_bytes<E, D, kLayout>(kHeads, 2);
    auto kernel = qk_norm_rope_bwd_kernel<E, D, kLayout, kHeads>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess)
        return e;
    const int qc = (p.Hq + kHeads - 1) / kHeads, kc = (p.Hkv + kHeads - 1) / kHeads;
    const int blocks = blocks_for<E, D, kLayout>(p.T * (qc + kc), kNormRopeBwdBlocks);
    kernel<<<blocks, kThreads, kSmem, s>>>(p, qc, kc);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weight_grad_kernel, (const float *)p.partial, blocks, D, p.dq_weight, p.dk_weight);
}

template <class E, int D>
cudaError_t launch(const NormRopeParams &p, bool backward, cudaStream_t s)
{
    if (p.interleaved)
        return backward ? launch_bwd<E, D, kPairs>(p, s) : launch_fwd<E, D, kPairs>(p, s);
    if (p.rot == D)
        return backward ? launch_bwd<E, D, kWhole>(p, s) : launch_fwd<E, D, kWhole>(p, s);
    return backward ? launch_bwd<E, D, kPart>(p, s) : launch_fwd<E, D, kPart>(p, s);
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
