// Attention of packed query rows over a shared prefix and their requests' own
// paged keys, on the CUDA cores (fp32 inputs, whose results tf32 could not
// hold), and the launch that joins the pieces of both types.
//
//   o = softmax([q Kp^T, q Kr^T] / sqrt(d)) [Vp; Vr]
// for the prefix' keys p and the request's own keys r, by pieces of the keys
// whose (o, lse) are joined with
//   M = max_i lse_i, L = M + ln sum e^{lse_i - M}, o = sum e^{lse_i - L} o_i.
//
// A CTA takes its stretch of the work (paged_sched.cuh).  It brings 128 (d = 64) or
// 64 keys and values at a time into shared memory, by asynchronous copies one such
// turn ahead of the arithmetic, in blocks of 32 keys.  A warp takes up to 8 rows of
// the unit through a block: lane (x, y) of 8 x 4 scores keys x, x + 8, .. for rows y
// and y + 4, and owns columns 4x.. of each 32 of the same rows of the output, so that
// every value read from shared memory serves several products
// and a row's maximum and factors stay in its lanes.  A unit of few rows leaves warps
// over: they are then cut into 2 or 4 key groups, which take the turn's blocks in
// parallel and join their rows at the end of the piece.
// Measured: 5 requests of 2 tokens, 4 key heads of 64, behind 4097 keys 20.5 us (4 key
// groups and these tiles; with one row or two a warp, every block through all 16, it
// took 41); one row of 4 heads of 64 over 100000 keys 62 us, 3.3 TB/s; 8 heads of 128 over
// 60000 keys with 20 rows each 274 us, 18.0 TFLOP/s, and 512 rows over 4608 keys 340 us, 26.8
// TFLOP/s of the visible pairs (a step of 4 columns is six 16-byte shared loads for 32
// products a lane; which of the two pipes binds has not been counted).
// Drafted tokens (kTree) in tiles of 32 keys: 5 requests of 3 to 13 tokens, 4 key heads of 64, behind
// 4097 keys 30.2 us (with tiles of 128 43).  Four rows a lane instead of two would read shared memory
// less but spilled (32 us).
// A unit of few rows is bound by one warp's way through a block, not by the loads: the
// same with a producer warp and TMA, which brings them earlier, took 82 us for a row of
// 100000 keys that took 68.
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "paged_sched.cuh"
#include "ptx_sm103.cuh"
#include "tc_common.cuh"

namespace rsa {
namespace {

using namespace paged;

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kRows = 128;            // rows of a unit
constexpr int kWarpRows = 8;
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

// 2 or 4 values side by side.
template <int N>
__device__ __forceinline__ void load(const float *p, float (&x)[N])
{
    if constexpr (N == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x, x[1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ void store(float *p, const float (&x)[N])
{
    if constexpr (N == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}
template <int N>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[N])
{
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        w[i] = tc::pack_bf16(x[2 * i], x[2 * i + 1]);
    if constexpr (N == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = w[0];
}

// 16 bytes to shared memory; zeros if not `there`.
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

template <int D>
struct Smem {
    static constexpr int kBlocks = D == 64 ? 4 : 2, kTurn = kBlocks * kKeys;  // of a turn
    // (rows are padded so that 8 rows of K and 4 of the others fall into different banks)
    float q[kRows][D + 4];
    float k[2][kTurn][D + 4];
    float v[2][kTurn][D];
    float p[kWarps][kWarpRows][kKeys + 8];  // a warp's probabilities of its block
    int64_t sum[kWarps];
    Stretch st;
};

// The ids of the pages of this thread's keys (j, j + step, ...; below j1) ...
template <int kCopies>
__device__ __forceinline__ void look_up(const PrefixAttnParams &p, const Piece &x, int64_t j, int step, int64_t j1, int (&ids)[kCopies])
{
#pragma unroll
    for (int i = 0; i < kCopies; ++i, j += step)
        ids[i] = j < j1 ? x.pages[j >> p.page_shift] : 0;
}

// ... and the copies of them: 16 bytes of each key and value, from column 4 * piece.
template <int D, int kCopies>
__device__ __forceinline__ void fetch(const PrefixAttnParams &p, const Piece &x, Smem<D> &s, int buffer, int key, int piece, int step,
                                      int64_t j0, int64_t j1, const int (&ids)[kCopies])
{
    const float *kc = static_cast<const float *>(p.k_cache), *vc = static_cast<const float *>(p.v_cache);
#pragma unroll
    for (int i = 0; i < kCopies; ++i, key += step) {
        const int64_t j = j0 + key;
        if (j < j1) {
            const bool there = ids[i] >= 0 && ids[i] < p.n_pages;  // (the keys of another id count as zeros)
            if (!there)
                record_bad_index(p.err, kSiteCachePage, ids[i]);
            const int64_t row = (((int64_t)(there ? ids[i] : 0) * p.Hkv + x.head) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
            copy_async(&s.k[buffer][key][piece * 4], kc + row * D + piece * 4, there);
            copy_async(&s.v[buffer][key][piece * 4], vc + row * D + piece * 4, there);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// A lane's rows of a piece: y and y + 4 of its warp's.
template <int D>
struct Rows {
    static constexpr int H = D / 32;
    float m[2], l[2];  // (l: of this lane's keys)
    float4 o[2][H];
    int see[2];  // they see keys [0, see) of the segment
};

// What the rows' masks say of the keys from the piece's `drafted` on.
struct Masks {
    const PrefixAttnParams &p;
    int tok, row0, drafted;  // the piece's first token, the warp's first row

    // 32 bits of row row0 + i, from key j on.
    __device__ __forceinline__ uint32_t bits(int i, int j) const
    {
        return mask_bits(p.mask + (tok + (row0 + i) / p.G) * p.mask_stride, p.words, j - drafted);
    }
};

__device__ __forceinline__ void add_product(float4 &o, float p, const float4 &v)
{
    const float2 pp = make_float2(p, p);
    const float2 a = __ffma2_rn(pp, make_float2(v.x, v.y), make_float2(o.x, o.y));
    const float2 b = __ffma2_rn(pp, make_float2(v.z, v.w), make_float2(o.z, o.w));
    o = make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void scale_by(float4 &o, float a) { o.x *= a, o.y *= a, o.z *= a, o.w *= a; }

// A warp's first 4 J rows, whose queries are q, through one block of nk keys from key j0 on.
template <int D, int J, bool kTree>
__device__ __forceinline__ void block(Rows<D> &r, const float (*q)[D + 4], const float (*ks)[D + 4], const float (*vs)[D],
                                      float (*ps)[kKeys + 8], int nk, int j0, float scale, const Masks &masks)
{
    constexpr int H = Rows<D>::H;
    const int x = threadIdx.x & 7, y = (threadIdx.x & 31) >> 3;
    float2 dot[4][J];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
            dot[i][j] = make_float2(0.f, 0.f);
    // (Past the last key or row it reads what lies there; those scores are not used.)
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 u[J];
#pragma unroll
        for (int j = 0; j < J; ++j)
            u[j] = *reinterpret_cast<const float4 *>(&q[y + 4 * j][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = *reinterpret_cast<const float4 *>(&ks[x + 8 * i][c]);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                dot[i][j] = __ffma2_rn(make_float2(u[j].x, u[j].y), make_float2(w.x, w.y), dot[i][j]);
                dot[i][j] = __ffma2_rn(make_float2(u[j].z, u[j].w), make_float2(w.z, w.w), dot[i][j]);
            }
        }
    }
    float sc[4][J], mx[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int lim = min(nk, r.see[j] - j0);
        uint32_t bits = 0xffffffffu;
        if (kTree && j0 + kKeys > masks.drafted && lim > 0)  // (a row that is none sees no key)
            bits = masks.bits(y + 4 * j, j0);
        mx[j] = r.m[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sc[i][j] = x + 8 * i < lim && (!kTree || (bits >> (x + 8 * i) & 1)) ? (dot[i][j].x + dot[i][j].y) * scale : -INFINITY;
            mx[j] = fmaxf(mx[j], sc[i][j]);
        }
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
#pragma unroll
        for (int j = 0; j < J; ++j)
            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], d));
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const float base = mx[j] == -INFINITY ? 0.f : mx[j], alpha = expf(r.m[j] - base);
        r.m[j] = mx[j];
        r.l[j] *= alpha;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float pj = expf(sc[i][j] - base);
            r.l[j] += pj;
            ps[y + 4 * j][x + 8 * i] = pj;
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
            scale_by(r.o[j][h], alpha);
    }
    __syncwarp();
    int k = 0;
#pragma unroll 1
    for (; k + 4 <= nk; k += 4) {
        float4 pk[J];
#pragma unroll
        for (int j = 0; j < J; ++j)
            pk[j] = *reinterpret_cast<const float4 *>(&ps[y + 4 * j][k]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 v = *reinterpret_cast<const float4 *>(&vs[k + e][32 * h + 4 * x]);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    add_product(r.o[j][h], e == 0 ? pk[j].x : (e == 1 ? pk[j].y : (e == 2 ? pk[j].z : pk[j].w)), v);
            }
    }
#pragma unroll 1
    for (; k < nk; ++k)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(&vs[k][32 * h + 4 * x]);
#pragma unroll
            for (int j = 0; j < J; ++j)
                add_product(r.o[j][h], ps[y + 4 * j][k], v);
        }
    __syncwarp();  // ps is written again with the next block
}

template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads) prefix_attn_f32_kernel(const __grid_constant__ PrefixAttnParams p)
{
    constexpr int H = D / 32, kBlocks = Smem<D>::kBlocks, kTurn = Smem<D>::kTurn;
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>(raw);
    const int warp = threadIdx.x >> 5, lane_x = threadIdx.x & 7, y = (threadIdx.x & 31) >> 3;
    const int G = p.G;
    const int worker = blockIdx.x;
    const float scale = 1.0f / sqrtf((float)D);

    if constexpr (kTree)
        ptx::wait_for_launch_before();
    const Stretch st = find_stretch<kThreads, false>(p, worker, s.sum, &s.st);
    ptx::launch_dependents();
    Walk<false> walk;
    walk.begin(p, st, worker);
    Piece x;
    while (walk.next(p, x)) {
        const int rows = (int)x.ntok * G;
        __syncthreads();  // the last piece's rows are done with q, and with the ring
#pragma unroll 4
        for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), c = i % (D / 4) * 4;
            const int64_t at = (int64_t)(x.tok + row / G) * p.q_token_stride + (x.head * G + row % G) * p.q_head_stride + c;
            *reinterpret_cast<float4 *>(&s.q[row][c]) = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at);
        }
        // kWarpRows rows a warp, or fewer, and as many key groups of such warps as there
        // are warps and blocks for.
        const int row_groups = (rows + kWarpRows - 1) / kWarpRows, per = (rows + row_groups - 1) / row_groups;
        int key_groups = kBlocks;
        while (row_groups * key_groups > kWarps)
            key_groups >>= 1;
        const int kg = warp / row_groups, row0 = (warp - kg * row_groups) * per;
        const bool works = kg < key_groups;
        const Masks masks{p, x.tok, row0, x.drafted};
        Rows<D> r;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = row0 + y + 4 * j;
            r.m[j] = -INFINITY;
            r.l[j] = 0.f;
            r.see[j] = row < rows ? (int)max((int64_t)0, min((int64_t)x.keys, x.see0 + row / G)) : 0;
#pragma unroll
            for (int h = 0; h < H; ++h)
                r.o[j][h] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const int64_t most = min((int64_t)x.keys, x.see0 + (x.ntok - 1));  // the keys that any row sees
        const int64_t j1 = min(most, (int64_t)x.t1 << p.tile_shift);
        const int64_t j00 = (int64_t)x.t0 << p.tile_shift;
        // A turn: this thread copies 16 bytes of kCopies keys, whose pages' ids it read
        // a turn before.  Keys past the last one are not copied.
        constexpr int kPieces = D / 4, kCopies = kTurn * kPieces / kThreads, kStep = kThreads / kPieces;
        const int piece = threadIdx.x % kPieces, key0 = threadIdx.x / kPieces;
        int ids[kCopies];
        look_up<kCopies>(p, x, j00 + key0, kStep, j1, ids);
        fetch<D, kCopies>(p, x, s, 0, key0, piece, kStep, j00, j1, ids);
        look_up<kCopies>(p, x, j00 + kTurn + key0, kStep, j1, ids);
        int buffer = 0;
        for (int64_t j0 = j00; j0 < j1; j0 += kTurn, buffer ^= 1) {
            fetch<D, kCopies>(p, x, s, buffer ^ 1, key0, piece, kStep, j0 + kTurn, j1, ids);
            look_up<kCopies>(p, x, j0 + 2 * kTurn + key0, kStep, j1, ids);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();  // every thread's copies of this turn
            for (int b = works ? kg : kBlocks; b < kBlocks; b += key_groups) {
                const int64_t jb = j0 + b * kKeys;
                if (jb >= j1)
                    break;
                const int nk = (int)min((int64_t)kKeys, j1 - jb);
                if (per <= 4)
                    block<D, 1, kTree>(r, &s.q[row0], &s.k[buffer][b * kKeys], &s.v[buffer][b * kKeys], s.p[warp], nk, (int)jb, scale, masks);
                else
                    block<D, 2, kTree>(r, &s.q[row0], &s.k[buffer][b * kKeys], &s.v[buffer][b * kKeys], s.p[warp], nk, (int)jb, scale, masks);
            }
            __syncthreads();  // the turn is done with: its buffer is filled next
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int d = 1; d < 8; d <<= 1)
                r.l[j] += __shfl_xor_sync(0xffffffffu, r.l[j], d);
        // The key groups' rows are joined in their order, through the ring.
        float(*scratch)[D + 4] = s.k[0];  // [key group - 1][row]: o, m, l
        static_assert(sizeof s.k >= sizeof(float) * kRows * (D + 4), "scratch");
        if (key_groups > 1) {
            if (works && kg > 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = row0 + y + 4 * j;
                    if (y + 4 * j >= per || row >= rows)
                        continue;
                    float *w = scratch[(kg - 1) * rows + row];
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        *reinterpret_cast<float4 *>(w + 32 * h + lane_x * 4) = r.o[j][h];
                    if (lane_x == 0) {
                        w[D] = r.m[j];
                        w[D + 1] = r.l[j];
                    }
                }
            }
            __syncthreads();
        }
        if (kg > 0)
            continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = row0 + y + 4 * j;
            if (y + 4 * j >= per || row >= rows)
                continue;
            for (int g = 1; g < key_groups; ++g) {
                const float *w = scratch[(g - 1) * rows + row];
                const float mn = fmaxf(r.m[j], w[D]), base = mn == -INFINITY ? 0.f : mn;
                const float a = expf(r.m[j] - base), b = expf(w[D] - base);
                r.m[j] = mn;
                r.l[j] = r.l[j] * a + w[D + 1] * b;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    scale_by(r.o[j][h], a);
                    add_product(r.o[j][h], b, *reinterpret_cast<const float4 *>(w + 32 * h + lane_x * 4));
                }
            }
            const int token = x.tok + row / G;
            const int hq = x.head * G + row % G;
            const bool empty = !(r.l[j] > 0.f) && r.l[j] == r.l[j];
            const float inv = empty ? 0.f : 1.f / r.l[j];
            const int64_t at = (int64_t)token * p.Hq + hq, slot = (int64_t)worker * kPrefixUnitRows + row;
            float *dst, *lse;
            if (is_result(p, x)) {
                dst = static_cast<float *>(p.out) + at * D;
                lse = p.lse + at;
            } else if (x.first) {
                dst = p.home_o[x.seg > 0] + at * D;
                lse = p.home_lse[x.seg > 0] + at;
            } else {
                dst = p.slot_o + slot * D;
                lse = p.slot_lse + slot;
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                scale_by(r.o[j][h], inv);
                *reinterpret_cast<float4 *>(dst + 32 * h + lane_x * 4) = r.o[j][h];
            }
            if (lane_x == 0)
                *lse = empty ? -INFINITY : r.m[j] + logf(r.l[j]);
        }
    }
}

// ---- joining -----------------------------------------------------------------------

// The request of a token: the last r with cu_q[r] <= token (requests without
// tokens share their successor's row), by 32-way search; -1 behind the last one.
__device__ __forceinline__ int request_of(const PrefixAttnParams &p, int token)
{
    const int lane = threadIdx.x & 31;
    if (token >= p.cu_q[p.R] || token < p.cu_q[0])
        return -1;
    int64_t lo = 0, n = p.R;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int64_t step = (n + 31) / 32;
        const bool below = lane * step < n && p.cu_q[lo + lane * step] <= token;
        const unsigned vote = __ballot_sync(0xffffffffu, below);
        if (!vote)
            return -1;  // (only where cu_q does not ascend)
        const int k = 31 - __clz(vote);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return (int)lo;
}

// The same for each lane's own token, by two levels of 32: every 32nd part's first row and
// then, of each lane's part, its own.
__device__ __forceinline__ int lane_request_of(const PrefixAttnParams &p, int token)
{
    const int lane = threadIdx.x & 31;
    if (!__any_sync(0xffffffffu, token < p.cu_q[p.R]))
        return -1;
    int64_t lo = 0, n = p.R;  // this lane's answer is in [lo, lo + n)
    // the first level is the same for all lanes: they read its 32 rows together
    const int64_t step = (n + 31) / 32;
    const int begin = lane * step < n ? p.cu_q[lane * step] : INT_MAX;
    int part = -1;
#pragma unroll
    for (int k = 0; k < 32; ++k)
        part += __shfl_sync(0xffffffffu, begin, k) <= token;
    const bool there = part >= 0 && token < p.cu_q[p.R];
    lo = max(part, 0) * step;
    n = min(step, n - lo);
    while (n > 1) {  // (with up to 1024 requests five reads of a few lines)
        const int64_t half = (n + 1) / 2;
        if (p.cu_q[lo + half] <= token)
            lo += half, n -= half;
        else
            n = half;
    }
    return there ? (int)lo : -1;
}

// Places of the line before request r's segment and in all, where the R < 32 requests'
// segments are a lane each: follows from the lengths alone, so a warp can work it out
// while the attention launch still computes (2 us less for a short call).  With more
// requests that would cost every warp a scan, and it takes the sums that worker 0 has left.
struct Sums {
    int64_t before, total;            // of this lane's request; of all
    int64_t pairs_before, all_pairs;  // the same for the even groups

    // r: this lane's request; few: R < 32.
    __device__ __forceinline__ Sums(const PrefixAttnParams &p, int r, bool few)
    {
        const int lane = threadIdx.x & 31;
        pairs_before = all_pairs = 0;
        r = max(r, 0);
        if (few) {
            int64_t x = 0, y = 0;
            if (lane <= p.R) {
                const Segment g = segment<true>(p, lane);
                x = g.line;
                y = g.pair_line;
            }
            scan(x, r, before, total);
            if (p.side_by_side)
                scan(y, r, pairs_before, all_pairs);
        } else {
            total = p.plan[p.R + 1];
            before = p.plan[1 + r];
            if (p.side_by_side) {
                all_pairs = p.pair_plan[p.R + 1];
                pairs_before = p.pair_plan[1 + r];
            }
        }
    }
    // x: of the lane's segment.
    __device__ __forceinline__ static void scan(int64_t x, int r, int64_t &before, int64_t &total)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        before = __shfl_sync(0xffffffffu, x, r);  // (segments 0 to r lie before 1 + r)
        total = __shfl_sync(0xffffffffu, x, 31);
    }
};

// The pieces of one key head's rows of a token in one segment: their home, then one
// slot for each worker after the first.
struct Pieces {
    int64_t slot;  // row of the first query head's first slot; the next worker's are kPrefixUnitRows further
    int n;
};

// Segment g, before which lie `before` and `pairs_before` places of its parts of the line.
__device__ __forceinline__ Pieces pieces_of(const PrefixAttnParams &p, const Segment &g, int64_t before, int64_t pairs_before,
                                            const Line &line, int token, int head)
{
    const int i = token - g.tok0;
    if (g.tiles == 0 || i < 0 || i >= g.ntok)  // (outside: only where cu_q does not ascend)
        return Pieces{0, 0};
    const int group = i / p.unit_tokens;
    int64_t at;
    if (group < 2 * g.pairs) {
        at = (group & 1 ? line.odd : 0) + pairs_before + ((int64_t)head * g.pairs + (group >> 1)) * g.unit_line();
    } else {
        const int64_t unit = (int64_t)head * g.singles + (group - 2 * g.pairs) - g.skip;
        if (unit < 0)
            return Pieces{0, 1};  // a whole unit that is not on the line
        at = line.rest + before + unit * g.unit_line();
    }
    at += g.unit;  // the unit's first tile
    const int64_t w0 = at / line.share, w1 = (at + (int64_t)(g.tiles - 1) * g.cost) / line.share;
    return Pieces{(w0 + 1) * kPrefixUnitRows + (i % p.unit_tokens) * p.G, (int)(w1 - w0) + 1};
}

// Where piece i of a row lies: (o, lse).
struct Locate {
    const PrefixAttnParams &p;
    int64_t row;
    int g;          // query head within the key head
    Pieces pc[2];   // prefix, own

    __device__ __forceinline__ void operator()(int i, int d, const float *&o, const float *&lse) const
    {
        const int s = i >= pc[0].n;
        const int k = i - (s ? pc[0].n : 0);
        const int64_t slot = (s ? pc[1].slot : pc[0].slot) + g + (int64_t)(k - 1) * kPrefixUnitRows;
        o = k == 0 ? (s ? p.home_o[1] : p.home_o[0]) + row * d : p.slot_o + slot * d;
        lse = k == 0 ? (s ? p.home_lse[1] : p.home_lse[0]) + row : p.slot_lse + slot;
    }
};

// Pieces [from, end) of a row, for the whole warp.  Lane i brings the lse of piece i, so that all
// of them are in flight together, and with them the first kAhead rows of o.  Lane c owns columns
// [c * PER, (c + 1) * PER).
template <int D, int kAhead>
struct Fold {
    static constexpr int PER = D / 32;
    float M, L, acc[PER];

    __device__ __forceinline__ void pieces(int from, int end, const Locate &locate)
    {
        const int lane = threadIdx.x & 31;
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int c = 0; c < PER; ++c)
            acc[c] = 0.f;
        for (int i0 = from; i0 < end; i0 += 32) {
            const int m = min(32, end - i0);
            const float *o = nullptr, *at = nullptr;
            if (lane < m)
                locate(i0 + lane, D, o, at);
            const float lse = lane < m ? *at : -INFINITY;
            // The first rows of o are under way before their weights are known, kAhead at a time.
            float v[kAhead][PER];
            auto fetch_rows = [&](int i) {
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const float *oi = reinterpret_cast<const float *>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (i + e) & 31));
                    if (i + e < m)
                        load(oi + lane * PER, v[e]);
                }
            };
            fetch_rows(0);
            const float mn = fmaxf(M, warp_max(lse));
            const float base = mn == -INFINITY ? 0.f : mn;
            const float a = expf(M - base), w = expf(lse - base);
            L = L * a + warp_sum(w);
            M = mn;
#pragma unroll
            for (int c = 0; c < PER; ++c)
                acc[c] *= a;
#pragma unroll 1
            for (int i = 0;;) {
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const float wi = __shfl_sync(0xffffffffu, w, (i + e) & 31);
                    if (i + e < m)
#pragma unroll
                        for (int c = 0; c < PER; ++c)
                            acc[c] = fmaf(wi, v[e][c], acc[c]);
                }
                i += kAhead;
                if (i >= m)
                    break;
                fetch_rows(i);
            }
        }
    }
    template <class E>
    __device__ __forceinline__ void write(const PrefixAttnParams &p, int64_t row) const
    {
        const int lane = threadIdx.x & 31;
        const bool empty = !(L > 0.f) && L == L;  // (a NaN stays one)
        const float inv = empty ? 0.f : 1.f / L;
        float y[PER];
#pragma unroll
        for (int c = 0; c < PER; ++c)
            y[c] = acc[c] * inv;
        store(static_cast<E *>(p.out) + row * D + lane * PER, y);
        if (lane == 0)
            p.lse[row] = empty ? -INFINITY : M + logf(L);
    }
};

// Up to four rows that follow one another with up to eight pieces each: lane 8 q + i has row q's
// piece i, so that the rows' maxima, weights and sums are worked out together (row after row they
// were most of 232 instructions a row of three pieces, now 147; the launch for 65536 rows 20.9 ->
// 17.5 us).  The same results as Fold's in every bit.
template <class E, int D, int kAhead>
__device__ __forceinline__ void fold_four(const PrefixAttnParams &p, const Locate &locate, int n, int rows)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31, q_lane = lane >> 3, i_lane = lane & 7;
    const bool here = i_lane < n && q_lane < rows;
    const float *o = nullptr, *at = nullptr;
    if (i_lane < n)
        locate(i_lane, D, o, at);
    const float lse = here ? at[q_lane] : -INFINITY;
    float v[kAhead][4][PER], acc[4][PER];
    auto fetch_rows = [&](int i) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const float *oi =
                reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (i + e) & 7)) +
                lane * PER;
            if (i + e >= n)
                continue;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < rows)
                    load(oi + q * D, v[e][q]);
        }
    };
    fetch_rows(0);
    float M = lse;
#pragma unroll
    for (int b = 4; b > 0; b >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, b));
    const float w = expf(lse - (M == -INFINITY ? 0.f : M));
    float L = w;
#pragma unroll
    for (int b = 4; b > 0; b >>= 1)
        L += __shfl_xor_sync(0xffffffffu, L, b);
    const bool empty = !(L > 0.f) && L == L;  // (a NaN stays one)
    const float inv = empty ? 0.f : 1.f / L;
    if (i_lane == 0 && q_lane < rows)
        p.lse[locate.row + q_lane] = empty ? -INFINITY : M + logf(L);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < PER; ++c)
            acc[q][c] = 0.f;
#pragma unroll 1
    for (int i = 0;;) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float wi = __shfl_sync(0xffffffffu, w, 8 * q + ((i + e) & 7));
                if (i + e < n && q < rows)
#pragma unroll
                    for (int c = 0; c < PER; ++c)
                        acc[q][c] = fmaf(wi, v[e][q][c], acc[q][c]);
            }
        i += kAhead;
        if (i >= n)
            break;
        fetch_rows(i);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float f = __shfl_sync(0xffffffffu, inv, 8 * q);
        float y[PER];
#pragma unroll
        for (int c = 0; c < PER; ++c)
            y[c] = acc[q][c] * f;
        if (q < rows)
            store(static_cast<E *>(p.out) + (locate.row + q) * D + lane * PER, y);
    }
}

// Few rows: kParts warps a row (token, query head), each with a run of its pieces.
template <class E, int D, int kParts>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ PrefixAttnParams p)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5, part = warp % kParts;
    // (spare warps repeat a row)
    const int64_t row = min((int64_t)blockIdx.x * (kJoinWarps / kParts) + warp / kParts, p.T * p.Hq - 1);
    const int token = (int)(row / p.Hq);
    const int hq = (int)(row - (int64_t)token * p.Hq), head = hq / p.G;
    const int r = request_of(p, token);
    const Segment g[2] = {segment<true>(p, 0), r < 0 ? Segment() : segment<true>(p, 1 + r)};
    const bool few = p.R < 32;
    if (!few)
        ptx::wait_for_launch_before();
    const Sums sums(p, r, few);
    const Line line(p, sums.all_pairs, sums.total);
    Locate locate{p, row, hq - head * p.G, {{0, 0}, {0, 0}}};
    if (r >= 0) {
        locate.pc[0] = pieces_of(p, g[0], 0, 0, line, token, head);
        locate.pc[1] = pieces_of(p, g[1], sums.before, sums.pairs_before, line, token, head);
    }
    // Every thread waits, also where it has nothing to join: the launch after this one
    // waits only for this one.
    if (few)
        ptx::wait_for_launch_before();
    if (r < 0 || (locate.pc[1].n == 1 && p.prefix_len == 0))
        return;  // a row behind the last request stays as it is; a single piece went straight to out
    const int n = locate.pc[0].n + locate.pc[1].n, run = (n + kParts - 1) / kParts, end = min(n, (part + 1) * run);
    Fold<D, 4> f;
    f.pieces(part * run, end, locate);
    if constexpr (kParts > 1) {
        __shared__ float s_part[kJoinWarps][D + 2];
        if (part > 0) {
#pragma unroll
            for (int c = 0; c < PER; ++c)
                s_part[warp][lane * PER + c] = f.acc[c];
            if (lane == 0) {
                s_part[warp][D] = f.M;
                s_part[warp][D + 1] = f.L;
            }
        }
        // (named barriers of one row's warps: another row's may have returned)
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + warp / kParts), "n"(kParts * 32) : "memory");
        if (part > 0)
            return;
#pragma unroll
        for (int i = 1; i < kParts; ++i) {
            const float *w = s_part[warp + i];
            const float mn = fmaxf(f.M, w[D]), base = mn == -INFINITY ? 0.f : mn;
            const float a = expf(f.M - base), b = expf(w[D] - base);
            f.M = mn;
            f.L = f.L * a + w[D + 1] * b;
#pragma unroll
            for (int c = 0; c < PER; ++c)
                f.acc[c] = f.acc[c] * a + w[lane * PER + c] * b;
        }
    }
    f.template write<E>(p, row);
}

// Many rows: an item is up to kJoinRows rows of a (token, key head), and a warp takes every
// so-manieth.  Where the pieces of its next 32 items lie its lanes work out at once: done row
// by row, that search and its divisions took most of the launch's time (46080 rows of 3
// pieces 56 us, 622592 rows with nothing to join 365 us).
template <class E, int D, int kJoinRows, int kAhead, int kBlocks>
__global__ void __launch_bounds__(kJoinThreads, kBlocks) prefix_join_rows_kernel(const __grid_constant__ PrefixAttnParams p)
{
    const int lane = threadIdx.x & 31, cuts = (p.G + kJoinRows - 1) / kJoinRows;
    const int64_t items = p.T * p.Hkv * cuts, warps = (int64_t)gridDim.x * kJoinWarps;
    const int64_t first = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    const bool few = p.R < 32;
    const Segment prefix = segment<true>(p, 0);
    bool waited = false;
    for (int64_t i0 = first; i0 < items; i0 += 32 * warps) {
        const int64_t item = i0 + lane * warps;
        const bool there = item < items;
        const int64_t head_row = (there ? item : items - 1) / cuts;  // token * Hkv + head
        const int g0 = (int)((there ? item : items - 1) - head_row * cuts) * kJoinRows;
        const int token = (int)(head_row / p.Hkv), head = (int)(head_row - (int64_t)token * p.Hkv);
        const int r = lane_request_of(p, token);
        const Segment g = segment<true>(p, 1 + max(r, 0));
        if (!few && !waited) {
            ptx::wait_for_launch_before();
            waited = true;
        }
        const Sums sums(p, r, few);
        const Line line(p, sums.all_pairs, sums.total);
        Pieces pre{0, 0}, own{0, 0};
        if (r >= 0) {
            pre = pieces_of(p, prefix, 0, 0, line, token, head);
            own = pieces_of(p, g, sums.before, sums.pairs_before, line, token, head);
        }
        if (!waited)
            ptx::wait_for_launch_before();
        waited = true;
        // (rows behind the last request stay as they are; a single piece went straight to out)
        const unsigned todo = __ballot_sync(0xffffffffu, there && r >= 0 && !(own.n == 1 && p.prefix_len == 0));
#pragma unroll 1
        for (unsigned left = todo; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const int64_t row0 = __shfl_sync(0xffffffffu, head_row * p.G + g0, k);
            Locate locate{p, row0, __shfl_sync(0xffffffffu, g0, k),
                          {{__shfl_sync(0xffffffffu, pre.slot, k), __shfl_sync(0xffffffffu, pre.n, k)},
                           {__shfl_sync(0xffffffffu, own.slot, k), __shfl_sync(0xffffffffu, own.n, k)}}};
            const int n = locate.pc[0].n + locate.pc[1].n;
            int rows = min(kJoinRows, p.G - locate.g);
            if constexpr (kJoinRows == 4) {
                if (n <= 8) {
                    fold_four<E, D, kAhead>(p, locate, n, rows);
                    continue;
                }
            }
#pragma unroll 1
            for (; rows > 0; --rows, ++locate.g, ++locate.row) {
                Fold<D, kJoinRows == 1 ? kAhead : 4> f;
                f.pieces(0, n, locate);
                f.template write<E>(p, locate.row);
            }
        }
    }
    if (!waited)
        ptx::wait_for_launch_before();
}

template <int D>
cudaError_t simt(const PrefixAttnParams &p_in, cudaStream_t s)
{
    PrefixAttnParams p = p_in;
    p.unit_tokens = p.light_tokens = kRows / p.G;
    p.tile_shift = kTileShift;
    p.light_tile = p.heavy_tile = 2;
    p.unit = 3;
    p.unit_shift = 31;
    p.side_by_side = 0;
    if (p.mask) {
        // Trees are short calls: tiles of 32 keys, which even out what the SMs get (40 tokens of 8
        // heads behind 4097 keys 43 -> 33 us, 2 requests of 16 tokens behind 2000 31.6 -> 20.6;
        // tiles of 64 36 and 23).  A unit of over 64 rows takes a block's time twice.
        p.tile_shift = 5;
        p.light_tokens = 64 / p.G;
        p.light_tile = 1;
        p.heavy_tile = 2;
        p.unit = 4;
    }
    auto kernel = p.mask ? prefix_attn_f32_kernel<D, true> : prefix_attn_f32_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
    if (e != cudaSuccess)
        return e;
    if (p.mask) {
        e = launch_early(kernel, dim3((unsigned)p.workers), kThreads, sizeof(Smem<D>), s, 1, p);
    } else {
        kernel<<<p.workers, kThreads, sizeof(Smem<D>), s>>>(p);
        e = cudaGetLastError();
    }
    return e != cudaSuccess ? e : launch_prefix_join(p, s);
}

template <class E, int D, int kJoinRows, int kAhead, int kBlocks>
cudaError_t join_rows(const PrefixAttnParams &p, cudaStream_t s)
{
    const int64_t items = p.T * p.Hkv * ((p.G + kJoinRows - 1) / kJoinRows), blocks = (items + kJoinWarps - 1) / kJoinWarps;
    const dim3 grid((unsigned)(blocks < 152 * kBlocks ? blocks : 152 * kBlocks));
    return launch_early(prefix_join_rows_kernel<E, D, kJoinRows, kAhead, kBlocks>, grid, kJoinThreads, 0, s, 1, p);
}

// Up to a row for each SM: four warps a row, since the fewer the rows, the more pieces
// has each (19 pieces a row in 64 rows, a call of 24.7 us takes 22.4; with 5 pieces a
// row in 256 it would take 20.0 instead of 19.1).  Then a row a warp while the SMs hold
// them at once, else four rows together, for the loads in flight.
template <class E, int D>
cudaError_t join_any(const PrefixAttnParams &p, cudaStream_t s)
{
    constexpr int kParts = 4;
    const int64_t rows = p.T * p.Hq;
    if (rows <= 152) {
        const dim3 grid((unsigned)((rows * kParts + kJoinWarps - 1) / kJoinWarps));
        return launch_early(prefix_join_kernel<E, D, kParts>, grid, kJoinThreads, 0, s, 1, p);
    }
    return rows <= 152 * 32 ? join_rows<E, D, 1, 8, 2>(p, s) : join_rows<E, D, 4, 3, 2>(p, s);
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

cudaError_t launch_prefix_join(const PrefixAttnParams &p, cudaStream_t s)
{
    if (p.d == 128)
        return p.f32 ? join_any<float, 128>(p, s) : join_any<__nv_bfloat16, 128>(p, s);
    if (p.d == 64)
        return p.f32 ? join_any<float, 64>(p, s) : join_any<__nv_bfloat16, 64>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace rsa
