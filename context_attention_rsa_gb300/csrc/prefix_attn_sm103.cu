// Attention of packed query rows over a shared prefix and their requests' own
// paged keys, on the sm_103a tensor cores (bf16).
//
//   o = softmax([q Kp^T, q Kr^T] / sqrt(d)) [Vp; Vr], by pieces of the keys
// whose (o, lse) the joining launch puts together (prefix_attn_f32.cu).
//
// One CTA on each SM takes an equal stretch of all key tiles (paged_sched.cuh)
// and goes through its pieces.  Warp roles as in the block kernel:
//   warp 8      producer of Q and K: the piece's query rows (one 4-D TMA box a
//               128-row tile: G heads of floor(128 / G) tokens, so any group size is
//               loaded without a gather), then K tiles into every other slot of a ring
//               in shared memory, one box a page, each lane loading the page whose id
//               it read from the table one tile ahead.  It also walks the work for
//               the others and hands them each piece.
//   warp 10     producer of V, the other slots, walking by itself: a box takes the
//               issuing warp about 80 cycles, and one warp for K and V paced the loads
//               (4 long contexts 447 -> 425 us, pages of 16 behind 100000 keys 278 ->
//               254, short units 3 to 13 % less).
//   warp 9      one thread issues the MMAs: S_t = Q K^T from shared memory,
//               O_t += P_t V with P in TMEM.
//   warps 0-7   softmax, two threads a row (warps w and w + 4), in turn on the
//               two S tiles in TMEM.
// A piece runs in one of two forms, by its number of rows:
//   two tiles   more than 128 rows: S_0 and S_1 are the two row tiles against
//               the same key tile, as in the block kernel, so that a key tile
//               serves 256 rows; bound by the softmax chain of each tile.
//   one tile    up to 128 rows: S_0 and S_1 take the key tiles in turn, the S
//               MMAs two tiles ahead of PV and on into the next pieces; O_0 and
//               O_1 take the pieces in turn, so that a piece's result is written
//               while the next one is under way.  Warps without a row of the
//               piece only pass the barriers on, so a decode step's few rows
//               cost little and HBM is the bound.
// Rows past the keys are not trusted: a score of such a key is masked, but its
// 0 * NaN would reach O through V.  So they are never loaded: the segment's last,
// shorter tile is brought in groups of 8 rows; V's groups without keys lie outside the
// tensor map, which fills them with zeros (K's stay what they were: masked whatever
// they are), and the box of a group of v < 8 keys
// starts 8 - v rows early, on keys that are there already or before the page, on
// zeros.  The softmax masks those columns; the keys' order within a tile does not
// matter to it.
// The phases of all barriers run on over the CTA's pieces; one-tile pieces take
// the two Q tiles in turn, so that the next piece's loads are under way while
// one computes; O is written again once every softmax thread has read it.
//
// Measured (64 query heads over 8 key heads of 128; GB/s of the keys and values that
// have to be read, TFLOP/s of the visible pairs):
//   4 requests of 131072 to 262144 own keys       426 us, 6.95 TB/s, the rate of a copy
//   8 requests of 4 tokens, 32 key heads, behind
//     100000 keys in pages of 16                   255 us, 6.5 TB/s, 0.96 of a copy
//   608 requests behind 262144 keys               3760 us, 1389 TFLOP/s, 0.74 of cuBLAS (ten calls;
//     after a hundred, power-capped, 4080 us; keys of zeros, which cost less power, 3235 us)
//   512 new tokens with 32768 before them          421 us, 1316 TFLOP/s; a prompt of 8192 without
//     a past 1673 us, 657 TFLOP/s: its places count tiles that its rows do not see
//   64 requests of 4 to 2000 keys behind 32768      91 us: 40 us of two-tile steps and
//     18 of short units if perfectly shared; the scan 2, the first loads 5, a piece's end
//     6 (its 256 rows, 16 bytes a lane and store) and the joining launch 5 us
//   1 request of 1000 keys                        14.5 us, nearly all latency
// A step takes 2850 cycles, 4400 next to a CTA that runs short units, and what made short
// units faster by more code made the whole slower: as if two neighbouring SMs shared an
// instruction cache that the kernel's code fills (read from timings, not from a counter).
// P is rounded to bf16 for the MMA (2^-8 of each probability at most; the sum l takes it
// before that): with the result's own rounding 0.0021 to 0.0024 from the 64-bit
// answer, where rounding that answer alone gives 0.0017.
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "paged_sched.cuh"
#include "ptx_sm103.cuh"
#include "tc_common.cuh"

namespace rsa {
namespace {

using namespace tc;
using namespace paged;

constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f;  // log2 units the maximum may rise before O is rescaled
// Places of a key tile (kUnitCost for a unit): a step of two row tiles takes 1.5 us, of
// one 1.0, a short unit some 1.5 more.  Other weights (4:2:3, 3:3:4, 6:4:5, 4:4:6 for unit,
// one and two row tiles) move single batches by up to 10 % either way and none all.
constexpr int kLightTile = 2, kHeavyTile = 3;
constexpr float kLn2 = 0.69314718055994531f;

// A piece as the producer hands it to the other roles.
struct Work {
    int tiles;            // key tiles that any of its rows sees; -1: no piece follows
    int two;              // two row tiles against each key tile
    int t0, keys;         // its first tile; the segment's keys
    int64_t see0;         // unit token i sees keys [0, min(keys, see0 + i))
    int tok, ntok, head;  // the unit's tokens and key head
    int to;               // where its rows go: kHome + (0 prefix, 1 own), kSlot or kResult
};
constexpr int kHome = 0, kSlot = 2, kResult = 3;

__device__ __forceinline__ Work work_of(const Piece &x, const PrefixAttnParams &p)
{
    const int64_t seen = min((int64_t)x.keys, x.see0 + (x.ntok - 1));
    const int end = min(x.t1, seen > 0 ? (int)((seen + kTileKeys - 1) / kTileKeys) : 0);
    Work w;
    w.tiles = max(0, end - x.t0);
    w.two = x.ntok > p.light_tokens;
    w.t0 = x.t0;
    w.keys = x.keys;
    w.see0 = x.see0;
    w.tok = x.tok;
    w.ntok = x.ntok;
    w.head = x.head;
    w.to = !x.first ? kSlot : (is_result(p, x) ? kResult : kHome + (x.seg > 0));
    return w;
}

template <int D>
struct Cfg {
    static constexpr int kSoftmaxThreads = 256;
    static constexpr int kProducerWarp = 8;
    static constexpr int kMmaWarp = 9;
    static constexpr int kValueWarp = 10;
    static constexpr int kThreads = 352;
    static constexpr int kHalves = D / 64;              // 128-byte halves of a row
    static constexpr uint32_t kTileBytes = kHalves * 128u * 128u;
    // A Q tile is two (d = 64: one) boxes of 128 rows x 128 bytes.  A K or V tile is
    // made of groups of 8 rows, the group's first halves and then its second ones (8
    // rows x 128 bytes each, a swizzle atom): so one box brings a whole page, in the
    // order it lies in memory, and the MMA still finds each half's atoms evenly spaced.
    static constexpr uint32_t kQBoxBytes = 128u * 128u;
    static constexpr uint32_t kGroupBytes = kHalves * 1024u;
    static constexpr int kStages = D == 128 ? 4 : 8;    // a power of two: slots and phases are bits of the load's number
    static constexpr int kStageBits = D == 128 ? 2 : 3;
    static constexpr int kPairs = kStages / 2, kPairBits = kStageBits - 1;  // a tile's K and V lie in one pair of slots
    static constexpr uint32_t kKVOff = 2 * kTileBytes;  // after the two Q tiles
    static constexpr uint32_t kBarOff = kKVOff + kStages * kTileBytes;
    static constexpr uint32_t kXchOff = kBarOff + 512;  // [2 S tiles][2 halves][128 rows] maxima, then sums
    static constexpr uint32_t kSumOff = kXchOff + 2 * 2048;
    static constexpr int kWork = 8;                       // pieces handed out and not yet taken by every role
    static constexpr uint32_t kWorkOff = kSumOff + 256;   // their descriptions
    static constexpr uint32_t kSmemBytes = kWorkOff + kWork * sizeof(Work) + 1024;
    static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
    static constexpr int kQF = 0;            // one for each Q tile
    static constexpr int kKVF = kQF + 2;
    static constexpr int kKVE = kKVF + kStages;
    static constexpr int kSF = kKVE + kStages;
    static constexpr int kPF = kSF + 2;
    static constexpr int kOF = kPF + 2;
    static constexpr int kQFree = kOF + 2;    // one for each Q tile: every S MMA of its piece is done
    static constexpr int kOFree = kQFree + 2; // one for each O: every softmax thread has read the piece's
    static constexpr int kWF = kOFree + 2;    // a piece's description is there
    static constexpr int kWE = kWF + kWork;   // ... has been read by the MMA thread and the softmax warps
    static constexpr int kDrain = kWE + kWork;
    static constexpr int kNumBars = kDrain + 1;
    static_assert(kNumBars * 8 + 8 <= 512, "barrier area");
    static_assert(sizeof(Stretch) + 8 * (kThreads / 32) <= 256, "scan area");
};

// The two warps that share rows (w and w + 4, pair w mod 4): named barriers 2 to
// 5, 64 threads each, returning whether `v` holds in all of them.  A pair votes
// after every wait, so that both its warps give up together; no barrier but the
// kernel's last one joins two pairs, which may give up at different places.
__device__ __forceinline__ bool pair_bar_and(int pair, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "barrier.cta.red.and.pred po, %2, 64, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(2 + pair)
        : "memory");
    return r != 0;
}

// Bits [0, n) of 64, n clamped.
__device__ __forceinline__ uint64_t columns(int n)
{
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

// The thread that issues the MMAs.  (Everything it does in a step is inlined: a
// lambda called from two places is not, and what it refers to then lives in memory.)
template <int D>
struct Issuer {
    using C = Cfg<D>;
    uint32_t tmem, bars;
    uint64_t dq0, dk0, dv0;  // descriptors of the first Q tile, K and V slot
    uint64_t lim_ns;
    volatile int *abort_flag;
    unsigned int *err;
    uint32_t q_use0 = 0, q_use1 = 0, p_use0 = 0, p_use1 = 0, o_use0 = 0, o_use1 = 0;  // uses of the Q tiles, of S and P, of O

    __device__ __forceinline__ bool wait(int bar, uint32_t phase, int site)
    {
        // (inlined here only: the issuer paces the short steps; the other roles' waits shrink the code by being called)
        return ptx::mbar_wait(bars + 8u * (uint32_t)bar, phase & 1, lim_ns, abort_flag, err, site);
    }
    __device__ __forceinline__ bool ready(int bar, uint32_t phase) { return ptx::mbar_test_wait(bars + 8u * (uint32_t)bar, phase & 1); }
    __device__ __forceinline__ void commit(int bar) { ptx::mma_commit(bars + 8u * (uint32_t)bar); }
    // The load numbered n has landed (tile i's K is load 2i, its V load 2i + 1); may be overwritten.
    __device__ __forceinline__ bool full(uint32_t n) { return wait(C::kKVF + (n & (C::kStages - 1)), n >> C::kStageBits, 0x71); }
    __device__ __forceinline__ void free_slot(uint32_t n) { commit(C::kKVE + (n & (C::kStages - 1))); }
    __device__ __forceinline__ bool q_full(int t) { return wait(C::kQF + t, t ? q_use1++ : q_use0++, 0x70); }
    __device__ __forceinline__ void q_free()
    {
        commit(C::kQFree + 0);
        commit(C::kQFree + 1);
    }
    __device__ __forceinline__ bool p_full(int t)
    {
        const bool got = wait(C::kPF + t, t ? p_use1++ : p_use0++, 0x72);
        ptx::tc_fence_after();
        return got;
    }
    // The piece that last used O has been read.
    __device__ __forceinline__ bool o_free(int o)
    {
        const uint32_t n = o ? o_use1++ : o_use0++;
        return n == 0 || wait(C::kOFree + o, n - 1, 0x73);
    }
    __device__ __forceinline__ void issue_qk(int t, int q_tile, int slot)
    {
        const uint64_t qa = dq0 + ((q_tile * C::kTileBytes) >> 4), kb = dk0 + ((slot * C::kTileBytes) >> 4);
        const uint32_t dst = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t q_off = ((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4;
            const uint32_t k_off = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
            ptx::mma_ss(dst, qa + q_off, kb + k_off, ptx::idesc_bf16_f32(128, 128, false), kk > 0);
        }
        commit(C::kSF + t);
    }
    __device__ __forceinline__ void issue_pv(int o, int t, int slot, bool acc)
    {
        const uint64_t vb = dv0 + ((slot * C::kTileBytes) >> 4);
        const uint32_t dst = tmem + (o ? C::kColO1 : C::kColO0), pa = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ts(dst, pa + kk * 8, vb + ((kk * 2 * C::kGroupBytes) >> 4), ptx::idesc_bf16_f32(128, D, true),
                        (acc || kk > 0) ? 1u : 0u);
    }
    // Key tile j of n against two row tiles, the piece's first tile being `done`: PV of
    // both, each followed by its S of the next tile.  (One copy for all slots: with the
    // descriptors as constants, a copy for each pair of slots, a step was no faster and
    // the code 2 KB larger.)
    __device__ __forceinline__ bool step(uint32_t done, int j, int n)
    {
        const int pair = (done + j) & (C::kPairs - 1), kV = 2 * pair + 1, kK = 2 * ((pair + 1) & (C::kPairs - 1));
        const uint32_t tile = done + j;
        const bool more = j + 1 < n;
        if (!wait(C::kKVF + kV, tile >> C::kPairBits, 0x71) || !p_full(0))
            return false;
        issue_pv(0, 0, kV, j > 0);
        if (more) {
            if (!wait(C::kKVF + kK, (tile + 1) >> C::kPairBits, 0x71))
                return false;
            issue_qk(0, 0, kK);
        } else {
            commit(C::kOF + 0);
        }
        if (!p_full(1))
            return false;
        issue_pv(1, 1, kV, j > 0);
        commit(C::kKVE + kV);
        if (more) {
            issue_qk(1, 1, kK);
            commit(C::kKVE + kK);
            if (j + 2 == n)
                q_free();  // that was the last S MMA
        } else {
            commit(C::kOF + 1);
        }
        return true;
    }
};

// What a softmax thread keeps of a row's tiles so far.
struct Row {
    float m, l;   // kept maximum in log2 units, this half's sum
    int allowed;  // keys [0, allowed) of the segment are visible
};

// The scores of this thread's 64 keys of a tile (half h of it), masked; their
// maximum is returned.  lim: keys of the tile that the row sees; held: keys of the
// tile.
__device__ __forceinline__ float read_scores(uint32_t tS, int h, int lim, int held, uint32_t (&s)[64])
{
    ptx::tc_fence_after();
    ptx::tmem_ld64(tS + 64 * h, s);
    ptx::tmem_ld_wait64(s);
    if (lim < kTileKeys) {
        // Column c is key c, except in the last group of 8 of a shorter tile: its
        // keys end where the group ends (see the producer).
        const int last = (held - 1) & ~7, gap = last + 8 - held;
        const uint64_t seen = columns(min(lim, last) - 64 * h) |
                              (columns(min(lim + gap, last + 8) - 64 * h) & ~columns(last + gap - 64 * h));
        const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (!(lo & (1u << i)))
                s[i] = f2u(-INFINITY);
            if (!(hi & (1u << i)))
                s[i + 32] = f2u(-INFINITY);
        }
    }
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 64; i += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            m4[k] = fmax3(m4[k], u2f(s[i + 2 * k]), u2f(s[i + 2 * k + 1]));
    }
    return fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
}

// The maximum moves only when it grows by more than kRescale: l and, if a PV has
// written it (`old_o`), this half's columns of O are then multiplied by what 2^-m
// became.
template <int D>
__device__ __forceinline__ void raise_max(Row &r, float mnew, uint32_t tO, int h, bool old_o)
{
    const bool need = mnew > -INFINITY && (r.m == -INFINITY || mnew > r.m + kRescale);
    if (!__any_sync(0xffffffffu, need))
        return;
    float alpha = 1.f;
    if (need) {
        alpha = r.m == -INFINITY ? 0.f : ptx::ex2(r.m - mnew);
        r.l *= alpha;
        r.m = mnew;
    }
    if (old_o) {
        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
        for (int k = 0; k < D / 64; ++k) {
            uint32_t o[32];
            const uint32_t ta = tO + h * (D / 2) + k * 32;
            ptx::tmem_ld32(ta, o);
            ptx::tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 y = __fmul2_rn(make_float2(u2f(o[i]), u2f(o[i + 1])), a2);
                o[i] = f2u(y.x);
                o[i + 1] = f2u(y.y);
            }
            ptx::tmem_st32(ta, o);
        }
    }
}

// p = 2^(s log2(e) / sqrt(d) - m), rounded to bf16 for the MMA (the sum l takes
// them in fp32); keys [64h, 64h + 64) go to packed columns [32h, 32h + 32) over S,
// and `bar` learns that they are there.
__device__ __forceinline__ void write_probabilities(uint32_t tS, int h, float sl2, Row &r, const uint32_t (&s)[64], uint32_t bar)
{
    const float neg = r.m == -INFINITY ? 0.f : -r.m;
    const float2 c2 = make_float2(sl2, sl2), n2 = make_float2(neg, neg);
    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t pk[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float2 y = __ffma2_rn(make_float2(u2f(s[2 * i]), u2f(s[2 * i + 1])), c2, n2);
        const float p0 = ptx::ex2(y.x), p1 = ptx::ex2(y.y);
        acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(p0, p1));
        pk[i] = pack_bf16(p0, p1);
    }
    ptx::tmem_st32(tS + 32 * h, pk);
    ptx::tmem_st_wait();
    ptx::tc_fence_before();
    ptx::mbar_arrive(bar);
    const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
    r.l += a.x + a.y;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k8,
                       const __grid_constant__ CUtensorMap tm_v8, const __grid_constant__ PrefixAttnParams p)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sQ = base, sKV = base + C::kKVOff, bars = base + C::kBarOff;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + C::kBarOff + 8 * C::kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + C::kBarOff + 8 * C::kNumBars + 4);
    auto BAR = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = blockIdx.x;
    const int TT = p.light_tokens;  // tokens of a row tile
    const uint64_t lim_ns = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(BAR(C::kKVF + s), 1);
            ptx::mbar_init(BAR(C::kKVE + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(BAR(C::kSF + t), 1);
            ptx::mbar_init(BAR(C::kPF + t), C::kSoftmaxThreads);
            ptx::mbar_init(BAR(C::kOF + t), 1);
            ptx::mbar_init(BAR(C::kQF + t), 1);
            ptx::mbar_init(BAR(C::kQFree + t), 1);
            ptx::mbar_init(BAR(C::kOFree + t), C::kSoftmaxThreads);
        }
        for (int i = 0; i < C::kWork; ++i) {
            ptx::mbar_init(BAR(C::kWF + i), 1);
            ptx::mbar_init(BAR(C::kWE + i), 1 + C::kSoftmaxThreads / 32);
        }
        ptx::mbar_init(BAR(C::kDrain), 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == C::kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (warp == C::kProducerWarp && lane == 0) {
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    int64_t *s_sum = reinterpret_cast<int64_t *>(gbase + C::kSumOff);
    const Stretch st = find_stretch<C::kThreads>(p, worker, s_sum, reinterpret_cast<Stretch *>(s_sum + C::kThreads / 32));
    ptx::launch_dependents();  // the joining launch finds its rows' pieces while this one computes
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    Work *work = reinterpret_cast<Work *>(gbase + C::kWorkOff);

    if (warp == C::kProducerWarp || warp == C::kValueWarp) {
        // ============================ producers =============================
        const bool values = warp == C::kValueWarp;  // V; the other one brings Q and K and hands out the pieces
        const int page = 1 << p.page_shift, per_tile = kTileKeys >> p.page_shift;
        const int none = (int)(p.n_pages * p.Hkv);  // outside the maps: zeros
        uint32_t ld = values, q_use[2] = {0, 0};  // (a tile's K is load 2i, its V load 2i + 1)
        int q_slot = 0;
        uint32_t pieces = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t phase, int site) {
            return __all_sync(0xffffffffu, ptx::mbar_wait_called(BAR(bar), phase & 1, lim_ns, abort_flag, p.err, site)) != 0;
        };
        Walk walk;
        Batch segments;
        walk.begin(st);
        Piece x;
        for (bool more = true; ok && more; ++pieces) {
            more = walk.next(p, x, [&](int i) { return segments.get(p, i); });
            const Work f = work_of(x, p);
            if (!values) {
                const int at = pieces % C::kWork;
                if (pieces >= C::kWork)
                    ok = wait(C::kWE + at, pieces / C::kWork - 1, 0x65);
                if (!ok)
                    break;
                if (lane == 0) {
                    if (more)
                        work[at] = f;
                    else
                        work[at].tiles = -1;
                    ptx::mbar_arrive(BAR(C::kWF + at));
                }
            }
            if (!more || f.tiles == 0)
                continue;
            // What this lane loads of a tile: a page of a full tile, a group of 8 rows of
            // the segment's last, shorter one.  Its page's id is read a tile ahead.
            auto key_of = [&](int held) { return lane * (held < kTileKeys ? 8 : page); };
            auto held_of = [&](int tile) { return min(kTileKeys, x.keys - tile * kTileKeys); };
            auto look = [&](int tile) {
                const int held = held_of(tile), key = key_of(held);
                return key < held ? x.pages[tile * per_tile + (key >> p.page_shift)] : 0;
            };
            int id = look(x.t0);
            const int q0 = f.two ? 0 : q_slot, q1 = f.two ? 2 : q_slot + 1;
#pragma unroll 1
            for (int t = q0; ok && !values && t < q1; ++t) {
                if (q_use[t] > 0)
                    ok = wait(C::kQFree + t, q_use[t] - 1, 0x61);
                if (!ok)
                    break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(BAR(C::kQF + t), (uint32_t)(C::kHalves * 128 * p.G * TT));
                    for (int b = 0; b < C::kHalves; ++b)
                        ptx::tma_load_4d(sQ + t * C::kTileBytes + b * C::kQBoxBytes, &tm_q, BAR(C::kQF + t), b * 64, 0, x.head,
                                         x.tok + (t - q0) * TT);
                }
                ++q_use[t];
            }
            if (!f.two)
                q_slot ^= 1;
            for (int i = 0; ok && i < f.tiles; ++i) {
                const int held = held_of(x.t0 + i), key = key_of(held);
                const bool full = held == kTileKeys;
                int row = none;  // (a group without keys, or of a page that is none: zeros)
                if (key < held) {
                    if (id >= 0 && id < p.n_pages)
                        row = id * p.Hkv + x.head;
                    else
                        record_bad_index(p.err, kSiteCachePage, id);
                }
                // a group of v < 8 keys ends with them: its box starts 8 - v rows early, on
                // rows of the same page or, before its first, on zeros
                const int first = (key & (page - 1)) - max(0, key + 8 - held);
                if (i + 1 < f.tiles)
                    id = look(x.t0 + i + 1);
                // (K of keys that are none is not brought: their scores are masked whatever they are)
                const int groups = values ? kTileKeys / 8 : (held + 7) >> 3;
                const int slot = ld & (C::kStages - 1);
                const uint32_t use = ld >> C::kStageBits;
                if (use > 0)
                    ok = wait(C::kKVE + slot, use - 1, values ? 0x63 : 0x62);
                if (!ok)
                    break;
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(BAR(C::kKVF + slot), groups * C::kGroupBytes);
                __syncwarp();
                const uint32_t dst = sKV + slot * C::kTileBytes;
                if (full) {
                    if (lane < per_tile)
                        ptx::tma_load_5d(dst + lane * (page >> 3) * C::kGroupBytes, values ? &tm_v : &tm_k, BAR(C::kKVF + slot), 0, 0, 0,
                                         0, row);
                } else if (lane < groups) {
                    ptx::tma_load_4d(dst + lane * C::kGroupBytes, values ? &tm_v8 : &tm_k8, BAR(C::kKVF + slot), 0, first, 0, row);
                }
                ld += 2;
            }
        }
        // Every copy this warp started lands before the CTA can exit.
        volatile int no_abort = 0;
        for (int t = 0; t < 2; ++t)
            if (q_use[t] > 0)
                ptx::mbar_wait_called(BAR(C::kQF + t), (q_use[t] - 1) & 1, lim_ns, &no_abort, p.err, 0x64);
        for (uint32_t n = ld > C::kStages + values ? ld - C::kStages : values; n < ld; n += 2)  // the last load of each slot
            ptx::mbar_wait_called(BAR(C::kKVF + (n & (C::kStages - 1))), n >> C::kStageBits & 1, lim_ns, &no_abort, p.err, 0x64);
        __syncwarp();
    } else if (warp == C::kMmaWarp) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            Issuer<D> mma;
            mma.tmem = tmem;
            mma.bars = bars;
            mma.dq0 = ptx::smem_desc_sw128(sQ, 16, 1024);
            mma.dk0 = ptx::smem_desc_sw128(sKV, 16, C::kGroupBytes);
            mma.dv0 = ptx::smem_desc_sw128(sKV, 1024, C::kGroupBytes);
            mma.lim_ns = lim_ns;
            mma.abort_flag = abort_flag;
            mma.err = p.err;
            // The piece whose S MMAs are issued, and the one whose PVs are: the first is up
            // to two tiles ahead of the second, so at most three pieces lie after the second.
            uint32_t done = 0, ahead = 0;  // tiles whose PV, whose S has been issued
            uint32_t taken = 0;            // descriptions read
            int n = 0, two = 0, i = 0;     // the first's tiles (0: to be read, -1: none), form and tile
            int back_n = 0, back_i = 0, ahead0 = 0, ahead1 = 0, ahead2 = 0, waiting = 0;
            int q_slot = 0, o_slot = 0;
            bool ok = true;
            for (;;) {
                // ---- S, as far ahead as may be ----
                while (ok && n >= 0 && (n == 0 || (!two && ahead - done < 2))) {
                    if (n == 0) {
                        // (While a PV is to be issued only if the next piece is there: the
                        // producer may be waiting for the rows that this PV completes.)
                        const int at = taken % C::kWork;
                        if (ahead > done && !mma.ready(C::kWF + at, taken / C::kWork))
                            break;
                        ok = mma.wait(C::kWF + at, taken / C::kWork, 0x75);
                        if (!ok)
                            break;
                        n = work[at].tiles;
                        two = work[at].two;
                        ptx::mbar_arrive(BAR(C::kWE + at));
                        ++taken;
                        i = 0;
                        if (n != 0) {
                            ahead0 = waiting == 0 ? n : ahead0;
                            ahead1 = waiting == 1 ? n : ahead1;
                            ahead2 = waiting == 2 ? n : ahead2;
                            ++waiting;
                        }
                        continue;
                    }
                    ok = (i > 0 || mma.q_full(q_slot)) && mma.full(2 * ahead);
                    if (!ok)
                        break;
                    mma.issue_qk(ahead & 1, q_slot, (2 * ahead) & (C::kStages - 1));
                    mma.free_slot(2 * ahead);
                    ++ahead;
                    if (++i == n) {
                        mma.commit(C::kQFree + q_slot);
                        q_slot ^= 1;
                        n = 0;
                    }
                }
                if (!ok || (n < 0 && ahead == done))
                    break;
                if (back_i == back_n) {
                    back_i = 0;
                    back_n = ahead0;
                    ahead0 = ahead1;
                    ahead1 = ahead2;
                    --waiting;
                }
                if (n > 0 && two && ahead == done) {
                    // ---- a piece with two row tiles, by itself ----
                    ok = mma.q_full(0) && mma.q_full(1) && mma.full(2 * done);
                    if (!ok)
                        break;
                    const int first = (2 * done) & (C::kStages - 1);
                    mma.issue_qk(0, 0, first);
                    mma.issue_qk(1, 1, first);
                    mma.free_slot(2 * done);
                    if (n == 1)
                        mma.q_free();
                    ok = mma.o_free(0) && mma.o_free(1);
                    for (int j = 0; ok && j < n; ++j) {
                        ok = mma.step(done, j, n);
                    }
                    done += n;
                    ahead = done;
                    back_i = back_n;
                    n = 0;
                    continue;
                }
                // ---- PV of a piece with one row tile ----
                const uint32_t v = 2 * done + 1;
                ok = (back_i > 0 || mma.o_free(o_slot)) && mma.full(v) && mma.p_full(done & 1);
                if (!ok)
                    break;
                mma.issue_pv(o_slot, done & 1, v & (C::kStages - 1), back_i > 0);
                mma.free_slot(v);
                ++done;
                if (++back_i == back_n) {
                    mma.commit(C::kOF + o_slot);
                    o_slot ^= 1;
                }
            }
            if (taken > 0) {
                // Every MMA this thread issued has finished before TMEM is freed.
                mma.commit(C::kDrain);
                volatile int no_abort = 0;
                ptx::mbar_wait_called(BAR(C::kDrain), 0, lim_ns, &no_abort, p.err, 0x74);
            }
        }
        __syncwarp();
    } else {
        // ============================== softmax ==============================
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;  // half of the keys and columns, row of the tile
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float *xch = reinterpret_cast<float *>(gbase + C::kXchOff), *xl = xch + 512;
        const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(d)
        const int row_tok = row / p.G, row_g = row - row_tok * p.G;
        uint32_t done = 0;                                // tiles before this piece
        uint32_t s_use0 = 0, s_use1 = 0, o_use0 = 0, o_use1 = 0;  // uses of S and of O before now
        int o_slot = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t phase, int site) {
            return __all_sync(0xffffffffu, ptx::mbar_wait_called(BAR(bar), phase & 1, lim_ns, abort_flag, p.err, site)) != 0;
        };

        // The last piece's rows, whose O is still being computed while the next piece's
        // first scores are: written after those.
        struct {
            float m[2], l[2];  // of the row in each row tile
            int at, slot;      // its description; its first O
            bool on;
        } late;
        late.on = false;
        auto write_late = [&]() -> bool {
            late.on = false;
            const Work &w = work[late.at];
            const bool has_o = w.tiles > 0;
#pragma unroll 1
            for (int e = 0; e <= w.two; ++e) {
                const int ti = row_tok + e * TT, token = w.tok + ti, hq = w.head * p.G + row_g;
                const bool valid = row_tok < TT && ti < w.ntok, any = __any_sync(0xffffffffu, valid);
                const float m = e ? late.m[1] : late.m[0];
                float l = e ? late.l[1] : late.l[0];
                if (has_o) {
                    const bool got = wait(C::kOF + late.slot, late.slot ? o_use1++ : o_use0++, 0x81);
                    xl[(e * 2 + h) * 128 + row] = l;
                    if (!pair_bar_and(warp & 3, got))
                        return false;
                    ptx::tc_fence_after();
                    l += xl[(e * 2 + (h ^ 1)) * 128 + row];
                }
                const bool empty = !(l > 0.f) && l == l;
                const float inv = empty ? 0.f : 1.f / l;
                // where the row goes: the result, the worker's slot or the row's home
                const int64_t at = (int64_t)token * p.Hq + hq, own = (int64_t)worker * kPrefixUnitRows + (ti * p.G + row_g);
                const bool bf16 = w.to == kResult;
                float *po, *pl;
                if (w.to == kResult) {
                    po = reinterpret_cast<float *>(static_cast<__nv_bfloat16 *>(p.out) + at * D);
                    pl = p.lse + at;
                } else if (w.to == kSlot) {
                    po = p.slot_o + own * D;
                    pl = p.slot_lse + own;
                } else {
                    po = p.home_o[w.to] + at * D;
                    pl = p.home_lse[w.to] + at;
                }
                if (valid && h == 0)
                    *pl = empty ? -INFINITY : (m + ptx::lg2(l)) * kLn2;
                if (any) {
#pragma unroll 1
                    for (int k = 0; k < D / 64; ++k) {
                        const int col = h * (D / 2) + k * 32;
                        uint32_t o[32];
                        if (has_o) {
                            ptx::tmem_ld32(lanes + (late.slot ? C::kColO1 : C::kColO0) + col, o);
                            ptx::tmem_ld_wait(o);
                        }
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = has_o ? u2f(o[i]) * inv : 0.f;
                        if (valid) {
                            if (bf16) {
                                uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(po) + col);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    dst[i] =
                                        make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                                   pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                            } else {
                                float4 *dst = reinterpret_cast<float4 *>(po + col);
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (has_o) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(BAR(C::kOFree + late.slot));
                }
                late.slot ^= 1;
            }
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(BAR(C::kWE + late.at));
            return true;
        };

        for (uint32_t pieces = 0; ok; ++pieces) {
            const int at = pieces % C::kWork;
            ok = pair_bar_and(warp & 3, wait(C::kWF + at, pieces / C::kWork, 0x83));
            if (!ok)
                break;
            const Work &f = work[at];  // given back when its rows have been written
            const int tiles = max(f.tiles, 0), t0 = f.t0, keys = f.keys;
            const bool two = f.two != 0, last = f.tiles < 0;
            Row r[2];  // of the two row tiles; with one, of it
            uint32_t s[64];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                // A lane without a row need not mask anything: what it computes reaches
                // only the same lane's O, which nobody reads.
                const int ti = row_tok + (two ? t * TT : 0);
                const bool has = row_tok < TT && ti < f.ntok;
                r[t] = Row{-INFINITY, 0.f, has ? (int)max((int64_t)0, min((int64_t)keys, f.see0 + ti)) : INT_MAX};
            }
            if (two && tiles > 0) {
                if (late.on)
                    ok = write_late();
                for (int j = 0; ok && j < tiles; ++j) {
                    const int key0 = (t0 + j) * kTileKeys;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const bool busy = __any_sync(0xffffffffu, r[t].allowed != INT_MAX);
                        float mx = -INFINITY;
                        const bool got = wait(C::kSF + t, (t ? s_use1 : s_use0) + j, 0x80);
                        if (got && busy) {
                            mx = read_scores(lanes + (t ? C::kColS1 : C::kColS0), h, r[t].allowed - key0,
                                             min(kTileKeys, keys - key0), s);
                            xch[(t * 2 + h) * 128 + row] = mx;
                        }
                        // Both halves of the rows have read S before P is written over it.
                        ptx::tc_fence_before();
                        ok = pair_bar_and(warp & 3, got);
                        ptx::tc_fence_after();
                        if (!ok)
                            break;
                        if (busy) {
                            mx = fmaxf(mx, xch[(t * 2 + (h ^ 1)) * 128 + row]) * sl2;
                            // (the commit that signalled this S also covered the PV before it: O is stable)
                            raise_max<D>(r[t], mx, lanes + (t ? C::kColO1 : C::kColO0), h, j > 0);
                            write_probabilities(lanes + (t ? C::kColS1 : C::kColS0), h, sl2, r[t], s, BAR(C::kPF + t));
                        } else {
                            // (rows of P that nobody wrote only reach the same rows of O)
                            ptx::mbar_arrive(BAR(C::kPF + t));
                        }
                    }
                }
                s_use0 += tiles;
                s_use1 += tiles;
            } else {
                const bool busy = __any_sync(0xffffffffu, r[0].allowed != INT_MAX);
#pragma unroll 1
                for (int j = 0; ok && (j < tiles || late.on); ++j) {
                    if (j < tiles) {
                        const int key0 = (t0 + j) * kTileKeys, t = (done + j) & 1;
                        const uint32_t tS = lanes + (t ? C::kColS1 : C::kColS0);
                        float mx = -INFINITY;
                        const bool got = wait(C::kSF + t, t ? s_use1++ : s_use0++, 0x80);
                        if (got && busy) {
                            mx = read_scores(tS, h, r[0].allowed - key0, min(kTileKeys, keys - key0), s);
                            xch[(t * 2 + h) * 128 + row] = mx;
                        }
                        ptx::tc_fence_before();
                        ok = pair_bar_and(warp & 3, got);
                        ptx::tc_fence_after();
                        if (!ok)
                            break;
                        if (busy) {
                            mx = fmaxf(mx, xch[(t * 2 + (h ^ 1)) * 128 + row]) * sl2;
                            if (j > 0 && __any_sync(0xffffffffu, mx > r[0].m + kRescale)) {
                                // O may still be under the PV of the tile before: that one frees its V slot.
                                const uint32_t v = 2 * (done + j) - 1;
                                ok = pair_bar_and(warp & 3, wait(C::kKVE + (v & (C::kStages - 1)), v >> C::kStageBits, 0x82));
                                if (!ok)
                                    break;
                                ptx::tc_fence_after();
                            }
                            raise_max<D>(r[0], mx, lanes + (o_slot ? C::kColO1 : C::kColO0), h, j > 0);
                            write_probabilities(tS, h, sl2, r[0], s, BAR(C::kPF + t));
                        } else {
                            ptx::mbar_arrive(BAR(C::kPF + t));
                        }
                    }
                    if (late.on)
                        ok = write_late();
                }
            }
            if (!ok || last)
                break;
            done += tiles;
            late.at = at;
            late.m[0] = r[0].m;
            late.l[0] = r[0].l;
            late.m[1] = r[1].m;
            late.l[1] = r[1].l;
            late.slot = two ? 0 : o_slot;
            late.on = true;
            if (tiles > 0 && !two)
                o_slot ^= 1;
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch(const PrefixAttnParams &p_in, cudaStream_t s)
{
    PrefixAttnParams p = p_in;
    const int TT = 128 / p.G;
    p.unit_tokens = 2 * TT;
    p.light_tokens = TT;
    p.light_tile = kLightTile;
    p.heavy_tile = kHeavyTile;
    CUtensorMap mq, mk, mv, mk8, mv8;
    const uint64_t page = 1ull << p.page_shift, heads = (uint64_t)(p.n_pages * p.Hkv), halves = D / 64;
    const uint64_t qd[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.Hkv, (uint64_t)p.T};
    const uint64_t qs[3] = {(uint64_t)p.q_head_stride * 2, (uint64_t)p.G * p.q_head_stride * 2, (uint64_t)p.q_token_stride * 2};
    const uint32_t qb[4] = {64, (uint32_t)p.G, 1, (uint32_t)TT};
    // A page of a key head as [group of 8 rows][half][row][64]; 8 rows of it as [half][row][64].
    const uint64_t kd[5] = {64, 8, halves, page / 8, heads};
    const uint64_t ks[4] = {D * 2, 128, D * 16, page * D * 2};
    const uint32_t kb[5] = {64, 8, (uint32_t)halves, (uint32_t)page / 8, 1};
    const uint64_t gd[4] = {64, page, halves, heads};
    const uint64_t gs[3] = {D * 2, 128, page * D * 2};
    const uint32_t gb[4] = {64, 8, (uint32_t)halves, 1};
    if (!make_bf16_map_sw128(&mq, p.q, 4, qd, qs, qb) || !make_bf16_map_sw128(&mk, p.k_cache, 5, kd, ks, kb) ||
        !make_bf16_map_sw128(&mv, p.v_cache, 5, kd, ks, kb) || !make_bf16_map_sw128(&mk8, p.k_cache, 4, gd, gs, gb) ||
        !make_bf16_map_sw128(&mv8, p.v_cache, 4, gd, gs, gb))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg<D>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    prefix_attn_kernel<D><<<p.workers, Cfg<D>::kThreads, Cfg<D>::kSmemBytes, s>>>(mq, mk, mv, mk8, mv8, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_prefix_join(p, s);
}

}  // namespace

cudaError_t launch_prefix_attn_bf16(const PrefixAttnParams &p, cudaStream_t s)
{
    if (p.d == 128)
        return launch<128>(p, s);
    if (p.d == 64)
        return launch<64>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace rsa
