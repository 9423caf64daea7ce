// Attention of packed query rows over a shared prefix and their requests' own
// paged keys, on the sm_103a tensor cores (bf16).
//
//   o = softmax([q Kp^T, q Kr^T] / sqrt(d)) [Vp; Vr], by pieces of the keys
// whose (o, lse) the joining launch puts together (prefix_attn_f32.cu).
//
// One CTA on each SM takes an equal stretch of all key tiles (paged_sched.cuh)
// and goes through its pieces.  Warp roles as in the block kernel:
//   warp 8      producer: the piece's query rows (one 4-D TMA box a 128-row
//               tile: G heads of floor(128 / G) tokens, so any group size is
//               loaded without a gather), then K and V tiles through a ring of
//               shared-memory slots, one TMA box a page and 64 columns, each
//               lane loading the page whose id it read from the table one tile
//               ahead.
//   warp 9      one thread issues the MMAs: S_t = Q K^T from shared memory,
//               O_t += P_t V with P in TMEM.
//   warps 0-7   softmax on S_0 and S_1 in turn, two threads a row.
// A piece runs in one of two forms, by its number of rows:
//   two tiles   more than 128 rows: S_0 and S_1 are the two row tiles against
//               the same key tile, as in the block kernel, so that a key tile
//               serves 256 rows; bound by the softmax chain of each tile.
//   one tile    up to 128 rows: S_0 and S_1 are the same rows against the even
//               and the odd key tiles, two independent chains that keep the
//               loads going; their (m, l, O) lie in the same TMEM lanes and are
//               put together by the thread that owns the row.  Warps without a
//               row of the piece only keep the barriers' count, so a decode
//               step's few rows cost little and HBM is the bound.
// Rows past the keys are not trusted: a score of such a key is masked, but its
// 0 * NaN would reach O through V.  So they are never loaded: a tile's boxes of
// pages it does not have lie outside the tensor map, which fills them with
// zeros, and the box of a page that is v < page keys long starts v - page rows
// before the page, so that its first page - v rows are zeros and its keys end
// where the box ends.  The softmax masks those columns; the keys' order within
// a tile does not matter to it.
// The phases of all barriers run on over the CTA's pieces; one-tile pieces take
// the two Q tiles in turn, so that the next piece's loads are under way while
// one computes; O is written again once every softmax thread has read it.
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
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
    static constexpr int kSoftmaxThreads = 256;
    static constexpr int kProducerWarp = 8;
    static constexpr int kMmaWarp = 9;
    static constexpr int kThreads = 320;
    static constexpr int kBoxes = D / 64;               // 128-byte-wide boxes of a tile
    static constexpr uint32_t kBoxBytes = 128u * 128u;  // 128 rows x 128 bytes
    static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
    static constexpr int kStages = D == 128 ? 4 : 8;    // a power of two: slots and phases are bits of the load's number
    static constexpr int kStageBits = D == 128 ? 2 : 3;
    static constexpr uint32_t kKVOff = 2 * kTileBytes;  // after the two Q tiles
    static constexpr uint32_t kBarOff = kKVOff + kStages * kTileBytes;
    static constexpr uint32_t kXchOff = kBarOff + 256;  // [2 streams][2 halves][128 rows] maxima, then sums
    static constexpr uint32_t kSumOff = kXchOff + 2 * 2048;
    static constexpr uint32_t kSmemBytes = kSumOff + 256 + 1024;
    static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
    static constexpr int kQF = 0;            // one for each Q tile
    static constexpr int kKVF = kQF + 2;
    static constexpr int kKVE = kKVF + kStages;
    static constexpr int kSF = kKVE + kStages;
    static constexpr int kPF = kSF + 2;
    static constexpr int kOF = kPF + 2;
    static constexpr int kQFree = kOF + 2;    // one for each Q tile: every S MMA of its piece is done
    static constexpr int kOFree = kQFree + 2; // every softmax thread has read the piece's O
    static constexpr int kDrain = kOFree + 1;
    static constexpr int kNumBars = kDrain + 1;
    static_assert(kNumBars * 8 + 8 <= 256, "barrier area");
    static_assert(sizeof(Stretch) + 8 * (kThreads / 32) <= 256, "scan area");
};

// How a piece runs; every role works it out for itself.
struct Form {
    int tiles;   // key tiles that any of its rows sees
    bool two;    // two row tiles against each key tile
    int n[2];    // steps of S_0 and S_1
};

__device__ __forceinline__ Form form_of(const Piece &x, int tokens_per_tile)
{
    const int64_t seen = min((int64_t)x.keys, x.see0 + (x.ntok - 1));
    const int end = min(x.t1, seen > 0 ? (int)((seen + kTileKeys - 1) / kTileKeys) : 0);
    Form f;
    f.tiles = max(0, end - x.t0);
    f.two = x.ntok > tokens_per_tile;
    f.n[0] = f.two ? f.tiles : (f.tiles + 1) >> 1;
    f.n[1] = f.two ? f.tiles : f.tiles >> 1;
    return f;
}

// Bits [0, n) of 64, n clamped.
__device__ __forceinline__ uint64_t columns(int n)
{
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PrefixAttnParams p)
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
    const int TT = 128 / p.G, TU = 2 * TT;  // tokens of a row tile and of a unit
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
        }
        ptx::mbar_init(BAR(C::kOFree), C::kSoftmaxThreads);
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
    const Stretch st = find_stretch<C::kThreads>(p, TU, worker, s_sum, reinterpret_cast<Stretch *>(s_sum + C::kThreads / 32));
    ptx::launch_dependents();  // the joining launch finds its rows' pieces while this one computes
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    Walk walk;
    walk.begin(st);
    Piece x;

    if (warp == C::kProducerWarp) {
        // ============================= producer =============================
        const int page = 1 << p.page_shift, per_tile = kTileKeys >> p.page_shift;
        const int none = (int)(p.n_pages * p.Hkv);  // outside the maps: zeros
        uint32_t ld = 0, q_use[2] = {0, 0};
        int q_slot = 0;
        uint32_t landed[C::kStages];  // uses of each slot
        for (int s = 0; s < C::kStages; ++s)
            landed[s] = 0;
        bool ok = true;
        while (ok && walk.next(p, TU, x)) {
            const Form f = form_of(x, TT);
            if (f.tiles == 0)
                continue;
            // This lane's page of a tile: its row of the maps and the row of the page
            // the box starts at.
            auto page_row = [&](int tile, int &first) -> int {
                const int left = x.keys - tile * kTileKeys - (lane << p.page_shift);  // keys from this page on
                first = left < page ? left - page : 0;
                if (lane >= per_tile || left <= 0) {
                    first = 0;
                    return none;
                }
                const int id = x.pages[tile * per_tile + lane];
                if (id < 0 || id >= p.n_pages) {
                    record_bad_index(p.err, 0x55, id);
                    return none;
                }
                return id * p.Hkv + x.head;
            };
            int first, row = page_row(x.t0, first);
            const int q0 = f.two ? 0 : q_slot, q1 = f.two ? 2 : q_slot + 1;
#pragma unroll 1
            for (int t = q0; ok && t < q1; ++t) {
                if (q_use[t] > 0)
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(BAR(C::kQFree + t), (q_use[t] - 1) & 1, lim_ns, abort_flag,
                                                                p.err, 0x61));
                if (!ok)
                    break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(BAR(C::kQF + t), (uint32_t)(C::kBoxes * 128 * p.G * TT));
                    for (int b = 0; b < C::kBoxes; ++b)
                        ptx::tma_load_4d(sQ + t * C::kTileBytes + b * C::kBoxBytes, &tm_q, BAR(C::kQF + t), b * 64, 0, x.head,
                                         x.tok + (t - q0) * TT);
                }
                ++q_use[t];
            }
            if (!f.two)
                q_slot ^= 1;
            for (int i = 0; ok && i < f.tiles; ++i) {
                int next_first = 0;
                const int next_row = i + 1 < f.tiles ? page_row(x.t0 + i + 1, next_first) : none;
#pragma unroll 1
                for (int v = 0; v < 2; ++v, ++ld) {
                    const int slot = ld & (C::kStages - 1);
                    const uint32_t use = ld >> C::kStageBits;
                    if (use > 0)
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(BAR(C::kKVE + slot), (use - 1) & 1, lim_ns, abort_flag,
                                                                    p.err, 0x62));
                    if (!ok)
                        break;
                    if (lane == 0)
                        ptx::mbar_arrive_expect_tx(BAR(C::kKVF + slot), C::kTileBytes);
                    __syncwarp();
                    if (lane < per_tile)
#pragma unroll
                        for (int b = 0; b < C::kBoxes; ++b)
                            ptx::tma_load_3d(sKV + slot * C::kTileBytes + b * C::kBoxBytes + lane * page * 128,
                                             v ? &tm_v : &tm_k, BAR(C::kKVF + slot), b * 64, first, row);
                    landed[slot] = use + 1;
                }
                row = next_row;
                first = next_first;
            }
        }
        // Every copy this warp started lands before the CTA can exit.
        volatile int no_abort = 0;
        for (int t = 0; t < 2; ++t)
            if (q_use[t] > 0)
                ptx::mbar_wait(BAR(C::kQF + t), (q_use[t] - 1) & 1, lim_ns, &no_abort, p.err, 0x64);
        for (int s = 0; s < C::kStages; ++s)
            if (landed[s])
                ptx::mbar_wait(BAR(C::kKVF + s), (landed[s] - 1) & 1, lim_ns, &no_abort, p.err, 0x64);
        __syncwarp();
    } else if (warp == C::kMmaWarp) {
        // ============================ MMA issuer ============================
        if (lane == 0) {
            const uint32_t idesc_qk = ptx::idesc_bf16_f32(128, 128, false);
            const uint32_t idesc_pv = ptx::idesc_bf16_f32(128, D, true);
            const uint64_t dq0 = ptx::smem_desc_sw128(sQ, 16, 1024);
            const uint64_t dk0 = ptx::smem_desc_sw128(sKV, 16, 1024);
            const uint64_t dv0 = ptx::smem_desc_sw128(sKV, C::kBoxBytes, 1024);
            uint32_t ld = 0, pieces = 0, steps[2] = {0, 0};  // loads, pieces and S steps before this piece
            uint32_t q_use[2] = {0, 0};
            int q_slot = 0;
            bool ok = true, any = false;
            auto full = [&](uint32_t n) {  // the load numbered n has landed
                return ptx::mbar_wait(BAR(C::kKVF + (n & (C::kStages - 1))), (n >> C::kStageBits) & 1, lim_ns, abort_flag,
                                      p.err, 0x71);
            };
            auto free_slot = [&](uint32_t n) { ptx::mma_commit(BAR(C::kKVE + (n & (C::kStages - 1)))); };
            auto issue_qk = [&](int t, int q_tile, uint32_t n) {
                const uint64_t qa = dq0 + ((q_tile * C::kTileBytes) >> 4);
                const uint64_t kb = dk0 + (((n & (C::kStages - 1)) * C::kTileBytes) >> 4);
                const uint32_t dst = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
                    ptx::mma_ss(dst, qa + off, kb + off, idesc_qk, kk > 0);
                }
                ptx::mma_commit(BAR(C::kSF + t));
            };
            auto issue_pv = [&](int t, uint32_t n, bool acc) {
                const uint64_t vb = dv0 + (((n & (C::kStages - 1)) * C::kTileBytes) >> 4);
                const uint32_t dst = tmem + (t ? C::kColO1 : C::kColO0);
                const uint32_t pa = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    ptx::mma_ts(dst, pa + kk * 8, vb + ((kk * 2048) >> 4), idesc_pv, (acc || kk > 0) ? 1u : 0u);
            };
            auto p_full = [&](int t, int j) {
                const bool got = ptx::mbar_wait(BAR(C::kPF + t), (steps[t] + j) & 1, lim_ns, abort_flag, p.err, 0x72);
                ptx::tc_fence_after();
                return got;
            };
            while (ok && walk.next(p, TU, x)) {
                const Form f = form_of(x, TT);
                if (f.tiles == 0)
                    continue;
                const int n = f.tiles;
                any = true;
                // tile i's K is load ld + 2i, its V load ld + 2i + 1
                auto q_full = [&](int t) {
                    return ptx::mbar_wait(BAR(C::kQF + t), q_use[t]++ & 1, lim_ns, abort_flag, p.err, 0x70);
                };
                if (f.two) {
                    ok = q_full(0) && q_full(1) && full(ld);
                    if (!ok)
                        break;
                    issue_qk(0, 0, ld);
                    issue_qk(1, 1, ld);
                    free_slot(ld);
                    auto q_free = [&] {
                        ptx::mma_commit(BAR(C::kQFree + 0));
                        ptx::mma_commit(BAR(C::kQFree + 1));
                    };
                    if (n == 1)
                        q_free();
                    if (pieces > 0)
                        ok = ptx::mbar_wait(BAR(C::kOFree), (pieces - 1) & 1, lim_ns, abort_flag, p.err, 0x73);
                    for (int j = 0; ok && j < n; ++j) {
                        const uint32_t v = ld + 2 * j + 1, k = v + 1;
                        const bool more = j + 1 < n;
                        ok = full(v) && p_full(0, j);
                        if (!ok)
                            break;
                        issue_pv(0, v, j > 0);
                        if (more) {
                            ok = full(k);
                            if (!ok)
                                break;
                            issue_qk(0, 0, k);
                        } else {
                            ptx::mma_commit(BAR(C::kOF + 0));
                        }
                        ok = p_full(1, j);
                        if (!ok)
                            break;
                        issue_pv(1, v, j > 0);
                        free_slot(v);
                        if (more) {
                            issue_qk(1, 1, k);
                            free_slot(k);
                            if (j + 2 == n)
                                q_free();  // that was the last S MMA
                        } else {
                            ptx::mma_commit(BAR(C::kOF + 1));
                        }
                    }
                } else {
                    const int q = q_slot;
                    q_slot ^= 1;
                    ok = q_full(q) && full(ld);
                    if (!ok)
                        break;
                    issue_qk(0, q, ld);
                    free_slot(ld);
                    if (n > 1) {
                        ok = full(ld + 2);
                        if (!ok)
                            break;
                        issue_qk(1, q, ld + 2);
                        free_slot(ld + 2);
                    }
                    if (n <= 2)
                        ptx::mma_commit(BAR(C::kQFree + q));
                    if (pieces > 0)
                        ok = ptx::mbar_wait(BAR(C::kOFree), (pieces - 1) & 1, lim_ns, abort_flag, p.err, 0x73);
                    for (int i = 0; ok && i < n; ++i) {  // tile i is step i / 2 of stream i mod 2
                        const int t = i & 1;
                        const uint32_t v = ld + 2 * i + 1;
                        ok = full(v) && p_full(t, i >> 1);
                        if (!ok)
                            break;
                        issue_pv(t, v, i > 1);
                        free_slot(v);
                        if (i + 2 < n) {
                            const uint32_t k = ld + 2 * (i + 2);
                            ok = full(k);
                            if (!ok)
                                break;
                            issue_qk(t, q, k);
                            free_slot(k);
                            if (i + 3 == n)
                                ptx::mma_commit(BAR(C::kQFree + q));
                        } else {
                            ptx::mma_commit(BAR(C::kOF + t));
                        }
                    }
                }
                ld += 2 * n;
                steps[0] += f.n[0];
                steps[1] += f.n[1];
                ++pieces;
            }
            if (any) {
                // Every MMA this thread issued has finished before TMEM is freed.
                ptx::mma_commit(BAR(C::kDrain));
                volatile int no_abort = 0;
                ptx::mbar_wait(BAR(C::kDrain), 0, lim_ns, &no_abort, p.err, 0x74);
            }
        }
        __syncwarp();
    } else {
        // ============================== softmax ==============================
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;  // half of the keys and columns, row of the tile
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS[2] = {lanes + C::kColS0, lanes + C::kColS1}, tO[2] = {lanes + C::kColO0, lanes + C::kColO1};
        float *xch = reinterpret_cast<float *>(gbase + C::kXchOff), *xl = xch + 512;
        const float sl2 = 1.4426950408889634f / sqrtf((float)D);  // log2(e) / sqrt(d)
        const int row_tok = row / p.G, row_g = row - row_tok * p.G;
        uint32_t steps[2] = {0, 0}, drains[2] = {0, 0};
        bool ok = true;
        while (ok && walk.next(p, TU, x)) {
            const Form f = form_of(x, TT);
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // kept maxima in log2 units, this half's sums
            // Keys [0, allowed) of the segment are visible to the stream's row.  A lane
            // without a row need not mask anything: what it computes reaches only the
            // same lane's O, which nobody reads.
            int allowed[2];
            bool valid[2], busy[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int ti = row_tok + (f.two ? t * TT : 0);
                valid[t] = row_tok < TT && ti < x.ntok && (f.two || t == 0);
                const bool has = row_tok < TT && ti < x.ntok;
                allowed[t] = has ? (int)max((int64_t)0, min((int64_t)x.keys, x.see0 + ti)) : INT_MAX;
                busy[t] = __any_sync(0xffffffffu, has);
            }
            for (int j = 0; ok && j < f.n[0]; ++j) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t == 1 && j >= f.n[1])
                        continue;  // the same for every softmax thread
                    const int key0 = (x.t0 + (f.two ? j : 2 * j + t)) * kTileKeys;
                    uint32_t s[64];
                    float mx = -INFINITY;
                    bool got = true;
                    if (busy[t]) {
                        got = ptx::mbar_wait(BAR(C::kSF + t), (steps[t] + j) & 1, lim_ns, abort_flag, p.err, 0x80);
                        got = __all_sync(0xffffffffu, got);
                        if (got) {
                            ptx::tc_fence_after();
                            ptx::tmem_ld64(tS[t] + 64 * h, s);
                            ptx::tmem_ld_wait64(s);
                            const int lim = allowed[t] - key0;  // keys of the tile that the row sees
                            if (lim < kTileKeys) {
                                // Column c is key c, except in the segment's last page: its keys end
                                // where the page's box ends (see the producer).
                                const int page = 1 << p.page_shift, held = min(kTileKeys, x.keys - key0);
                                const int last = (held - 1) & ~(page - 1), gap = last + page - held;
                                const uint64_t seen = (columns(min(lim, last) - 64 * h) |
                                                       (columns(min(lim + gap, last + page) - 64 * h) &
                                                        ~columns(last + gap - 64 * h)));
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
                            mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
                            xch[(t * 2 + h) * 128 + row] = mx;
                        }
                    }
                    // Both halves of every row have read S (and know whether every wait
                    // succeeded) before P is written over it.
                    ptx::tc_fence_before();
                    ok = softmax_bar_and<256>(got);
                    ptx::tc_fence_after();
                    if (!ok)
                        break;
                    if (busy[t]) {
                        mx = fmaxf(mx, xch[(t * 2 + (h ^ 1)) * 128 + row]);
                        const float mnew = mx * sl2;
                        const bool need = mnew > -INFINITY && (m[t] == -INFINITY || mnew > m[t] + kRescale);
                        if (__any_sync(0xffffffffu, need)) {
                            float alpha = 1.f;
                            if (need) {
                                alpha = m[t] == -INFINITY ? 0.f : ptx::ex2(m[t] - mnew);
                                l[t] *= alpha;
                                m[t] = mnew;
                            }
                            if (j > 0) {
                                // the commit that signalled this S also covered the PV before it: O is stable
                                const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
                                for (int k = 0; k < D / 64; ++k) {
                                    uint32_t o[32];
                                    const uint32_t ta = tO[t] + h * (D / 2) + k * 32;
                                    ptx::tmem_ld32(ta, o);
                                    ptx::tmem_ld_wait(o);
#pragma unroll
                                    for (int i = 0; i < 32; i += 2) {
                                        const float2 r = __fmul2_rn(make_float2(u2f(o[i]), u2f(o[i + 1])), a2);
                                        o[i] = f2u(r.x);
                                        o[i + 1] = f2u(r.y);
                                    }
                                    ptx::tmem_st32(ta, o);
                                }
                            }
                        }
                        // p = 2^(s log2(e) / sqrt(d) - m), rounded to bf16 for the MMA (the sum l keeps
                        // them in fp32); keys [64h, 64h + 64) go to packed columns [32h, 32h + 32).
                        const float neg = m[t] == -INFINITY ? 0.f : -m[t];
                        const float2 c2 = make_float2(sl2, sl2), n2 = make_float2(neg, neg);
                        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                         make_float2(0.f, 0.f)};
                        uint32_t pk[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 y = __ffma2_rn(make_float2(u2f(s[2 * i]), u2f(s[2 * i + 1])), c2, n2);
                            const float p0 = ptx::ex2(y.x), p1 = ptx::ex2(y.y);
                            acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(p0, p1));
                            pk[i] = pack_bf16(p0, p1);
                        }
                        ptx::tmem_st32(tS[t] + 32 * h, pk);
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(BAR(C::kPF + t));
                        const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
                        l[t] += a.x + a.y;
                    } else {
                        // (rows of P that nobody wrote only reach the same rows of O)
                        ptx::mbar_arrive(BAR(C::kPF + t));
                    }
                }
            }
            if (!ok)
                break;
            // ---- the piece's (o, lse) ----
            bool fin = true;
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (f.n[t] > 0) {
                    fin = fin && ptx::mbar_wait(BAR(C::kOF + t), drains[t] & 1, lim_ns, abort_flag, p.err, 0x81);
                    fin = __all_sync(0xffffffffu, fin);
                    ++drains[t];
                    steps[t] += f.n[t];
                    xl[(t * 2 + h) * 128 + row] = l[t];
                }
            ok = softmax_bar_and<256>(fin);
            if (!ok)
                break;
            ptx::tc_fence_after();
            float inv[2] = {0.f, 0.f}, lse[2];  // weights of the unnormalised O, and the results' lse
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (f.n[t] > 0)
                    l[t] += xl[(t * 2 + (h ^ 1)) * 128 + row];
            if (f.two) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bool empty = !(l[t] > 0.f) && l[t] == l[t];
                    inv[t] = empty ? 0.f : 1.f / l[t];
                    lse[t] = empty ? -INFINITY : (m[t] + ptx::lg2(l[t])) * kLn2;
                }
            } else {
                const float M = fmaxf(m[0], m[1]);
                const float w0 = m[0] == -INFINITY ? 0.f : ptx::ex2(m[0] - M), w1 = m[1] == -INFINITY ? 0.f : ptx::ex2(m[1] - M);
                const float L = l[0] * w0 + l[1] * w1;
                const bool empty = !(L > 0.f) && L == L;
                inv[0] = empty ? 0.f : w0 / L;
                inv[1] = empty ? 0.f : w1 / L;
                lse[0] = empty ? -INFINITY : (M + ptx::lg2(L)) * kLn2;
                lse[1] = -INFINITY;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!f.two && t == 1)
                    continue;
                const int ti = row_tok + (f.two ? t * TT : 0);
                const int token = x.tok + ti;
                const int hq = x.head * p.G + row_g;
                const Place d = place(p, x, worker, token, hq, ti * p.G + row_g);
                if (valid[t] && h == 0)
                    *(d.final_ ? p.lse + ((int64_t)token * p.Hq + hq) : d.lse) = lse[t];
                if (!busy[t])
                    continue;  // the whole warp
#pragma unroll 1
                for (int k = 0; k < D / 64; ++k) {
                    const int col = h * (D / 2) + k * 32;
                    float v[32];
                    uint32_t o[32];
                    if (f.n[t] > 0) {
                        ptx::tmem_ld32(tO[t] + col, o);
                        ptx::tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = u2f(o[i]) * inv[t];
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = 0.f;
                    }
                    if (!f.two && f.n[1] > 0) {
                        ptx::tmem_ld32(tO[1] + col, o);
                        ptx::tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = fmaf(u2f(o[i]), inv[1], v[i]);
                    }
                    if (valid[t]) {
                        if (d.final_) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                                                   ((int64_t)token * p.Hq + hq) * D + col);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                dst[i] =
                                    make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                               pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(d.o + col);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (f.tiles > 0) {
                ptx::tc_fence_before();
                ptx::mbar_arrive(BAR(C::kOFree));
            }
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
cudaError_t launch(const PrefixAttnParams &p, cudaStream_t s)
{
    const int TT = 128 / p.G;
    CUtensorMap mq, mk, mv;
    const int64_t page = 1ll << p.page_shift;
    const uint64_t qd[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.Hkv, (uint64_t)p.T};
    const uint64_t qs[3] = {(uint64_t)p.q_head_stride * 2, (uint64_t)p.G * p.q_head_stride * 2, (uint64_t)p.q_token_stride * 2};
    const uint32_t qb[4] = {64, (uint32_t)p.G, 1, (uint32_t)TT};
    const uint64_t kd[3] = {(uint64_t)D, (uint64_t)page, (uint64_t)(p.n_pages * p.Hkv)};
    const uint64_t ks[2] = {(uint64_t)D * 2, (uint64_t)(page * D * 2)};
    const uint32_t kb[3] = {64, (uint32_t)page, 1};
    if (!make_bf16_map_sw128(&mq, p.q, 4, qd, qs, qb) || !make_bf16_map_sw128(&mk, p.k_cache, 3, kd, ks, kb) ||
        !make_bf16_map_sw128(&mv, p.v_cache, 3, kd, ks, kb))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg<D>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    prefix_attn_kernel<D><<<p.workers, Cfg<D>::kThreads, Cfg<D>::kSmemBytes, s>>>(mq, mk, mv, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_prefix_join(p, 2 * TT, s);
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
