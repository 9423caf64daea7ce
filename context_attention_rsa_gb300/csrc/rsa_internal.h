// Internal declarations shared by the librsa translation units: launch
// parameter blocks, the launchers each kernel file exports, and status helpers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/rsa.h"

#define RSA_TRY(x)                     \
    do {                               \
        rsa_status st_ = (x);          \
        if (st_ != RSA_OK)             \
            return st_;                \
    } while (0)

namespace rsa {

// Device error word values.
constexpr unsigned int kDevErrTimeout = 0x100u;  // OR-ed with the wait's site code in the low byte
constexpr unsigned int kDevErrBounds = 0x200u;   // a bounds check failed (RSA_DEBUG build, or index data)

// The device-side error record.  Kernels get a pointer to `word` and OR codes
// into it.  The first failed bounds check since the record was cleared also
// leaves its site (never 0) and its index.
struct DeviceError {
    unsigned int word;
    unsigned int bad_site;
    long long bad_index;
};

// Record an index that lies outside its range: the first one's site code and
// value (any: -1 is as likely as another).  For index data that only the device
// sees (lengths, page ids, slots, positions), in every build; the caller skips
// the access.
__device__ __forceinline__ void record_bad_index(unsigned int *err, unsigned int site, long long idx)
{
    DeviceError *e = reinterpret_cast<DeviceError *>(err);
    if (atomicCAS(&e->bad_site, 0u, site) == 0u)
        e->bad_index = idx;
    atomicOr(&e->word, kDevErrBounds);
}

#ifdef RSA_DEBUG
// Bounds check of an RSA_DEBUG build: false (and recorded, without a trap) if
// `ok` is false; the caller then skips the access.
__device__ __forceinline__ bool debug_check(bool ok, unsigned int *err, unsigned int site, long long idx)
{
    if (!ok && err)
        record_bad_index(err, site, idx);
    return ok;
}
#define RSA_DCHECK(cond, err, site, idx) ::rsa::debug_check((cond), (err), (site), (long long)(idx))
#else
#define RSA_DCHECK(cond, err, site, idx) true
#endif

// Sites of index data (rsa.h names them; the other kernels' codes are all below 0x90).
constexpr unsigned int kSitePlanPage = 0x90, kSitePosition = 0x91, kSiteSlot = 0x92, kSiteQueryRows = 0x93, kSiteKvLen = 0x94,
                       kSiteCachePage = 0x95;

// Position axes of a rotation (time, height, width, one more).
constexpr int kMaxRopeAxes = 4;

// Most pairs one kernel launch takes; longer pair lists are split.
constexpr int kMaxPairsPerLaunch = 32;

// What a block-attention epilogue does with a pair's (o, lse).
enum EpilogueMode : int {
    kStore = 0,       // write (o, lse) to out/lse
    kMergeAcc = 1,    // fold into the fp32 accumulator in place: acc/lse <- merge(acc/lse, o/lse)
    kMergeFinal = 2,  // fold with the accumulator and write the result to out/lse (acc read only)
};

// One (query chunk, KV chunk) pair inside a block-attention launch.  Output
// row r of head bh goes to out[(bh * out_T + out_t0 + r) * d] and
// lse[bh * out_T + out_t0 + r]; a merging epilogue reads the accumulator row
// at the same index of `acc` (and the running lse from `lse`).
struct PairDesc {
    int64_t q_off;   // global position of the first query row
    int64_t q_row0;  // row of the first query inside each head of the Q tensor
    int64_t kv_off;  // global position of the first key (causal mask)
    int64_t kv_row0; // row of the first key inside each head of the K/V tensors
    void *out;       // bf16 or fp32 (out_f32)
    float *lse;
    int64_t out_T;   // row pitch of out/lse per head
    int64_t out_t0;  // first row of this pair inside each head
    int out_f32;     // 1: fp32 output, 0: bf16 output
    int mode;        // EpilogueMode
    const float *acc;  // fp32 accumulator (kMergeAcc: same as out; kMergeFinal: read only)
    int64_t split_stride;  // out/lse rows between consecutive key splits of this pair
    int64_t out_rows;      // rows out, lse (and acc) hold from their base pointers (bounds checks)
};

struct BlockParams {
    int B, H;
    int64_t T;              // rows per head of K and V
    int64_t q_T;            // rows per head of the Q tensor (T, or the decode rows)
    int d;
    int causal;
    int64_t q_len, kv_len;  // rows per pair, keys per pair
    int64_t kv_split;       // keys per split of a pair's key range (0: one split)
    int n_split;            // splits per pair; split s covers keys [s*kv_split, (s+1)*kv_split)
    int npairs;
    int n_qgroups;          // query-row groups per pair (rows per CTA granularity)
    uint64_t wait_limit_ns;
    int tc_kernel;          // tensor-core kernel choice: 0 automatic (one-SM), 1 one-SM, 2 two-SM where it applies
    int acc_staged;         // set by the one-SM launcher: merging epilogues read the accumulator staged by TMA
    unsigned int *err;      // device error word
    PairDesc pairs[kMaxPairsPerLaunch];
};

// One pair's rows inside a merge launch.  Row rr (0 <= rr < rows_per_pair)
// of the pair is head bh = rr / Tc, position t = rr % Tc; its accumulator row
// is bh * T + acc_t0 + t and its partial row is rr.
struct MergePair {
    int64_t acc_t0;
    const void *o_blk;
    const float *lse_blk;
    int final_;  // 1: write out/lse_out, 0: update o_acc/lse_acc in place
    int pad_;
};

struct MergeParams {
    int64_t rows_per_pair, Tc, T;
    int npairs, d;
    int blk_f32, out_f32;
    float *o_acc;
    float *lse_acc;
    void *out;
    float *lse_out;
    unsigned int *err;  // device error word (bounds checks of RSA_DEBUG builds)
    MergePair pairs[kMaxPairsPerLaunch];
};

// One step's plan over a paged cache (rsa_page_plan).
constexpr int kPagePlanMaxRequests = 16384;  // three ints a request in shared memory
struct PagePlanParams {
    const int32_t *cached_len, *new_len;
    int R, page_shift, max_pages;
    int64_t n_pages;
    int32_t *block_table;
    int64_t table_stride;
    const int32_t *free_pages;
    int64_t n_free;
    const int64_t *free_start;
    int64_t pos0, max_tokens;
    int32_t *cu_new, *kv_len;
    int64_t *slot_map, *positions, *info;
    unsigned int *err;
};

// A [T, H, d] operand of the head norm: rows of d contiguous elements, the
// strides of tokens and heads in elements.
struct HeadRows {
    void *data;
    int64_t token_stride, head_stride;
};

// Norm and rotation of query and key heads (rsa_qk_norm_rope_fwd and _bwd).
struct NormRopeParams {
    int64_t T;
    int Hq, Hkv, d, f32;
    HeadRows q, k, v;            // inputs (v only with a cache)
    HeadRows dq_out, dk_out;     // backward: gradients of the outputs
    HeadRows q_out, k_out;       // results (backward: gradients of the inputs); k_out.data may be NULL with a cache
    const void *q_weight, *k_weight;  // [d] of the inputs' type, or NULL for ones
    float eps;
    const int64_t *positions;    // [n_axes, T]
    int n_axes, rot, interleaved;
    int axis_end[kMaxRopeAxes];  // frequency pairs of axes 0..a end before axis_end[a]
    const float *cos_sin;        // [max_pos, rot]
    int64_t max_pos;
    const int64_t *slot_map;     // [T] or NULL: no cache
    void *k_cache, *v_cache;     // [n_pages, Hkv, page, d]
    int64_t n_pages;
    int page_shift;
    float *partial;              // backward: [blocks, 2, d]
    float *dq_weight, *dk_weight;  // backward: [d] each
    unsigned int *err;
};

// Attention of packed query rows over a shared prefix and their requests' own
// paged keys (rsa_prefix_attn_fwd).
struct PrefixAttnParams {
    const void *q;               // [T, Hq, d], strides in elements
    int64_t q_token_stride, q_head_stride;
    const void *k_cache, *v_cache;  // [n_pages, Hkv, page, d]
    int64_t T;
    int Hq, Hkv, G, d, f32;      // G = Hq / Hkv
    int64_t n_pages;
    int page_shift;
    const int32_t *cu_q, *kv_len;  // [R + 1], [R]
    int R;
    const int32_t *block_table;  // [R, max_pages], rows table_stride apart
    int64_t table_stride;
    int max_pages;
    const int32_t *prefix_pages;
    int64_t prefix_len;
    void *out;                   // [T, Hq, d]
    float *lse;                  // [T, Hq]
    // workspace (see paged_sched.cuh)
    int64_t *plan;               // [R + 2]
    float *home_o[2], *home_lse[2];  // [T * Hq, d] and [T * Hq]: a row's first piece of the prefix, of its own keys
    float *slot_o, *slot_lse;    // [workers, 256, d] and [workers, 256]: a worker's first piece, begun by another
    // how the launcher's kernel cuts the work
    int workers;
    int unit_tokens;             // query tokens of a unit at most
    int light_tokens;            // a unit of more tokens than this costs heavy_tile places a key tile, else light_tile
    int light_tile, heavy_tile;
    uint64_t wait_limit_ns;
    unsigned int *err;
};
constexpr int kPrefixMaxWorkers = 160;   // CTAs of the attention launch: one on each SM
constexpr int kPrefixUnitRows = 256;     // query rows of one unit at most
constexpr int kPrefixMaxGroup = 128;     // query heads per key head at most

// Launchers (no validation; the C ABI layer validates).  They return the
// cudaError_t of the launch.
cudaError_t launch_block_attn_bf16(const void *q, const void *k, const void *v,
                                   const BlockParams &p, cudaStream_t s);
cudaError_t launch_block_attn_f32(const float *q, const float *k, const float *v,
                                  const BlockParams &p, cudaStream_t s);
cudaError_t launch_merge(const MergeParams &p, cudaStream_t s);
// Fold S partials [S][rows][d] (fp32 o, fp32 lse) into out [rows][d] and lse [rows].
cudaError_t launch_merge_splits(const float *o_part, const float *lse_part, int S, int64_t rows, int d,
                                void *out, int out_f32, float *lse, cudaStream_t s);
cudaError_t launch_page_plan(const PagePlanParams &p, cudaStream_t s);
cudaError_t launch_qk_norm_rope_fwd(const NormRopeParams &p, cudaStream_t s);
// Two launches: gradients and partial sums, then the sums of the weights' gradients.
cudaError_t launch_qk_norm_rope_bwd(const NormRopeParams &p, cudaStream_t s);
constexpr int kNormRopeBwdBlocks = 304;  // blocks of partial weight gradients: two on each of 152 SMs
cudaError_t launch_prefix_attn_bf16(const PrefixAttnParams &p, cudaStream_t s);
cudaError_t launch_prefix_attn_f32(const PrefixAttnParams &p, cudaStream_t s);
// Joins the pieces of every row: the second launch of the attention.
cudaError_t launch_prefix_join(const PrefixAttnParams &p, cudaStream_t s);
cudaError_t launch_selftest_wait(uint64_t limit_ns, unsigned int *err, cudaStream_t s);
// Two-pass ring self-attention (bf16, d = 128, T/N a multiple of 128): per
// query chunk, score pass into S [BH, Tc, T] fp32 (and per-tile row
// statistics [BH, Tc, T/128] float2), row softmax into P [BH, Tc, T] bf16
// (and lse), output pass into out.
cudaError_t launch_two_pass(const void *q, const void *k, const void *v, int64_t BH, int64_t T, int N, int causal,
                            void *out, float *lse, float *S, void *P, void *stats, uint64_t wait_limit_ns,
                            unsigned int *err, cudaStream_t s);

// bf16 TMA tensor map with 128-byte swizzle: dims and box innermost first,
// strides in bytes for dimensions 1..rank-1.  False if the driver rejects it.
bool make_bf16_map_sw128(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims,
                         const uint64_t *strides_bytes, const uint32_t *box);
// The same for fp32 elements.
bool make_f32_map_sw128(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims,
                        const uint64_t *strides_bytes, const uint32_t *box);

// Rows of one CTA of the tensor-core kernel (two 128-row tiles).
constexpr int kBf16RowsPerCta = 256;
// Rows of one CTA pair of the two-SM tensor-core kernel.
constexpr int kBf16RowsPerCluster = 512;

// The two-SM kernel serves d = 128 launches without key splits whose pairs
// have at least one full cluster of rows; launch_block_attn_bf16 picks it for
// those when BlockParams::tc_kernel asks for it (2), else the one-SM kernel.
bool block_attn_2sm_applies(const BlockParams &p);
cudaError_t launch_block_attn_bf16_2sm(const void *q, const void *k, const void *v, const BlockParams &p,
                                       cudaStream_t s);

// Device address of the __device__ variable at host-side stand-in `symbol`
// in the calling thread's current CUDA context, looked up with
// cudaGetSymbolAddress once per context.  The cache is keyed by the driver's
// unique context id, so a context created later (after cudaDeviceReset, for
// instance) gets a fresh lookup instead of a stale address.
rsa_status symbol_address(const void *symbol, void **out);

// Host-side checks and state shared by the C ABI's translation units.
// True if this launch is to fail by rsa_debug_inject_launch_failure (and the
// failure has been recorded in *st).
bool injected_failure(const char *what, rsa_status *st);
// The device error word of the calling thread's current context.
rsa_status device_error_word(unsigned int **out);
// The limit of every device-side wait (rsa_set_wait_limit_ns).
uint64_t wait_limit_ns();
// The bf16 kernels are built for sm_103a only.
rsa_status check_device_for(rsa_dtype dt);
// A device pointer argument: not NULL and 16-byte aligned.
rsa_status check_ptr(const void *p, const char *name);

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Set the thread's last-error text and return `st`.
rsa_status fail(rsa_status st, const char *fmt, ...);

}  // namespace rsa
