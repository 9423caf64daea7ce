// C ABI of the paged-cache operators: a step's plan, the norm and rotation of
// its heads with the cache write, and attention behind a shared prefix.
#include <cmath>
#include <cstring>

#include "rsa_internal.h"

using namespace rsa;

namespace {

// log2 of a page size this library serves, or -1.
int page_shift_of(int page_size)
{
    switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    }
    return -1;
}

rsa_status check_index_ptr(const void *p, const char *name)
{
    if (!p)
        return fail(RSA_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 7u)
        return fail(RSA_ERR_INVALID_ARG, "%s is not 8-byte aligned", name);
    return RSA_OK;
}

rsa_status check_i32_ptr(const void *p, const char *name)
{
    if (!p)
        return fail(RSA_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u)
        return fail(RSA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return RSA_OK;
}

bool overlap(const void *a, int64_t an, const void *b, int64_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x && y && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

rsa_status check_dtype(rsa_dtype dt)
{
    if (dt != RSA_F32 && dt != RSA_BF16)
        return fail(RSA_ERR_INVALID_ARG, "dtype %d is not RSA_F32 or RSA_BF16", (int)dt);
    return RSA_OK;
}

rsa_status check_head_dim(int d)
{
    if (d != 64 && d != 128)
        return fail(RSA_ERR_UNSUPPORTED, "head dimension d=%d not supported (64 or 128)", d);
    return RSA_OK;
}

// Strides of a [T, H, d] operand: rows that start on 16 bytes.
rsa_status check_strides(rsa_dtype dt, int64_t token_stride, int64_t head_stride, int d, const char *name)
{
    const int64_t unit = dt == RSA_F32 ? 4 : 8;
    if (token_stride < d || head_stride < d || token_stride % unit || head_stride % unit)
        return fail(RSA_ERR_INVALID_ARG,
                    "%s has strides of %lld (token) and %lld (head) elements: at least d and multiples of 16 bytes are "
                    "wanted",
                    name, (long long)token_stride, (long long)head_stride);
    return RSA_OK;
}

rsa_status check_heads(const rsa_heads &h, rsa_dtype dt, int d, const char *name)
{
    RSA_TRY(check_ptr(h.data, name));
    return check_strides(dt, h.token_stride, h.head_stride, d, name);
}

// The same for a result: no two of its rows may overlap.
rsa_status check_result(const rsa_heads &h, rsa_dtype dt, int64_t T, int H, int d, const char *name)
{
    RSA_TRY(check_heads(h, dt, d, name));
    if (h.token_stride < (H - 1) * h.head_stride + d && h.head_stride < (T - 1) * h.token_stride + d)
        return fail(RSA_ERR_INVALID_ARG, "%s has overlapping rows (strides %lld and %lld)", name,
                    (long long)h.token_stride, (long long)h.head_stride);
    return RSA_OK;
}

HeadRows rows(const rsa_heads &h) { return HeadRows{h.data, h.token_stride, h.head_stride}; }

// The memory of an operand: T x H rows of `row` bytes, `token` and `head` bytes apart
// (a plain array is one row; nothing at 0).
struct Region {
    const char *name;
    int kind;  // a result may lie exactly on an input of the same kind (0: on none)
    int64_t at, end;  // the first row's beginning, the last one's end
    int64_t T, H, token, head, row;
};

constexpr int64_t kMostBytes = 1ll << 60;  // (more than an address space: sums and differences stay in 64 bits)

Region region(const char *name, const void *p, int64_t count, int64_t size)
{
    if (!p)
        return Region{};
    const int64_t bytes = count > kMostBytes / size ? kMostBytes : count * size, at = (int64_t) reinterpret_cast<uintptr_t>(p);
    return Region{name, 0, at, at + bytes, 1, 1, bytes, bytes, bytes};
}

Region region(const char *name, int kind, const rsa_heads &h, rsa_dtype dt, int64_t T, int64_t H, int d)
{
    if (!h.data)
        return Region{};
    const int64_t size = dt == RSA_F32 ? 4 : 2, at = (int64_t) reinterpret_cast<uintptr_t>(h.data);
    const __int128 n = ((__int128)(T - 1) * h.token_stride + (__int128)(H - 1) * h.head_stride + d) * size;
    auto bytes = [&](int64_t x) { return x > kMostBytes / size ? kMostBytes : x * size; };
    return Region{name, kind, at, at + (n > kMostBytes ? kMostBytes : (int64_t)n), T, H, bytes(h.token_stride), bytes(h.head_stride),
                  d * size};
}

bool same_rows(const Region &a, const Region &b)
{
    return a.at == b.at && a.T == b.T && a.H == b.H && (a.T == 1 || a.token == b.token) && (a.H == 1 || a.head == b.head);
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether a row of one lies on a row of the other.  Exact for rows with common strides,
// as cut from one packed buffer; of other regions that reach into one another it says yes.
bool rows_meet(Region a, Region b)
{
    if (a.end - a.at == kMostBytes || b.end - b.at == kMostBytes)
        return true;
    for (Region *r : {&a, &b}) {  // heads side by side are one row, tokens too
        if (r->head == r->row && r->H > 1) {
            r->row *= r->H;
            r->H = 1;
        }
        if (r->token == r->row && r->T > 1) {
            r->row *= r->T;
            r->T = 1;
        }
    }
    // the stride of a single token or head says nothing
    const int64_t token = a.T > 1 ? a.token : b.token, head = a.H > 1 ? a.head : b.head;
    if ((b.T > 1 && b.token != token) || (b.H > 1 && b.head != head))
        return true;
    // Row (t, h) of a lies on row (u, i) of b if -a.row < off + (t - u) token + (h - i) head < b.row.
    const int64_t off = a.at - b.at;
    auto meet = [&](int64_t x0, int64_t x1, int64_t x_stride, int64_t y0, int64_t y1, int64_t y_stride) {
        for (int64_t x = x0; x <= x1; ++x) {
            const int64_t at = off + x * x_stride;
            const int64_t lo = -floor_div(a.row - 1 + at, y_stride), hi = floor_div(b.row - 1 - at, y_stride);
            if (lo <= hi && lo <= y1 && hi >= y0)
                return true;
        }
        return false;
    };
    if (a.H + b.H <= a.T + b.T)
        return meet(1 - b.H, a.H - 1, head, 1 - b.T, a.T - 1, token);
    return meet(1 - b.T, a.T - 1, token, 1 - b.H, a.H - 1, head);
}

bool shares(const Region &a, const Region &b)
{
    return a.at < b.end && b.at < a.end && rows_meet(a, b);  // (what is not there ends at 0)
}

// No result shares memory with another operand, except exactly with its own input.
template <int kOut, int kIn>
rsa_status check_apart(const Region (&out)[kOut], const Region (&in)[kIn])
{
    for (int i = 0; i < kOut; ++i) {
        for (const Region &r : in)
            if (shares(out[i], r) && !(r.kind && r.kind == out[i].kind && same_rows(out[i], r)))
                return fail(RSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, r.name);
        for (int j = 0; j < i; ++j)
            if (shares(out[i], out[j]))
                return fail(RSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    }
    return RSA_OK;
}

rsa_status check_cache(int page_size, int64_t n_pages, int Hkv)
{
    if (page_shift_of(page_size) < 0)
        return fail(RSA_ERR_UNSUPPORTED, "page_size=%d not supported (16, 32, 64 or 128)", page_size);
    if (n_pages < 1 || n_pages > 0x7fffffffLL || n_pages * Hkv > 0x7fffffffLL)
        return fail(RSA_ERR_INVALID_ARG, "n_pages=%lld: at least 1 and at most 2^31-1 pages and key heads are wanted",
                    (long long)n_pages);
    return RSA_OK;
}

rsa_status norm_rope_params(const rsa_qk_norm_rope_args *a, NormRopeParams *p)
{
    if (!a)
        return fail(RSA_ERR_INVALID_ARG, "args is NULL");
    RSA_TRY(check_dtype(a->dt));
    if (a->T < 1 || a->Hq < 1 || a->Hkv < 1)
        return fail(RSA_ERR_INVALID_ARG, "T, Hq, Hkv must be >= 1 (got %lld, %d, %d)", (long long)a->T, a->Hq, a->Hkv);
    if (a->T > 0x7fffffffLL || (int64_t)a->Hq + 2ll * a->Hkv > 65536)
        return fail(RSA_ERR_UNSUPPORTED, "T=%lld or Hq + 2 Hkv too large", (long long)a->T);
    RSA_TRY(check_head_dim(a->d));
    RSA_TRY(check_heads(a->q, a->dt, a->d, "q"));
    RSA_TRY(check_heads(a->k, a->dt, a->d, "k"));
    if (a->q_weight)
        RSA_TRY(check_ptr(a->q_weight, "q_weight"));
    if (a->k_weight)
        RSA_TRY(check_ptr(a->k_weight, "k_weight"));
    if (!(a->eps >= 0.f) || std::isinf(a->eps))
        return fail(RSA_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", (double)a->eps);
    if (a->rot < 0 || a->rot > a->d || a->rot % 16)
        return fail(RSA_ERR_INVALID_ARG, "rot=%d must be a multiple of 16 in [0, d=%d]", a->rot, a->d);
    if (a->n_axes < 1 || a->n_axes > kMaxRopeAxes)
        return fail(RSA_ERR_INVALID_ARG, "n_axes=%d must be in [1, %d]", a->n_axes, kMaxRopeAxes);
    memset(p, 0, sizeof *p);
    if (a->rot > 0) {
        RSA_TRY(check_index_ptr(a->positions, "positions"));
        RSA_TRY(check_ptr(a->cos_sin, "cos_sin"));
        if (a->max_pos < 1)
            return fail(RSA_ERR_INVALID_ARG, "max_pos=%lld must be >= 1", (long long)a->max_pos);
        int at = 0;
        for (int i = 0; i < a->n_axes; ++i) {
            const int n = a->n_axes == 1 ? a->rot / 2 : a->sections[i];
            if (n < 0 || n > a->rot / 2)
                return fail(RSA_ERR_INVALID_ARG, "sections[%d]=%d is not in [0, rot/2=%d]", i, n, a->rot / 2);
            at += n;
            p->axis_end[i] = at;
        }
        if (at != a->rot / 2)
            return fail(RSA_ERR_INVALID_ARG, "sections add up to %d, not to rot/2=%d", at, a->rot / 2);
    }
    p->T = a->T;
    p->Hq = a->Hq;
    p->Hkv = a->Hkv;
    p->d = a->d;
    p->f32 = a->dt == RSA_F32;
    p->q = rows(a->q);
    p->k = rows(a->k);
    p->q_weight = a->q_weight;
    p->k_weight = a->k_weight;
    p->eps = a->eps;
    p->positions = a->positions;
    p->n_axes = a->n_axes;
    p->rot = a->rot;
    p->interleaved = a->interleaved ? 1 : 0;
    p->cos_sin = a->cos_sin;
    p->max_pos = a->max_pos;
    return RSA_OK;
}

// CTAs of the attention launch: the SMs of the current device.
rsa_status worker_count(int *n)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return fail(RSA_ERR_CUDA, "cannot query the SM count: %s", cudaGetErrorString(e));
    *n = sms < 1 ? 1 : (sms > kPrefixMaxWorkers ? kPrefixMaxWorkers : sms);
    return RSA_OK;
}

struct PrefixLayout {
    size_t plan, home_o, home_lse, slot_o, slot_lse, total;
};

PrefixLayout prefix_layout(int64_t T, int Hq, int d, int R)
{
    PrefixLayout w;
    const size_t rows_ = (size_t)T * Hq, slots = (size_t)kPrefixMaxWorkers * kPrefixUnitRows;
    w.plan = align256(((size_t)R + 2) * 8);
    w.home_o = align256(rows_ * d * 4);
    w.home_lse = align256(rows_ * 4);
    w.slot_o = align256(slots * d * 4);
    w.slot_lse = align256(slots * 4);
    w.total = w.plan + 2 * (w.home_o + w.home_lse) + w.slot_o + w.slot_lse;
    return w;
}

rsa_status check_prefix_shape(rsa_dtype dt, int64_t T, int Hq, int Hkv, int d, int R)
{
    RSA_TRY(check_dtype(dt));
    if (T < 1 || Hq < 1 || Hkv < 1 || R < 1)
        return fail(RSA_ERR_INVALID_ARG, "T, Hq, Hkv, R must be >= 1 (got %lld, %d, %d, %d)", (long long)T, Hq, Hkv, R);
    if (R > (1 << 30))
        return fail(RSA_ERR_UNSUPPORTED, "R=%d: more than 2^30 requests", R);
    if (Hq % Hkv)
        return fail(RSA_ERR_INVALID_ARG, "Hkv=%d does not divide Hq=%d", Hkv, Hq);
    RSA_TRY(check_head_dim(d));
    if (Hq / Hkv > kPrefixMaxGroup)
        return fail(RSA_ERR_UNSUPPORTED, "Hq / Hkv = %d exceeds %d query heads per key head", Hq / Hkv, kPrefixMaxGroup);
    if (T > (1ll << 30) || T * (int64_t)Hq > (1ll << 33))
        return fail(RSA_ERR_UNSUPPORTED, "T=%lld tokens of Hq=%d heads: too many rows", (long long)T, Hq);
    return RSA_OK;
}

}  // namespace

extern "C" {

rsa_status rsa_page_plan(const int32_t *cached_len, const int32_t *new_len, int R, int page_size, int64_t n_pages,
                         int32_t *block_table, int64_t table_stride, int max_pages, const int32_t *free_pages,
                         int64_t n_free, const int64_t *free_start, int64_t pos0, int64_t max_tokens, int32_t *cu_new,
                         int32_t *kv_len, int64_t *slot_map, int64_t *positions, int64_t *info, rsa_stream_t stream)
{
    if (R < 1 || max_tokens < 1 || max_pages < 1)
        return fail(RSA_ERR_INVALID_ARG, "R, max_tokens, max_pages must be >= 1 (got %d, %lld, %d)", R,
                    (long long)max_tokens, max_pages);
    if (R > kPagePlanMaxRequests)
        return fail(RSA_ERR_UNSUPPORTED, "R=%d exceeds %d requests", R, kPagePlanMaxRequests);
    RSA_TRY(check_cache(page_size, n_pages, 1));
    const int shift = page_shift_of(page_size);
    if (max_tokens > 0x7fffffffLL || n_free < 0 || n_free > 0x7fffffffLL || ((int64_t)max_pages << shift) > 0x7fffffffLL)
        return fail(RSA_ERR_INVALID_ARG, "max_tokens, n_free and max_pages * page_size must be in [0, 2^31-1]");
    if (table_stride < max_pages)
        return fail(RSA_ERR_INVALID_ARG, "table_stride=%lld is less than max_pages=%d", (long long)table_stride, max_pages);
    if (pos0 < 0)
        return fail(RSA_ERR_INVALID_ARG, "pos0=%lld must be >= 0", (long long)pos0);
    RSA_TRY(check_i32_ptr(cached_len, "cached_len"));
    RSA_TRY(check_i32_ptr(new_len, "new_len"));
    RSA_TRY(check_i32_ptr(block_table, "block_table"));
    if (n_free > 0)
        RSA_TRY(check_i32_ptr(free_pages, "free_pages"));
    if (free_start)
        RSA_TRY(check_index_ptr(free_start, "free_start"));
    RSA_TRY(check_i32_ptr(cu_new, "cu_new"));
    RSA_TRY(check_i32_ptr(kv_len, "kv_len"));
    RSA_TRY(check_ptr(slot_map, "slot_map"));
    RSA_TRY(check_ptr(positions, "positions"));
    RSA_TRY(check_index_ptr(info, "info"));
    // Every block reads the inputs while others write the outputs.
    const struct {
        const void *p;
        int64_t n;
        const char *name;
    } ins[] = {{cached_len, R * 4ll, "cached_len"}, {new_len, R * 4ll, "new_len"}, {free_pages, n_free * 4, "free_pages"},
               {free_start, 8, "free_start"}},
      outs[] = {{block_table, ((R - 1) * table_stride + max_pages) * 4, "block_table"},
                {cu_new, (R + 1) * 4ll, "cu_new"}, {kv_len, R * 4ll, "kv_len"}, {slot_map, max_tokens * 8, "slot_map"},
                {positions, max_tokens * 8, "positions"}, {info, 32, "info"}};
    for (const auto &o : outs) {
        for (const auto &i : ins)
            if (overlap(o.p, o.n, i.p, i.n))
                return fail(RSA_ERR_INVALID_ARG, "%s overlaps %s", o.name, i.name);
        for (const auto &q : outs)
            if (&q != &o && overlap(o.p, o.n, q.p, q.n))
                return fail(RSA_ERR_INVALID_ARG, "%s overlaps %s", o.name, q.name);
    }
    PagePlanParams p;
    memset(&p, 0, sizeof p);
    p.cached_len = cached_len;
    p.new_len = new_len;
    p.R = R;
    p.page_shift = shift;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.block_table = block_table;
    p.table_stride = table_stride;
    p.free_pages = free_pages;
    p.n_free = n_free;
    p.free_start = free_start;
    p.pos0 = pos0;
    p.max_tokens = max_tokens;
    p.cu_new = cu_new;
    p.kv_len = kv_len;
    p.slot_map = slot_map;
    p.positions = positions;
    p.info = info;
    RSA_TRY(device_error_word(&p.err));
    rsa_status inj;
    if (injected_failure("page plan launch", &inj))
        return inj;
    cudaError_t e = launch_page_plan(p, stream);
    if (e != cudaSuccess)
        return fail(RSA_ERR_CUDA, "page plan launch: %s", cudaGetErrorString(e));
    return RSA_OK;
}

rsa_status rsa_qk_norm_rope_fwd(const rsa_qk_norm_rope_args *args, rsa_heads q_out, rsa_heads k_out, rsa_heads v,
                                const int64_t *slot_map, void *k_cache, void *v_cache, int page_size, int64_t n_pages,
                                rsa_stream_t stream)
{
    NormRopeParams p;
    RSA_TRY(norm_rope_params(args, &p));
    RSA_TRY(check_result(q_out, args->dt, args->T, args->Hq, args->d, "q_out"));
    if (k_out.data || !slot_map)
        RSA_TRY(check_result(k_out, args->dt, args->T, args->Hkv, args->d, "k_out"));
    p.q_out = rows(q_out);
    p.k_out = rows(k_out);
    if (slot_map) {
        RSA_TRY(check_index_ptr(slot_map, "slot_map"));
        RSA_TRY(check_heads(v, args->dt, args->d, "v"));
        RSA_TRY(check_ptr(k_cache, "k_cache"));
        RSA_TRY(check_ptr(v_cache, "v_cache"));
        RSA_TRY(check_cache(page_size, n_pages, args->Hkv));
        p.slot_map = slot_map;
        p.v = rows(v);
        p.k_cache = k_cache;
        p.v_cache = v_cache;
        p.n_pages = n_pages;
        p.page_shift = page_shift_of(page_size);
    }
    // Rows are fetched some items ahead while other groups write theirs.
    const rsa_dtype dt = args->dt;
    const int64_t size = dt == RSA_F32 ? 4 : 2, T = args->T, cache = slot_map ? n_pages * args->Hkv * page_size * args->d : 0;
    const Region outs[] = {region("q_out", 1, q_out, dt, T, args->Hq, args->d), region("k_out", 2, k_out, dt, T, args->Hkv, args->d),
                           region("k_cache", p.k_cache, cache, size), region("v_cache", p.v_cache, cache, size)};
    const Region ins[] = {region("q", 1, args->q, dt, T, args->Hq, args->d), region("k", 2, args->k, dt, T, args->Hkv, args->d),
                          region("v", 0, slot_map ? v : rsa_heads{}, dt, T, args->Hkv, args->d),
                          region("q_weight", args->q_weight, args->d, size), region("k_weight", args->k_weight, args->d, size),
                          region("positions", args->rot ? args->positions : nullptr, args->n_axes * T, 8),
                          region("cos_sin", args->rot ? args->cos_sin : nullptr, args->max_pos, 4ll * args->rot),
                          region("slot_map", slot_map, T, 8)};
    RSA_TRY(check_apart(outs, ins));
    RSA_TRY(device_error_word(&p.err));
    rsa_status inj;
    if (injected_failure("head norm launch", &inj))
        return inj;
    cudaError_t e = launch_qk_norm_rope_fwd(p, stream);
    if (e != cudaSuccess)
        return fail(RSA_ERR_CUDA, "head norm launch: %s", cudaGetErrorString(e));
    return RSA_OK;
}

rsa_status rsa_qk_norm_rope_bwd_workspace_size(int d, size_t *bytes)
{
    if (!bytes)
        return fail(RSA_ERR_INVALID_ARG, "bytes is NULL");
    RSA_TRY(check_head_dim(d));
    *bytes = (size_t)kNormRopeBwdBlocks * 2 * d * 4;
    return RSA_OK;
}

rsa_status rsa_qk_norm_rope_bwd(const rsa_qk_norm_rope_args *args, rsa_heads dq_out, rsa_heads dk_out, rsa_heads dq,
                                rsa_heads dk, float *dq_weight, float *dk_weight, void *workspace, size_t ws_bytes,
                                rsa_stream_t stream)
{
    NormRopeParams p;
    RSA_TRY(norm_rope_params(args, &p));
    RSA_TRY(check_heads(dq_out, args->dt, args->d, "dq_out"));
    RSA_TRY(check_heads(dk_out, args->dt, args->d, "dk_out"));
    RSA_TRY(check_result(dq, args->dt, args->T, args->Hq, args->d, "dq"));
    RSA_TRY(check_result(dk, args->dt, args->T, args->Hkv, args->d, "dk"));
    if (dq_weight)
        RSA_TRY(check_ptr(dq_weight, "dq_weight"));
    if (dk_weight)
        RSA_TRY(check_ptr(dk_weight, "dk_weight"));
    size_t need = 0;
    RSA_TRY(rsa_qk_norm_rope_bwd_workspace_size(args->d, &need));
    RSA_TRY(check_ptr(workspace, "workspace"));
    if (ws_bytes < need)
        return fail(RSA_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
    p.dq_out = rows(dq_out);
    p.dk_out = rows(dk_out);
    p.q_out = rows(dq);
    p.k_out = rows(dk);
    p.partial = static_cast<float *>(workspace);
    p.dq_weight = dq_weight;
    p.dk_weight = dk_weight;
    const rsa_dtype dt = args->dt;
    const int64_t size = dt == RSA_F32 ? 4 : 2, T = args->T;
    const Region outs[] = {region("dq", 1, dq, dt, T, args->Hq, args->d), region("dk", 2, dk, dt, T, args->Hkv, args->d),
                           region("dq_weight", dq_weight, args->d, 4), region("dk_weight", dk_weight, args->d, 4),
                           region("workspace", workspace, (int64_t)need, 1)};
    const Region ins[] = {region("q", 1, args->q, dt, T, args->Hq, args->d), region("k", 2, args->k, dt, T, args->Hkv, args->d),
                          region("dq_out", 1, dq_out, dt, T, args->Hq, args->d), region("dk_out", 2, dk_out, dt, T, args->Hkv, args->d),
                          region("q_weight", args->q_weight, args->d, size), region("k_weight", args->k_weight, args->d, size),
                          region("positions", args->rot ? args->positions : nullptr, args->n_axes * T, 8),
                          region("cos_sin", args->rot ? args->cos_sin : nullptr, args->max_pos, 4ll * args->rot)};
    RSA_TRY(check_apart(outs, ins));
    RSA_TRY(device_error_word(&p.err));
    rsa_status inj;
    if (injected_failure("head norm backward launch", &inj))
        return inj;
    cudaError_t e = launch_qk_norm_rope_bwd(p, stream);
    if (e != cudaSuccess)
        return fail(RSA_ERR_CUDA, "head norm backward launch: %s", cudaGetErrorString(e));
    return RSA_OK;
}

rsa_status rsa_prefix_attn_workspace_size(rsa_dtype dt, int64_t T, int Hq, int Hkv, int d, int R, size_t *bytes)
{
    if (!bytes)
        return fail(RSA_ERR_INVALID_ARG, "bytes is NULL");
    RSA_TRY(check_prefix_shape(dt, T, Hq, Hkv, d, R));
    *bytes = prefix_layout(T, Hq, d, R).total;
    return RSA_OK;
}

rsa_status rsa_prefix_attn_fwd(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_cache,
                               const void *v_cache, rsa_dtype dt, int64_t T, int Hq, int Hkv, int d, int page_size,
                               int64_t n_pages, const int32_t *cu_q, const int32_t *kv_len, int R,
                               const int32_t *block_table, int64_t table_stride, int max_pages,
                               const int32_t *prefix_pages, int64_t prefix_len, void *out, float *lse, void *workspace,
                               size_t ws_bytes, rsa_stream_t stream)
{
    RSA_TRY(check_prefix_shape(dt, T, Hq, Hkv, d, R));
    RSA_TRY(check_cache(page_size, n_pages, Hkv));
    const int shift = page_shift_of(page_size);
    RSA_TRY(check_ptr(q, "q"));
    RSA_TRY(check_strides(dt, q_token_stride, q_head_stride, d, "q"));
    RSA_TRY(check_ptr(k_cache, "k_cache"));
    RSA_TRY(check_ptr(v_cache, "v_cache"));
    RSA_TRY(check_ptr(out, "out"));
    RSA_TRY(check_ptr(lse, "lse"));
    RSA_TRY(check_i32_ptr(cu_q, "cu_q"));
    RSA_TRY(check_i32_ptr(kv_len, "kv_len"));
    RSA_TRY(check_i32_ptr(block_table, "block_table"));
    if (max_pages < 1 || table_stride < max_pages || ((int64_t)max_pages << shift) > 0x7fffffffLL)
        return fail(RSA_ERR_INVALID_ARG,
                    "max_pages=%d (rows %lld apart): at least 1, at most the row and 2^31-1 keys are wanted", max_pages,
                    (long long)table_stride);
    if (prefix_len < 0 || prefix_len > (1ll << 31) - 128)  // (a tile's last key is still an int)
        return fail(RSA_ERR_INVALID_ARG, "prefix_len=%lld must be in [0, 2^31-128]", (long long)prefix_len);
    if (prefix_len > 0)
        RSA_TRY(check_i32_ptr(prefix_pages, "prefix_pages"));
    const PrefixLayout lay = prefix_layout(T, Hq, d, R);
    RSA_TRY(check_ptr(workspace, "workspace"));
    if (ws_bytes < lay.total)
        return fail(RSA_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu needed", ws_bytes, lay.total);
    // Rows are read again after others have been written; page ids are read while other
    // pieces' results are written, and the lengths by the joining launch again.
    const int64_t size = dt == RSA_F32 ? 4 : 2, cache = n_pages * Hkv * page_size * d * size;
    const struct {
        const void *p;
        int64_t n;
        const char *name;
    } bufs[] = {{q, ((T - 1) * q_token_stride + (Hq - 1) * q_head_stride + d) * size, "q"}, {k_cache, cache, "k_cache"},
                {v_cache, cache, "v_cache"}, {cu_q, (R + 1) * 4ll, "cu_q"}, {kv_len, R * 4ll, "kv_len"},
                {block_table, ((R - 1) * table_stride + max_pages) * 4, "block_table"},
                {prefix_len > 0 ? prefix_pages : nullptr, ((prefix_len + page_size - 1) >> shift) * 4, "prefix_pages"},
                {out, T * Hq * d * size, "out"}, {lse, T * Hq * 4, "lse"}, {workspace, (int64_t)lay.total, "workspace"}};
    for (int i = 7; i < 10; ++i)  // what is written
        for (int j = 0; j < i; ++j)
            if (overlap(bufs[i].p, bufs[i].n, bufs[j].p, bufs[j].n))
                return fail(RSA_ERR_INVALID_ARG, "%s overlaps %s", bufs[i].name, bufs[j].name);
    RSA_TRY(check_device_for(dt));
    PrefixAttnParams p;
    memset(&p, 0, sizeof p);
    p.q = q;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.d = d;
    p.f32 = dt == RSA_F32;
    p.n_pages = n_pages;
    p.page_shift = shift;
    p.cu_q = cu_q;
    p.kv_len = kv_len;
    p.R = R;
    p.block_table = block_table;
    p.table_stride = table_stride;
    p.max_pages = max_pages;
    p.prefix_pages = prefix_pages;
    p.prefix_len = prefix_len;
    p.out = out;
    p.lse = lse;
    char *w = static_cast<char *>(workspace);
    auto take = [&](size_t n) {
        char *at = w;
        w += n;
        return at;
    };
    p.plan = reinterpret_cast<int64_t *>(take(lay.plan));
    for (int i = 0; i < 2; ++i) {
        p.home_o[i] = reinterpret_cast<float *>(take(lay.home_o));
        p.home_lse[i] = reinterpret_cast<float *>(take(lay.home_lse));
    }
    p.slot_o = reinterpret_cast<float *>(take(lay.slot_o));
    p.slot_lse = reinterpret_cast<float *>(take(lay.slot_lse));
    RSA_TRY(worker_count(&p.workers));
    p.wait_limit_ns = wait_limit_ns();
    RSA_TRY(device_error_word(&p.err));
    rsa_status inj;
    if (injected_failure("prefix attention launch", &inj))
        return inj;
    cudaError_t e = dt == RSA_BF16 ? launch_prefix_attn_bf16(p, stream) : launch_prefix_attn_f32(p, stream);
    if (e != cudaSuccess)
        return fail(RSA_ERR_CUDA, "prefix attention launch: %s", cudaGetErrorString(e));
    return RSA_OK;
}

}  // extern "C"
