// hq_serving_api.cu -- host side of the serving operators declared in
// include/hq.h: rotation tables, argument checks and dispatch.  No allocation,
// no synchronisation; everything is enqueued on the caller's stream.
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <utility>

#include <cuda_runtime.h>

#include "../../include/hq.h"
#include "hq_paged.h"

namespace {

using namespace hq;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// An array the kernels can read: 16-byte accesses at every row.
bool readable(const hq_rows *r, int64_t tokens, int64_t heads)
{
    if (!r || !r->p || (r->dtype != HQ_BF16 && r->dtype != HQ_F32) || !aligned(r->p, 16)) return false;
    const int64_t unit = r->dtype == HQ_F32 ? 4 : 8;
    for (auto [stride, extent] : { std::pair<int64_t, int64_t>{ r->token_stride, tokens }, { r->head_stride, heads } })
        if (extent > 1 && (stride < 0 || stride % unit || stride > INT64_MAX / 16 / extent)) return false;
    return true;
}

// One the kernels can write: rows do not overlap either.
bool writable(const hq_rows *r, int64_t tokens, int64_t heads, int64_t dim)
{
    if (!readable(r, tokens, heads)) return false;
    const int64_t ts = tokens > 1 ? r->token_stride : 0, hs = heads > 1 ? r->head_stride : 0;
    if (tokens > 1 && ts < dim) return false;
    if (heads > 1 && hs < dim) return false;
    return tokens <= 1 || heads <= 1 || ts >= (heads - 1) * hs + dim || hs >= (tokens - 1) * ts + dim;
}

Rows rows_of(const hq_rows *r, int64_t tokens, int64_t heads)
{
    return Rows{ r->p, tokens > 1 ? r->token_stride : 0, heads > 1 ? r->head_stride : 0, r->dtype == HQ_F32 };
}

int check_pages(const hq_pages *p)
{
    if (!p || !p->k || !p->v || !aligned(p->k, 16) || !aligned(p->v, 16)) return HQ_ERR_ARG;
    if (p->pages < 0 || p->heads < 1 || p->page_size < 1) return HQ_ERR_ARG;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return HQ_ERR_ARG;
    if (p->heads > 65535 || p->page_size < 16 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)))
        return HQ_ERR_UNSUPPORTED;
    if (p->pages >= ((int64_t)1 << 31) / p->page_size) return HQ_ERR_UNSUPPORTED;
    std::pair<int64_t, int64_t> d[3] = { { p->page_stride, p->pages }, { p->head_stride, p->heads },
                                         { p->slot_stride, p->page_size } };
    for (int i = 0; i < 3; i++)  // by stride
        for (int j = i + 1; j < 3; j++)
            if (d[j].first < d[i].first) std::swap(d[i], d[j]);
    int64_t span = p->head_dim;
    for (auto [stride, extent] : d) {
        if (extent <= 1) continue;
        if (stride % 8 || stride < span || stride > INT64_MAX / 16 / extent) return HQ_ERR_ARG;
        span += stride * (extent - 1);
    }
    return HQ_OK;
}

int log2_of(int v)
{
    int s = 0;
    while ((1 << s) < v) s++;
    return s;
}

bool valid_rotary(int r, int d) { return r >= 16 && r <= 256 && r % 16 == 0 && r <= d; }

}  // namespace

extern "C" {

int hq_rope_frequencies(int rotary_dim, double base, const hq_rope_scaling *scaling, double *theta, float *amplitude)
{
    if (!theta || !amplitude || !valid_rotary(rotary_dim, 256) || !std::isfinite(base) || base <= 1.0) return HQ_ERR_ARG;
    const int kind = scaling ? scaling->kind : HQ_ROPE_PLAIN;
    if (kind < HQ_ROPE_PLAIN || kind > HQ_ROPE_YARN) return HQ_ERR_ARG;
    const double r = rotary_dim, f = kind == HQ_ROPE_PLAIN ? 1.0 : scaling->factor;
    if (!std::isfinite(f) || f <= 0.0 || (kind == HQ_ROPE_YARN && f < 1.0)) return HQ_ERR_ARG;
    double low = 0.0, high = 0.0, original = 0.0;
    if (kind == HQ_ROPE_BANDS || kind == HQ_ROPE_YARN) {
        low = scaling->low;
        high = scaling->high;
        original = scaling->original;
        if (!std::isfinite(high) || !(low > 0.0) || !(high > low) || !std::isfinite(original) || original <= 0.0)
            return HQ_ERR_ARG;
    }
    if (kind == HQ_ROPE_NTK) base *= std::pow(f, r / (r - 2.0));
    if (!std::isfinite(base) || base <= 1.0) return HQ_ERR_ARG;
    // the pair that makes n turns in the original context
    auto pair_at = [&](double n) { return r * std::log(original / (2.0 * M_PI * n)) / (2.0 * std::log(base)); };
    *amplitude = kind == HQ_ROPE_YARN ? (float)(0.1 * std::log(f) + 1.0) : 1.0f;
    double from = 0.0, to = 0.0;
    if (kind == HQ_ROPE_YARN) {
        from = std::fmax(std::floor(pair_at(high)), 0.0);
        to = std::fmin(std::ceil(pair_at(low)), r - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; i++) {
        const double t = std::pow(base, -2.0 * i / r);
        double keep = 1.0;  // the part of theta that is not stretched
        if (kind == HQ_ROPE_LINEAR) keep = 0.0;
        if (kind == HQ_ROPE_BANDS) keep = std::fmin(std::fmax((original * t / (2.0 * M_PI) - low) / (high - low), 0.0), 1.0);
        if (kind == HQ_ROPE_YARN) keep = 1.0 - std::fmin(std::fmax((i - from) / std::fmax(to - from, 0.001), 0.0), 1.0);
        theta[i] = t * keep + t / f * (1.0 - keep);
    }
    return HQ_OK;
}

int hq_rope_table(const double *theta, int pairs, uint64_t *turns)
{
    if (!theta || !turns || pairs < 0) return HQ_ERR_ARG;
    for (int i = 0; i < pairs; i++)
        if (!std::isfinite(theta[i])) return HQ_ERR_ARG;
    for (int i = 0; i < pairs; i++) {
        // theta / 2 pi in long double, its fraction of a turn as a 64-bit integer
        const long double t = (long double)theta[i] / (2.0L * 3.14159265358979323846264338327950288L);
        const long double scaled = std::rint((t - std::floor(t)) * 18446744073709551616.0L);
        turns[i] = scaled >= 18446744073709551616.0L ? 0u : (uint64_t)scaled;
    }
    return HQ_OK;
}

}  // extern "C"

namespace {

bool valid_turn(const int64_t *positions, const uint64_t *turns, int rotary_dim, int head_dim, int layout, float amplitude)
{
    if (layout != HQ_ROPE_HALF && layout != HQ_ROPE_INTERLEAVED) return false;
    if (!std::isfinite(amplitude)) return false;
    return valid_rotary(rotary_dim, head_dim) && positions && aligned(positions, 8) && turns && aligned(turns, 8);
}

int launch_pos(const PosArgs &a, void *stream)
{
    return launch_positions(a, (cudaStream_t)stream) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

}  // namespace

extern "C" {

int hq_rope(const hq_rows *x, const hq_rows *y, int64_t tokens, int heads, int head_dim, const int64_t *positions,
            const uint64_t *turns, int rotary_dim, int layout, float amplitude, int inverse, void *stream)
{
    if (tokens < 0 || heads < 0 || head_dim < 16 || head_dim > 256 || head_dim % 16) return HQ_ERR_ARG;
    if (heads > 65535 || tokens >= (int64_t)1 << 31) return HQ_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return HQ_OK;
    if (!valid_turn(positions, turns, rotary_dim, head_dim, layout, amplitude)) return HQ_ERR_ARG;
    if (!readable(x, tokens, heads) || !writable(y, tokens, heads, head_dim)) return HQ_ERR_ARG;
    PosArgs a{};
    a.x = rows_of(x, tokens, heads);
    a.y = rows_of(y, tokens, heads);
    a.tokens = tokens;
    a.heads = heads;
    a.head_dim = head_dim;
    a.rotary = rotary_dim;
    a.interleaved = layout == HQ_ROPE_INTERLEAVED;
    a.inverse = inverse != 0;
    a.amplitude = amplitude;
    a.positions = positions;
    a.turns = turns;
    return launch_pos(a, stream);
}

int hq_kv_append(const hq_rows *q, const hq_rows *q_out, int q_heads, const hq_rows *k, const hq_rows *v,
                 int64_t tokens, const int64_t *positions, const uint64_t *turns, int rotary_dim, int layout,
                 float amplitude, const int64_t *slots, const hq_pages *pages, void *stream, int32_t *d_status)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    if (tokens < 0 || q_heads < 0 || (q != nullptr) != (q_heads > 0) || (q_out != nullptr) != (q_heads > 0))
        return HQ_ERR_ARG;
    if (q_heads > 65535 || tokens >= (int64_t)1 << 31) return HQ_ERR_UNSUPPORTED;
    if (rotary_dim != 0 || turns) {
        if (!valid_turn(positions, turns, rotary_dim, pages->head_dim, layout, amplitude)) {
            if (tokens > 0) return HQ_ERR_ARG;
        }
    }
    if (tokens == 0) return HQ_OK;
    if (!slots || !aligned(slots, 8) || !readable(k, tokens, pages->heads) || !readable(v, tokens, pages->heads))
        return HQ_ERR_ARG;
    if (q && (!readable(q, tokens, q_heads) || !writable(q_out, tokens, q_heads, pages->head_dim))) return HQ_ERR_ARG;
    PosArgs a{};
    if (q) {
        a.x = rows_of(q, tokens, q_heads);
        a.y = rows_of(q_out, tokens, q_heads);
    }
    a.k = rows_of(k, tokens, pages->heads);
    a.v = rows_of(v, tokens, pages->heads);
    a.tokens = tokens;
    a.heads = q_heads;
    a.kvh = pages->heads;
    a.head_dim = pages->head_dim;
    a.rotary = rotary_dim;
    a.interleaved = layout == HQ_ROPE_INTERLEAVED;
    a.amplitude = amplitude;
    a.positions = positions;
    a.turns = turns;
    a.slots = slots;
    a.pk = static_cast<uint16_t *>(pages->k);
    a.pv = static_cast<uint16_t *>(pages->v);
    a.page_stride = pages->page_stride;
    a.head_stride = pages->head_stride;
    a.slot_stride = pages->slot_stride;
    a.nslots = pages->pages * pages->page_size;
    a.page_shift = log2_of(pages->page_size);
    a.status = d_status;
    return launch_pos(a, stream);
}

static int check_paged_sizes(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads, int head_dim,
                             int group)
{
    if (batch < 0 || tokens < 0 || max_q < 0 || max_kv < 0 || heads < 1 || group < 1) return HQ_ERR_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return HQ_ERR_ARG;
    if (batch >= (int64_t)1 << 24 || tokens >= (int64_t)1 << 31 || heads > 65535 || group > 65535 ||
        (int64_t)heads * group > 65535 || max_q > ((int64_t)1 << 30) / group || max_kv > (int64_t)1 << 30)
        return HQ_ERR_UNSUPPORTED;
    return HQ_OK;
}

int hq_paged_attention_workspace_bytes(int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv, int heads,
                                       int head_dim, int group, uint64_t *out)
{
    if (!out) return HQ_ERR_ARG;
    const int rc = check_paged_sizes(batch, tokens, max_q, max_kv, heads, head_dim, group);
    if (rc) return rc;
    // a window only ever needs less
    *out = paged_plan(batch, tokens, max_q, max_kv, heads, group, head_dim, 0).total;
    return HQ_OK;
}

static int paged_attention(const hq_rows *q, const int32_t *q_start, const int32_t *kv_len, int64_t batch, int64_t tokens,
                           int64_t max_q, int64_t max_kv, int group, const hq_pages *pages, const int32_t *table,
                           int64_t table_width, int64_t table_stride, float scale, int causal, int64_t window,
                           const hq_rows *out, float *lse, void *workspace, uint64_t workspace_bytes, void *stream,
                           int32_t *d_status, int stall_kind, int stall)
{
    int rc = check_pages(pages);
    if (rc) return rc;
    rc = check_paged_sizes(batch, tokens, max_q, max_kv, pages->heads, pages->head_dim, group);
    if (rc) return rc;
    const float scale_log2 = std::fabs(scale) * 1.44269504088896341f;  // infinite past 2.36e38
    if (!std::isfinite(scale_log2) || window < 0 || table_width < 0 || (batch > 1 && table_stride < table_width))
        return HQ_ERR_ARG;
    if (batch == 0 || tokens == 0 || max_q == 0) return HQ_OK;
    const int heads = pages->heads * group, d = pages->head_dim;
    if (!readable(q, tokens, heads) || q->dtype != HQ_BF16 || !writable(out, tokens, heads, d)) return HQ_ERR_ARG;
    if (!q_start || !kv_len || !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(lse, 4)) return HQ_ERR_ARG;
    if (table_width > 0 && (!table || !aligned(table, 4))) return HQ_ERR_ARG;
    const PagedPlan p = paged_plan(batch, tokens, max_q, max_kv, pages->heads, group, d, window);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < p.total) return HQ_ERR_WORKSPACE;
    PagedArgs a{};
    a.q = rows_of(q, tokens, heads);
    a.out = rows_of(out, tokens, heads);
    a.lse = lse;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.table = table;
    a.table_stride = table_stride;
    a.tokens = tokens;
    a.batch = (int)batch;
    a.max_q = (int)max_q;
    const int64_t held = table_width > ((int64_t)1 << 30) / pages->page_size ? (int64_t)1 << 30
                                                                             : table_width * pages->page_size;
    a.max_tokens = (int)(max_kv < held ? max_kv : held);
    a.heads = pages->heads;
    a.group = group;
    a.group_div = make_fastdiv((uint32_t)group);
    a.k = static_cast<const uint16_t *>(pages->k);
    a.v = static_cast<const uint16_t *>(pages->v);
    a.page_stride = pages->page_stride;
    a.head_stride = pages->head_stride;
    a.slot_stride = pages->slot_stride;
    a.pages = (uint32_t)pages->pages;
    a.page_shift = log2_of(pages->page_size);
    a.scale_log2 = scale == 0.0f ? 1.0f : scale_log2;
    a.q_mode = scale == 0.0f ? 2 : scale < 0.0f ? 1 : 0;
    a.causal = causal != 0;
    a.window = (int)(window > INT32_MAX ? 0 : window);  // wider than any cache: all
    a.stall_kind = stall_kind;
    a.stall = stall;
    a.status = d_status;
    return launch_paged(a, p, d, workspace, (cudaStream_t)stream) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

int hq_paged_attention(const hq_rows *q, const int32_t *q_start, const int32_t *kv_len, int64_t batch, int64_t tokens,
                       int64_t max_q, int64_t max_kv, int group, const hq_pages *pages, const int32_t *table,
                       int64_t table_width, int64_t table_stride, float scale, int causal, int64_t window,
                       const hq_rows *out, float *lse, void *workspace, uint64_t workspace_bytes, void *stream,
                       int32_t *d_status)
{
    return paged_attention(q, q_start, kv_len, batch, tokens, max_q, max_kv, group, pages, table, table_width, table_stride,
                           scale, causal, window, out, lse, workspace, workspace_bytes, stream, d_status, kStallNone, 0);
}

int hq_test_paged_attention_stalled(const hq_rows *q, const int32_t *q_start, const int32_t *kv_len, int64_t batch,
                                    int64_t tokens, int64_t max_q, int64_t max_kv, int group, const hq_pages *pages,
                                    const int32_t *table, int64_t table_width, int64_t table_stride, float scale, int causal,
                                    int64_t window, const hq_rows *out, float *lse, void *workspace,
                                    uint64_t workspace_bytes, void *stream, int32_t *d_status, int kind, int stalled)
{
    if ((kind != kStallCopy && kind != kStallProduct) || stalled < 0) return HQ_ERR_ARG;
    return paged_attention(q, q_start, kv_len, batch, tokens, max_q, max_kv, group, pages, table, table_width, table_stride,
                           scale, causal, window, out, lse, workspace, workspace_bytes, stream, d_status, kind, stalled);
}

int hq_attention_merge(const hq_rows *a, const float *lse_a, const hq_rows *b, const float *lse_b, int64_t tokens,
                       int heads, int head_dim, const hq_rows *out, float *lse, void *stream)
{
    if (tokens < 0 || heads < 0 || head_dim < 8 || head_dim > 1024 || head_dim % 8) return HQ_ERR_ARG;
    if (heads > 0 && tokens >= ((int64_t)1 << 32) / heads) return HQ_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return HQ_OK;
    if (!readable(a, tokens, heads) || !readable(b, tokens, heads) || !writable(out, tokens, heads, head_dim))
        return HQ_ERR_ARG;
    if (!lse_a || !lse_b || !aligned(lse_a, 4) || !aligned(lse_b, 4) || !aligned(lse, 4)) return HQ_ERR_ARG;
    // rows of lse are written while other threads still read these
    const uint64_t bytes = 4 * (uint64_t)tokens * heads;
    auto apart = [&](const float *r) { return (uintptr_t)lse + bytes <= (uintptr_t)r || (uintptr_t)r + bytes <= (uintptr_t)lse; };
    if (lse && !(apart(lse_a) && apart(lse_b))) return HQ_ERR_ARG;
    MergeArgs m{};
    m.a = rows_of(a, tokens, heads);
    m.b = rows_of(b, tokens, heads);
    m.out = rows_of(out, tokens, heads);
    m.lse_a = lse_a;
    m.lse_b = lse_b;
    m.lse = lse;
    m.tokens = tokens;
    m.heads = heads;
    m.head_dim = head_dim;
    return launch_merge(m, (cudaStream_t)stream) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

}  // extern "C"
