// cache_api.cu -- the C ABI of the paged cache (include/sel/cache.h, include/sel/cache_serving.h): argument checks and dispatch.
// Host code only.
#include <cmath>
#include <cstdint>

#include "../../include/sel/cache_serving.h"
#include "cache_internal.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffffLL;
constexpr int64_t kMaxPositions = kIntMax - 255;  // of a sequence: a tile's last position is an int too
constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void *p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? SEL_OK : SEL_ECUDA; }

// a * b of two non-negative numbers, or -1 past 2^62
int64_t product(int64_t a, int64_t b) { return b != 0 && a > (int64_t{1} << 62) / b ? -1 : a * b; }

int check_cache(const sel_cache *c, bool to_write)
{
    if (!c) return SEL_EINVAL;
    if (c->dtype != SEL_BF16 && c->dtype != SEL_E4M3) return SEL_EINVAL;
    const bool codes = c->dtype == SEL_E4M3;
    if (c->pages < 0 || c->page_size < 1 || c->d < 1) return SEL_EINVAL;
    if (c->pages > 0 && !c->data) return SEL_EINVAL;
    if (c->row_stride < 0 || c->page_stride < 0) return SEL_EINVAL;
    if (c->page_size > 1 && c->row_stride < c->d) return SEL_EINVAL;
    // rows of a cache that is written may not overlap
    if (to_write && c->pages > 1 && c->page_stride < c->d) return SEL_EINVAL;
    if (codes && c->pages > 0) {
        if (!c->scales) return SEL_EINVAL;
        const int64_t runs = (c->d + SEL_CACHE_GROUP - 1) / SEL_CACHE_GROUP;
        if (c->scale_row_stride < 0 || c->scale_page_stride < 0) return SEL_EINVAL;
        if (c->page_size > 1 && c->scale_row_stride < runs) return SEL_EINVAL;
        if (to_write && c->pages > 1 && c->scale_page_stride < runs) return SEL_EINVAL;
        if (!aligned(c->scales, 4)) return SEL_EALIGN;
    }
    if (!codes && c->scales) return SEL_EINVAL;
    if (product(c->pages, c->page_size) < 0 || c->d > kIntMax) return SEL_EUNSUPPORTED;
    const int64_t e = codes ? 1 : 2;
    if ((c->d * e) % 16 != 0 || (c->row_stride * e) % 16 != 0 || (c->page_stride * e) % 16 != 0 ||
        !aligned(c->data, 16))
        return SEL_EALIGN;
    return SEL_OK;
}

int check_table(const sel_cache *c, const int32_t *table, int64_t b, int64_t max_pages, int64_t table_stride,
                int64_t rows)
{
    if (b < 1 || max_pages < 0 || rows < 0 || rows % b != 0) return SEL_EINVAL;
    if (max_pages > 0 && (!table || (b > 1 && table_stride < max_pages))) return SEL_EINVAL;
    if (!aligned(table, 4)) return SEL_EALIGN;
    const int64_t positions = product(max_pages, c->page_size);
    if (positions < 0) return SEL_EUNSUPPORTED;
    return SEL_OK;
}

sel::CacheRef ref_of(const sel_cache *c)
{
    sel::CacheRef r{};
    r.data = c->data;
    r.scales = c->dtype == SEL_E4M3 ? c->scales : nullptr;
    r.pages = c->pages;
    r.page_size = c->page_size;
    r.d = c->d;
    r.page_stride = c->page_stride;
    r.row_stride = c->row_stride;
    r.scale_page_stride = c->scale_page_stride;
    r.scale_row_stride = c->scale_row_stride;
    return r;
}

sel::PageTable table_of(const int32_t *table, int64_t b, int64_t max_pages, int64_t stride, int64_t rows)
{
    sel::PageTable t{};
    t.table = table;
    t.max_pages = max_pages;
    t.stride = stride;
    t.rows_per_seq = rows / b;
    return t;
}


// What a row sees, for `positions` that a page table has: a window past them is none.
sel::Seen seen_by_window(int64_t positions, int64_t window, int64_t sinks)
{
    sel::Seen seen{};
    if (sinks < positions && window < positions - sinks) {
        seen.window = static_cast<int32_t>(window);
        seen.sinks = static_cast<int32_t>(sinks);
    }
    return seen;
}
sel::Seen seen_by_all(int64_t positions, int64_t shared)
{
    sel::Seen seen{};
    seen.shared = static_cast<int32_t>(shared < positions ? shared : positions);
    return seen;
}

// Positions of a page table, or -1 where the attention's arguments say that no scratch is needed.
int64_t attended(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b, int64_t max_pages, int64_t page_size)
{
    if (rows <= 0 || h < 1 || d < 1 || d > SEL_CACHE_ATTN_MAX_D || dv < 1 || dv > d || b < 1 || rows % b != 0 ||
        max_pages < 0 || page_size < 1)
        return -1;
    const int64_t cap = product(max_pages, page_size);
    return cap > kMaxPositions || product(rows, h) < 0 || rows * h > kIntMax ? -1 : cap;
}

// What the attention's entry points have in common; `limit` and `other` are window and sinks, or shared.
enum class Form { plain, window, shared };
struct AttnCall {
    const void *q;
    int64_t rows, h, q_row_stride, q_head_stride;
    const sel_cache *cache;
    const int32_t *page_table;
    int64_t b, max_pages, table_stride;
    const int32_t *end;
    const void *idx;
    int idx_dtype;
    int64_t n, idx_row_stride, dv;
    float scale;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    int32_t *err_flag;
    void *stream;
    Form form;
    int64_t limit, other;
};

int attention(const AttnCall &c)
{
    int st = check_cache(c.cache, false);
    if (st != SEL_OK) return st;
    st = check_table(c.cache, c.page_table, c.b, c.max_pages, c.table_stride, c.rows);
    if (st != SEL_OK) return st;
    if (c.h < 1 || c.dv < 1 || c.dv > c.cache->d || !std::isfinite(c.scale) || !std::isfinite(c.scale * kLog2e))
        return SEL_EINVAL;
    if (c.idx) {
        if (c.idx_dtype != SEL_I32 && c.idx_dtype != SEL_I64) return SEL_EINVAL;
        if (c.n < 0 || (c.rows > 1 && c.idx_row_stride < c.n)) return SEL_EINVAL;
        if (!aligned(c.idx, c.idx_dtype == SEL_I64 ? 8 : 4)) return SEL_EALIGN;
        if (c.n > kMaxPositions) return SEL_EUNSUPPORTED;
    }
    if (c.form == Form::window && (c.limit < 1 || c.other < 0)) return SEL_EINVAL;
    if (c.form == Form::shared && c.limit < 0) return SEL_EINVAL;
    if (c.rows == 0) return SEL_OK;
    if (!c.q || !c.out) return SEL_EINVAL;
    if (c.q_row_stride < 0 || c.q_head_stride < 0) return SEL_EINVAL;
    if (c.dv % 8 != 0 || !aligned(c.q, 16) || !aligned(c.out, 16) || !aligned(c.lse, 4) || !aligned(c.end, 4)) return SEL_EALIGN;
    if ((c.rows > 1 && c.q_row_stride % 8 != 0) || (c.h > 1 && c.q_head_stride % 8 != 0)) return SEL_EALIGN;
    if (c.cache->d > SEL_CACHE_ATTN_MAX_D || product(c.max_pages, c.cache->page_size) > kMaxPositions) return SEL_EUNSUPPORTED;
    if (product(c.rows, c.h) < 0 || c.rows * c.h > kIntMax) return SEL_EUNSUPPORTED;
    const int64_t cap = product(c.max_pages, c.cache->page_size);
    const sel::Seen seen = c.form == Form::window   ? seen_by_window(cap, c.limit, c.other)
                           : c.form == Form::shared ? seen_by_all(cap, c.limit)
                                                    : sel::Seen{};
    const size_t need = sel::cache_attention_workspace(c.rows, c.h, c.cache->d, c.dv, c.b, c.idx ? c.n : cap,
                                                       c.idx != nullptr, seen);
    if (need > 0) {
        if (!c.workspace || c.workspace_bytes < need) return SEL_EINVAL;
        if (!aligned(c.workspace, 256)) return SEL_EALIGN;
    }
    sel::CacheAttnArgs a{};
    a.c = ref_of(c.cache);
    a.t = table_of(c.page_table, c.b, c.max_pages, c.table_stride, c.rows);
    a.q = static_cast<const uint16_t *>(c.q);
    a.rows = c.rows;
    a.q_row_stride = c.q_row_stride;
    a.q_head_stride = c.q_head_stride;
    a.h = static_cast<int32_t>(c.h);
    a.d = static_cast<int32_t>(c.cache->d);
    a.dv = static_cast<int32_t>(c.dv);
    a.end = c.end;
    a.idx = c.idx;
    a.idx_i64 = c.idx_dtype == SEL_I64;
    a.n = c.idx ? static_cast<int32_t>(c.n) : 0;
    a.idx_row_stride = c.idx_row_stride;
    // (a scale of 0 becomes the smallest number, so that a masked score, an infinity, keeps the weight 0)
    a.scale_log2 = c.scale == 0.0f ? 1.4e-45f : c.scale * kLog2e;
    a.out = static_cast<uint16_t *>(c.out);
    a.lse = c.lse;
    a.err_flag = c.err_flag;
    a.ws = c.workspace;
    a.seen = seen;
    return status_of(sel::launch_cache_attention(a, static_cast<cudaStream_t>(c.stream)));
}

}  // namespace

extern "C" {

int sel_cache_write(const void *x, int x_dtype, int64_t tokens, int64_t x_stride, const void *slots, int slot_dtype,
                    const sel_cache *cache, int32_t *err_flag, void *stream)
{
    if (x_dtype != SEL_F32 && x_dtype != SEL_BF16) return SEL_EINVAL;
    if (slot_dtype != SEL_I32 && slot_dtype != SEL_I64) return SEL_EINVAL;
    const int st = check_cache(cache, true);
    if (st != SEL_OK) return st;
    if (tokens < 0) return SEL_EINVAL;
    if (tokens == 0) return SEL_OK;
    if (!x || !slots || (tokens > 1 && x_stride < cache->d)) return SEL_EINVAL;
    const int64_t e = x_dtype == SEL_F32 ? 4 : 2;
    if (!aligned(x, 16) || (tokens > 1 && (x_stride * e) % 16 != 0)) return SEL_EALIGN;
    if (!aligned(slots, slot_dtype == SEL_I64 ? 8 : 4)) return SEL_EALIGN;
    const int64_t runs = (cache->d + SEL_CACHE_GROUP - 1) / SEL_CACHE_GROUP;
    if (tokens > kIntMax / (16 * runs)) return SEL_EUNSUPPORTED;  // (16 lanes a run, 32-bit counts)
    sel::CacheWriteArgs a{};
    a.c = ref_of(cache);
    a.x = x;
    a.tokens = tokens;
    a.x_stride = x_stride;
    a.slots = slots;
    a.slots_i64 = slot_dtype == SEL_I64;
    a.x_bf16 = x_dtype == SEL_BF16;
    a.err_flag = err_flag;
    return status_of(sel::launch_cache_write(a, static_cast<cudaStream_t>(stream)));
}

int sel_cache_gather(const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                     int64_t table_stride, const void *idx, int idx_dtype, int64_t rows, int64_t n,
                     int64_t idx_row_stride, void *out, int32_t *err_flag, void *stream)
{
    if (idx_dtype != SEL_I32 && idx_dtype != SEL_I64) return SEL_EINVAL;
    int st = check_cache(cache, false);
    if (st != SEL_OK) return st;
    st = check_table(cache, page_table, b, max_pages, table_stride, rows);
    if (st != SEL_OK) return st;
    if (n < 0) return SEL_EINVAL;
    if (rows == 0 || n == 0) return SEL_OK;
    if (!idx || !out || (rows > 1 && idx_row_stride < n)) return SEL_EINVAL;
    if (!aligned(out, 16) || !aligned(idx, idx_dtype == SEL_I64 ? 8 : 4)) return SEL_EALIGN;
    if (product(rows, n) < 0 || cache->d > kIntMax / 256) return SEL_EUNSUPPORTED;
    sel::CacheGatherArgs a{};
    a.c = ref_of(cache);
    a.t = table_of(page_table, b, max_pages, table_stride, rows);
    a.idx = idx;
    a.idx_i64 = idx_dtype == SEL_I64;
    a.rows = rows;
    a.n = n;
    a.idx_row_stride = idx_row_stride;
    a.out = static_cast<uint16_t *>(out);
    a.err_flag = err_flag;
    return status_of(sel::launch_cache_gather(a, static_cast<cudaStream_t>(stream)));
}

int sel_cache_set_wait_limit(int64_t cycles)
{
    sel::set_cache_wait_cycles(cycles);
    return SEL_OK;
}

size_t sel_cache_attention_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b, int64_t max_pages,
                                          int64_t page_size, int idx_given, int64_t n)
{
    const int64_t cap = attended(rows, h, d, dv, b, max_pages, page_size);
    if (cap < 0 || n < 0 || n > kMaxPositions) return 0;
    return sel::cache_attention_workspace(rows, h, d, dv, b, idx_given ? n : cap, idx_given != 0, sel::Seen{});
}

int sel_cache_attention(const void *q, int64_t rows, int64_t h, int64_t q_row_stride, int64_t q_head_stride,
                        const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                        int64_t table_stride, const int32_t *end, const void *idx, int idx_dtype, int64_t n,
                        int64_t idx_row_stride, int64_t dv, float scale, void *out, float *lse, void *workspace,
                        size_t workspace_bytes, int32_t *err_flag, void *stream)
{
    return attention(AttnCall{q, rows, h, q_row_stride, q_head_stride, cache, page_table, b, max_pages, table_stride, end,
                              idx, idx_dtype, n, idx_row_stride, dv, scale, out, lse, workspace, workspace_bytes, err_flag,
                              stream, Form::plain, 0, 0});
}

size_t sel_cache_attention_window_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b,
                                                 int64_t max_pages, int64_t page_size, int64_t window, int64_t sinks)
{
    const int64_t cap = attended(rows, h, d, dv, b, max_pages, page_size);
    if (cap < 0 || window < 1 || sinks < 0) return 0;
    return sel::cache_attention_workspace(rows, h, d, dv, b, cap, false, seen_by_window(cap, window, sinks));
}

int sel_cache_attention_window(const void *q, int64_t rows, int64_t h, int64_t q_row_stride, int64_t q_head_stride,
                               const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                               int64_t table_stride, const int32_t *end, int64_t window, int64_t sinks, int64_t dv,
                               float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                               int32_t *err_flag, void *stream)
{
    return attention(AttnCall{q, rows, h, q_row_stride, q_head_stride, cache, page_table, b, max_pages, table_stride, end,
                              nullptr, SEL_I32, 0, 0, dv, scale, out, lse, workspace, workspace_bytes, err_flag, stream,
                              Form::window, window, sinks});
}

size_t sel_cache_attention_shared_workspace_size(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b,
                                                 int64_t max_pages, int64_t page_size, int64_t shared)
{
    const int64_t cap = attended(rows, h, d, dv, b, max_pages, page_size);
    if (cap < 0 || shared < 0) return 0;
    return sel::cache_attention_workspace(rows, h, d, dv, b, cap, false, seen_by_all(cap, shared));
}

int sel_cache_attention_shared(const void *q, int64_t rows, int64_t h, int64_t q_row_stride, int64_t q_head_stride,
                               const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                               int64_t table_stride, const int32_t *end, int64_t shared, int64_t dv, float scale,
                               void *out, float *lse, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                               void *stream)
{
    return attention(AttnCall{q, rows, h, q_row_stride, q_head_stride, cache, page_table, b, max_pages, table_stride, end,
                              nullptr, SEL_I32, 0, 0, dv, scale, out, lse, workspace, workspace_bytes, err_flag, stream,
                              Form::shared, shared, 0});
}

int sel_cache_append(const void *x, int x_dtype, int64_t tokens, int64_t x_stride, const sel_cache *cache,
                     const int32_t *page_table, int64_t b, int64_t max_pages, int64_t table_stride,
                     const void *positions, int pos_dtype, const sel_rotation *rotation, const void *q, int q_dtype,
                     int64_t h, int64_t q_row_stride, int64_t q_head_stride, void *q_out, int32_t *err_flag, void *stream)
{
    if (x_dtype != SEL_F32 && x_dtype != SEL_BF16) return SEL_EINVAL;
    if (pos_dtype != SEL_I32 && pos_dtype != SEL_I64) return SEL_EINVAL;
    int st = check_cache(cache, true);
    if (st != SEL_OK) return st;
    if (tokens < 0) return SEL_EINVAL;
    st = check_table(cache, page_table, b, max_pages, table_stride, tokens);
    if (st != SEL_OK) return st;
    const int64_t d = cache->d;
    if (!rotation || rotation->positions < 0 || rotation->first < 0 || rotation->rot < 1 || rotation->rot > d ||
        rotation->first > d - rotation->rot)
        return SEL_EINVAL;
    if (rotation->positions > 0 && (!rotation->table || (rotation->positions > 1 && rotation->stride < rotation->rot)))
        return SEL_EINVAL;
    if (q && ((q_dtype != SEL_F32 && q_dtype != SEL_BF16) || h < 1 || q_row_stride < 0 || q_head_stride < 0))
        return SEL_EINVAL;
    if (tokens == 0) return SEL_OK;
    if (!x || !positions || (tokens > 1 && x_stride < d) || (q && !q_out)) return SEL_EINVAL;
    const int64_t e = x_dtype == SEL_F32 ? 4 : 2, qe = q_dtype == SEL_F32 ? 4 : 2;
    if (!aligned(x, 16) || (tokens > 1 && (x_stride * e) % 16 != 0)) return SEL_EALIGN;
    if (!aligned(positions, pos_dtype == SEL_I64 ? 8 : 4)) return SEL_EALIGN;
    if (rotation->first % 8 != 0 || rotation->rot % 16 != 0 || !aligned(rotation->table, 16) ||
        (rotation->positions > 1 && rotation->stride % 4 != 0))
        return SEL_EALIGN;
    const int64_t runs = (d + SEL_CACHE_GROUP - 1) / SEL_CACHE_GROUP;
    if (tokens > kIntMax / (16 * runs) || d >= int64_t{1} << 30) return SEL_EUNSUPPORTED;  // (16 lanes a run, 32-bit counts)
    if (q) {
        if (!aligned(q, 16) || !aligned(q_out, 16)) return SEL_EALIGN;
        const int64_t by_rows = product(tokens - 1, q_row_stride), by_heads = product(h - 1, q_head_stride);
        const int64_t far = int64_t{1} << 56;  // (more elements than there are addresses for)
        if (by_rows < 0 || by_heads < 0 || by_rows > far || by_heads > far) return SEL_EUNSUPPORTED;
        if ((tokens > 1 && (q_row_stride * qe) % 16 != 0) || (h > 1 && (q_head_stride * qe) % 16 != 0)) return SEL_EALIGN;
        const int64_t each = product(h, d);
        if (each < 0 || each > kIntMax || tokens * each >= int64_t{1} << 40) return SEL_EUNSUPPORTED;  // (below 2^58)
        const bool same = q == q_out && q_dtype == SEL_BF16 && (tokens == 1 || q_row_stride == each) &&
                          (h == 1 || q_head_stride == d);
        const uint64_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(q_out);
        const uint64_t read = static_cast<uint64_t>((by_rows + by_heads + d) * qe), written = static_cast<uint64_t>(tokens * each) * 2;
        if (!same && from < to + written && to < from + read) return SEL_EINVAL;
    }
    sel::CacheAppendArgs a{};
    a.c = ref_of(cache);
    a.t = table_of(page_table, b, max_pages, table_stride, tokens);
    a.x = x;
    a.tokens = tokens;
    a.x_stride = x_stride;
    a.positions = positions;
    a.rotation = rotation->table;
    a.rot_rows = rotation->positions;
    a.rot_stride = rotation->stride;
    a.first = static_cast<int32_t>(rotation->first);
    a.rot = static_cast<int32_t>(rotation->rot);
    a.interleaved = rotation->interleaved != 0;
    a.pos_i64 = pos_dtype == SEL_I64;
    a.x_bf16 = x_dtype == SEL_BF16;
    a.q_bf16 = q_dtype == SEL_BF16;
    a.q = q;
    a.h = q ? h : 0;
    a.q_row_stride = q_row_stride;
    a.q_head_stride = q_head_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.err_flag = err_flag;
    return status_of(sel::launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
