// cache_api.cu -- the C ABI of the paged cache (include/sel/cache.h): argument checks and dispatch.
// Host code only.
#include <cmath>
#include <cstdint>

#include "../../include/sel/cache.h"
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
    if (rows <= 0 || h < 1 || d < 1 || d > SEL_CACHE_ATTN_MAX_D || dv < 1 || dv > d || b < 1 || rows % b != 0 ||
        max_pages < 0 || page_size < 1 || n < 0)
        return 0;
    const int64_t cap = product(max_pages, page_size);
    if (cap < 0 || cap > kMaxPositions || n > kMaxPositions || product(rows, h) < 0 || rows * h > kIntMax) return 0;
    return sel::cache_attention_workspace(rows, h, d, dv, b, idx_given ? n : cap, idx_given != 0);
}

int sel_cache_attention(const void *q, int64_t rows, int64_t h, int64_t q_row_stride, int64_t q_head_stride,
                        const sel_cache *cache, const int32_t *page_table, int64_t b, int64_t max_pages,
                        int64_t table_stride, const int32_t *end, const void *idx, int idx_dtype, int64_t n,
                        int64_t idx_row_stride, int64_t dv, float scale, void *out, float *lse, void *workspace,
                        size_t workspace_bytes, int32_t *err_flag, void *stream)
{
    int st = check_cache(cache, false);
    if (st != SEL_OK) return st;
    st = check_table(cache, page_table, b, max_pages, table_stride, rows);
    if (st != SEL_OK) return st;
    if (h < 1 || dv < 1 || dv > cache->d || !std::isfinite(scale) || !std::isfinite(scale * kLog2e))
        return SEL_EINVAL;
    if (idx) {
        if (idx_dtype != SEL_I32 && idx_dtype != SEL_I64) return SEL_EINVAL;
        if (n < 0 || (rows > 1 && idx_row_stride < n)) return SEL_EINVAL;
        if (!aligned(idx, idx_dtype == SEL_I64 ? 8 : 4)) return SEL_EALIGN;
        if (n > kMaxPositions) return SEL_EUNSUPPORTED;
    }
    if (rows == 0) return SEL_OK;
    if (!q || !out) return SEL_EINVAL;
    if (q_row_stride < 0 || q_head_stride < 0) return SEL_EINVAL;
    if (dv % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(end, 4)) return SEL_EALIGN;
    if ((rows > 1 && q_row_stride % 8 != 0) || (h > 1 && q_head_stride % 8 != 0)) return SEL_EALIGN;
    if (cache->d > SEL_CACHE_ATTN_MAX_D || product(max_pages, cache->page_size) > kMaxPositions) return SEL_EUNSUPPORTED;
    if (product(rows, h) < 0 || rows * h > kIntMax) return SEL_EUNSUPPORTED;
    const size_t need = sel_cache_attention_workspace_size(rows, h, cache->d, dv, b, max_pages, cache->page_size,
                                                           idx != nullptr, idx ? n : 0);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return SEL_EINVAL;
        if (!aligned(workspace, 256)) return SEL_EALIGN;
    }
    sel::CacheAttnArgs a{};
    a.c = ref_of(cache);
    a.t = table_of(page_table, b, max_pages, table_stride, rows);
    a.q = static_cast<const uint16_t *>(q);
    a.rows = rows;
    a.q_row_stride = q_row_stride;
    a.q_head_stride = q_head_stride;
    a.h = static_cast<int32_t>(h);
    a.d = static_cast<int32_t>(cache->d);
    a.dv = static_cast<int32_t>(dv);
    a.end = end;
    a.idx = idx;
    a.idx_i64 = idx_dtype == SEL_I64;
    a.n = idx ? static_cast<int32_t>(n) : 0;
    a.idx_row_stride = idx_row_stride;
    // (a scale of 0 becomes the smallest number, so that a masked score, an infinity, keeps the weight 0)
    a.scale_log2 = scale == 0.0f ? 1.4e-45f : scale * kLog2e;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.err_flag = err_flag;
    a.ws = workspace;
    return status_of(sel::launch_cache_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
