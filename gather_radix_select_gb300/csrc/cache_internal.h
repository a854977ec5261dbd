// cache_internal.h -- argument blocks and launchers of the paged-cache operators, shared by the
// C-ABI layer (cache_api.cu) and the kernels (cache*.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "sel_internal.h"

namespace sel {

constexpr int kCacheGroup = 128;   // elements that share a scale
constexpr int32_t kCacheInval = 1; // SEL_EINVAL

// A paged cache; strides in elements (bf16 or 1-byte codes).
struct CacheRef {
    void *data;
    float *scales;  // null: bf16 rows
    int64_t pages, page_size, d;
    int64_t page_stride, row_stride, scale_page_stride, scale_row_stride;
};

struct PageTable {
    const int32_t *table;
    int64_t max_pages, stride;
    int64_t rows_per_seq;  // rows of a call that belong to one sequence
};

struct CacheWriteArgs {
    CacheRef c;
    const void *x;
    int64_t tokens, x_stride;
    const void *slots;
    int32_t slots_i64;
    int32_t x_bf16;
    int32_t *err_flag;
};

struct CacheGatherArgs {
    CacheRef c;
    PageTable t;
    const void *idx;
    int32_t idx_i64;
    int64_t rows, n, idx_row_stride;
    uint16_t *out;
    int32_t *err_flag;
    int32_t pairs;  // positions of a CTA, set by the launcher
};

// What a row attends to of the positions below its end, where no list says it; 32 bits: so are positions.
struct Seen {
    int32_t window;  // the last `window` of them and those below `sinks`; 0: all
    int32_t sinks;
    int32_t shared;  // positions below this are the same rows for all sequences; 0: none
};

struct CacheAppendArgs {
    CacheRef c;
    PageTable t;
    const void *x;
    int64_t tokens, x_stride;
    const void *positions;
    const float *rotation;  // [rot_rows, rot_stride]: rot / 2 cosines, rot / 2 sines
    int64_t rot_rows, rot_stride;
    int32_t first, rot;     // the rotated run of a row
    int32_t interleaved;    // pairs are neighbours, else rot / 2 apart
    int32_t pos_i64, x_bf16, q_bf16;
    const void *q;          // nullable
    int64_t h, q_row_stride, q_head_stride;
    uint16_t *q_out;
    int32_t *err_flag;
};

struct CacheAttnArgs {
    CacheRef c;
    PageTable t;
    const uint16_t *q;
    int64_t rows, q_row_stride, q_head_stride;
    int32_t h, d, dv;
    const int32_t *end;  // nullable
    const void *idx;     // nullable: every position below end
    int32_t idx_i64;
    int32_t n;
    int64_t idx_row_stride;
    float scale_log2;    // scale * log2(e)
    uint16_t *out;
    float *lse;          // nullable
    int32_t *err_flag;   // nullable
    void *ws;
    Seen seen;           // without a list only
};

// Of `items` items dealt out in turn to `ctas` CTAs (no more than items), those of one CTA; up to 2^31 - 1 items.
constexpr int units_of(int items, int cta, int ctas)
{
    return static_cast<int>(static_cast<uint32_t>(items - 1 - cta) / static_cast<uint32_t>(ctas)) + 1;
}
static_assert(units_of(1, 0, 1) == 1 && units_of(305, 0, 152) == 3 && units_of(305, 1, 152) == 2, "");
static_assert(units_of(0x7fffffff, 0, 152) == 14128182 && units_of(0x7fffffff, 151, 152) == 14128181, "");

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t s);
cudaError_t launch_cache_gather(const CacheGatherArgs &a, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t s);
cudaError_t launch_cache_attention(const CacheAttnArgs &a, cudaStream_t s);

// Cycles after which a wait of the attention kernel gives up, from the next call on; negative: the usual ones.
void set_cache_wait_cycles(long long cycles);

// Workspace bytes of an attention call; launches nothing.
size_t cache_attention_workspace(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b, int64_t positions,
                                 bool idx_given, const Seen &seen);

#ifdef __CUDACC__
// Flat row offset (page * page_size + place) does not serve strided pages, so rows are found by page
// and place.  Returns false when the position or its page is outside the cache.
__device__ __forceinline__ bool find_row(const CacheRef &c, const PageTable &t, int64_t seq, int64_t pos,
                                         int64_t &page, int64_t &place)
{
    if (pos < 0) return false;
    int64_t col;
    if ((pos | c.page_size) >> 32 == 0) {  // the common case, without the 64-bit division
        const uint32_t p = static_cast<uint32_t>(pos), ps = static_cast<uint32_t>(c.page_size);
        const uint32_t q = p / ps;
        col = q;
        place = p - q * ps;
    } else {
        col = pos / c.page_size;
        place = pos - col * c.page_size;
    }
    if (col >= t.max_pages) return false;
    page = t.table[seq * t.stride + col];
    return page >= 0 && page < c.pages;
}
#endif

}  // namespace sel
