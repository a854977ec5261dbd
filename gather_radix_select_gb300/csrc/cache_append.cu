// cache_append.cu -- new rows appended to a paged cache at their positions, rotated on the way, and the same tokens'
// queries rotated alike, in one launch.
//
// A pair (u, v) of the run [first, first + rot) becomes (u cos - v sin, v cos + u sin), with the cosine and sine of
// the token's position and the pair's index out of a table.  Both products and their sum are rounded to fp32, each
// once (no fused multiply-add: the bits do not depend on which of the pair's values is formed where), the result once
// more to what it is held in.
//
// The first CTAs take the rows, by runs of 128 elements as in cache_write_kernel; a lane that holds 8 elements of a
// rotated run whose pairs lie half the run apart loads the 8 partners too (they are in L1 or on their way there: the
// other lanes' own).  The next ones take what is rotated of the queries, by units of 16 elements that make 8 pairs, so
// that whoever reads a value is who writes it and queries can be rotated where they are; the last ones copy the rest.
#include <cstdint>

#include "cache_internal.h"
#include "cache_rows.cuh"

namespace sel {
namespace {

constexpr int kThreads = 256;
constexpr int kCopies = 4;  // vectors of 8 elements that a thread copies, all under way at once

// n / d for n < 2^31, as a product (d >= 1): with 2^(l - 1) < d <= 2^l and m = ceil(2^(31 + l) / d), the product's error
// n (m d - 2^(31 + l)) / d is below 2^31 * d / d <= 2^(31 + l) / d, too small to reach the next integer.
struct Divisor {
    uint32_t d, m, shift;
};
__device__ __forceinline__ uint32_t divide(uint32_t n, Divisor by)
{
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * by.m) >> by.shift);
}
Divisor divisor_of(uint32_t d)
{
    uint32_t l = 0;
    while (l < 31 && (uint32_t{1} << l) < d) ++l;
    const uint64_t top = uint64_t{1} << (31 + l);
    return Divisor{d, static_cast<uint32_t>((top + d - 1) / d), 31 + l};
}

__device__ __forceinline__ void load8f(const float *p, float v[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float turned_first(float u, float v, float c, float s)
{
    return __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
}
__device__ __forceinline__ float turned_second(float u, float v, float c, float s)
{
    return __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
}

__device__ __forceinline__ int64_t position_of(const CacheAppendArgs &a, int64_t token)
{
    return a.pos_i64 ? __ldg(static_cast<const int64_t *>(a.positions) + token)
                     : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(a.positions) + token));
}

// What a row's place is found with: groups of lanes a token, tokens a sequence, log2 of the page's size (-1: none).
struct Rows {
    uint32_t items;
    Divisor groups, per_seq;
    int page_shift;
};

// 8 elements as they lie in memory, and their values.
template <bool BF16>
struct Raw {
    uint4 x[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        const uint4 *from = BF16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at)
                                 : reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) x[i] = __ldcs(from + i);
    }
    __device__ __forceinline__ void values(float v[8]) const
    {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(!BF16 ? w[i] : i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

// R runs of one token by a group of lanes, their loads side by side.
template <int R, bool BF16>
__device__ __forceinline__ void append_rows(const CacheAppendArgs &a, const Rows &by)
{
    const uint32_t lane = threadIdx.x & (kWriteLanes - 1);
    const unsigned half = 0xffffu << (threadIdx.x & 16);  // this group's lanes of the warp
    const uint32_t item = (blockIdx.x * kThreads + threadIdx.x) / kWriteLanes;
    if (item >= by.items) return;
    const uint32_t token = divide(item, by.groups), run0 = (item - token * by.groups.d) * R;
    const int64_t from = token * a.x_stride;
    const int e0 = static_cast<int>(run0 * kCacheGroup + lane * 8), d = static_cast<int>(a.c.d);
    Raw<BF16> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) raw[r].x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (e0 + r * kCacheGroup < d) raw[r].load(a.x, from + e0 + r * kCacheGroup);
    }
    const int64_t pos = position_of(a, token);
    if (pos < 0) return;
    int64_t col, place, page = -1;
    if (((pos | a.c.page_size) >> 32) == 0) {  // the common case, without the 64-bit division
        const uint32_t p = static_cast<uint32_t>(pos), ps = static_cast<uint32_t>(a.c.page_size);
        const uint32_t c = quotient(p, ps, by.page_shift);
        col = c;
        place = p - c * ps;
    } else {
        col = pos / a.c.page_size;
        place = pos - col * a.c.page_size;
    }
    if (col < a.t.max_pages) page = __ldg(a.t.table + divide(token, by.per_seq) * a.t.stride + col);
    const bool known = pos < a.rot_rows;
    const float *cos = a.rotation + (known ? pos * a.rot_stride : 0), *sin = cos + a.rot / 2;
    float v[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {  // (the angles do not wait for the page)
        raw[r].values(v[r]);
        const int e = e0 + r * kCacheGroup, at = e - a.first;  // place in the rotated run
        if (at < 0 || at >= a.rot || !known) continue;
        if (a.interleaved) {
            float c[4], s[4];
            *reinterpret_cast<float4 *>(c) = __ldg(reinterpret_cast<const float4 *>(cos + at / 2));
            *reinterpret_cast<float4 *>(s) = __ldg(reinterpret_cast<const float4 *>(sin + at / 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[r][2 * i], y = v[r][2 * i + 1];
                v[r][2 * i] = turned_first(x, y, c[i], s[i]);
                v[r][2 * i + 1] = turned_second(x, y, c[i], s[i]);
            }
        } else {
            const bool second = at >= a.rot / 2;
            const int j = second ? at - a.rot / 2 : at;
            float w[8], c[8], s[8];
            Raw<BF16> other;
            other.load(a.x, from + e + (second ? -(a.rot / 2) : a.rot / 2));
            load8f(cos + j, c);
            load8f(sin + j, s);
            other.values(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[r][i] = second ? turned_second(w[i], v[r][i], c[i], s[i]) : turned_first(v[r][i], w[i], c[i], s[i]);
        }
    }
    if (!known || page < 0 || page >= a.c.pages) {
        if (lane == 0 && run0 == 0 && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
        return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t run = run0 + r, e = static_cast<uint32_t>(e0 + r * kCacheGroup);
        if (run * kCacheGroup < static_cast<uint32_t>(d))
            store_run(a.c, page, place, run, e, lane, half, e < static_cast<uint32_t>(d), v[r]);
    }
}

__device__ __forceinline__ void store8(uint16_t *to, const float v[8])
{
    __nv_bfloat162 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<uint4 *>(o);
}

// Values that were bf16, as they were (a rounding would change the bits of some NaN).
__device__ __forceinline__ void keep8(uint16_t *to, const float v[8])
{
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4 *>(to) = make_uint4(o[0], o[1], o[2], o[3]);
}

// Units of the queries: `each` a head, `per_token` a token's.  Unit n of a CTA's, whose first one is unit `in_token` of
// token `token0`: its token, head and place among the head's.
struct Units {
    int64_t total;
    Divisor per_token, each;
};
struct Unit {
    int64_t token;
    uint32_t head;
    int at;
};
__device__ __forceinline__ Unit unit_of(const Units &u, int64_t token0, uint32_t n)
{
    const uint32_t t = divide(n, u.per_token), r = n - t * u.per_token.d, head = divide(r, u.each);
    return Unit{token0 + t, head, static_cast<int>(r - head * u.each.d)};
}

// 16 elements a thread: 8 pairs.
__device__ __forceinline__ void turn_queries(const CacheAppendArgs &a, const Units &of, uint32_t block)
{
    const int64_t first = static_cast<int64_t>(block) * kThreads, token0 = first / of.per_token.d;
    if (first + threadIdx.x >= of.total) return;
    const Unit n = unit_of(of, token0, static_cast<uint32_t>(first - token0 * of.per_token.d) + threadIdx.x);
    const int64_t pos = position_of(a, n.token);
    const int e = a.first + n.at * (a.interleaved ? 16 : 8), second = a.interleaved ? 8 : a.rot / 2;
    const int64_t from = n.token * a.q_row_stride + n.head * a.q_head_stride + e;
    float u[8], v[8];
    load8(a.q, a.q_bf16 != 0, from, u);
    load8(a.q, a.q_bf16 != 0, from + second, v);
    uint16_t *to = a.q_out + (n.token * a.h + n.head) * a.c.d + e;
    if (pos < 0 || pos >= a.rot_rows) {
        if (a.q_bf16) {
            keep8(to, u);
            keep8(to + second, v);
            return;
        }
    } else {
        const float *cos = a.rotation + pos * a.rot_stride + n.at * 8;
        float c[8], s[8];
        load8f(cos, c);
        load8f(cos + a.rot / 2, s);
        if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = u[2 * j], y = u[2 * j + 1], z = v[2 * j], w = v[2 * j + 1];
                u[2 * j] = turned_first(x, y, c[j], s[j]);
                u[2 * j + 1] = turned_second(x, y, c[j], s[j]);
                v[2 * j] = turned_first(z, w, c[4 + j], s[4 + j]);
                v[2 * j + 1] = turned_second(z, w, c[4 + j], s[4 + j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = u[j], y = v[j];
                u[j] = turned_first(x, y, c[j], s[j]);
                v[j] = turned_second(x, y, c[j], s[j]);
            }
        }
    }
    store8(to, u);
    store8(to + second, v);
}

// What of the queries is not rotated.
__device__ __forceinline__ void copy_queries(const CacheAppendArgs &a, const Units &of, uint32_t block)
{
    const int64_t first = static_cast<int64_t>(block) * (kThreads * kCopies), token0 = first / of.per_token.d;
    const uint32_t in_token = static_cast<uint32_t>(first - token0 * of.per_token.d) + threadIdx.x;
    int64_t from[kCopies], to[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const Unit n = unit_of(of, token0, in_token + i * kThreads);
        const int e = n.at * 8 + (n.at * 8 >= a.first ? a.rot : 0);
        from[i] = n.token * a.q_row_stride + n.head * a.q_head_stride + e;
        to[i] = first + threadIdx.x + i * kThreads < of.total ? (n.token * a.h + n.head) * a.c.d + e : -1;
    }
    if (a.q_bf16) {
        uint4 x[kCopies];
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            if (to[i] >= 0) x[i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + from[i]));
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            if (to[i] >= 0) *reinterpret_cast<uint4 *>(a.q_out + to[i]) = x[i];
    } else {
        float x[kCopies][8];
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            if (to[i] >= 0) load8(a.q, false, from[i], x[i]);
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            if (to[i] >= 0) store8(a.q_out + to[i], x[i]);
    }
}

// The bytes bound what has queries: 8192 tokens of 512 with 16 heads' queries, bf16, 48.7 us in a graph, 5.8 TB/s; all in
// one kind of unit, where every warp waited for some lane's angles, 110 us.  32 tokens with 64 heads' take 3 us: the
// position, then the page and the angles, then the store.
struct Blocks {
    uint32_t rows, turns;  // CTAs of the rows, of what is rotated of the queries; the rest copy
};

// Runs of a token that a group of lanes takes at most, where there are many, and CTAs an SM (64 registers, 48).  16384 rows
// of 512, bf16 to 8 bits: 7.9 us; 13.0 a run at a time (the position, its page and what follows from them formed four
// times), 9.3 by two runs.  From fp32, 4101 rows of 192 and 24 queries: 20.5 us, 21.3 with 64 registers.
template <bool BF16>
struct Shape {
    static constexpr int runs = BF16 ? 4 : 2, ctas = BF16 ? 4 : 5;
};

// Runs that a group of lanes takes of tokens of `runs` runs, where there are many: no more than a row has, since what is
// held for the others costs registers all the same.  65536 rows from bf16 to 8 bits by 1, 2 and 4 runs: of 128 elements
// 14.2, 14.2, 16.9 us, of 256 27.3, 17.3, 20.1, of 320 38.4, 31.7, 22.4, of 512 49.6, 34.2, 27.6; from fp32 by 1 and 2:
// of 128 13.6, 15.4, of 256 25.5, 19.8, of 384 36.1, 35.8, of 512 45.2, 37.3.
int deep_of(int64_t runs, bool bf16)
{
    const int most = bf16 ? Shape<true>::runs : Shape<false>::runs;
    return runs == 1 ? 1 : runs == 2 ? 2 : most;
}

template <int R, bool BF16>
__global__ void __launch_bounds__(kThreads, Shape<BF16>::ctas)
    cache_append_kernel(const CacheAppendArgs a, Blocks blocks, Rows rows, Units turns, Units copies)
{
    if (blockIdx.x < blocks.rows)
        append_rows<R, BF16>(a, rows);
    else if (blockIdx.x < blocks.rows + blocks.turns)
        turn_queries(a, turns, blockIdx.x - blocks.rows);
    else
        copy_queries(a, copies, blockIdx.x - blocks.rows - blocks.turns);
}

Units units_of_queries(const CacheAppendArgs &a, int64_t each)
{
    const int64_t per_token = a.h * each;
    return Units{a.tokens * per_token, divisor_of(static_cast<uint32_t>(per_token > 0 ? per_token : 1)),
                 divisor_of(static_cast<uint32_t>(each > 0 ? each : 1))};
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t s)
{
    const int64_t runs = (a.c.d + kCacheGroup - 1) / kCacheGroup;
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 1, per_block = kThreads / kWriteLanes;
    // few rows: a group of lanes for each run (rows of 512, bf16 to 8 bits, by one run and by four: 2432 rows 3.3 and 3.4 us,
    // 3500 4.5 and 3.6)
    const int64_t deep = a.tokens * runs > 4 * sms * per_block ? deep_of(runs, a.x_bf16 != 0) : 1;
    const int64_t groups = (runs + deep - 1) / deep, items = a.tokens * groups;
    const int64_t row_blocks = (items + per_block - 1) / per_block;
    // (rotated where they are, the queries' other elements stay)
    const Units turns = units_of_queries(a, a.rot / 16), copies = units_of_queries(a, a.q_out == a.q ? 0 : (a.c.d - a.rot) / 8);
    const int64_t turn_blocks = (turns.total + kThreads - 1) / kThreads;
    const int64_t grid = row_blocks + turn_blocks + (copies.total + kThreads * kCopies - 1) / (kThreads * kCopies);
    if (items > 0x7fffffffLL / kWriteLanes || a.h * a.c.d > 0x7fffffffLL || grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const Blocks blocks{static_cast<uint32_t>(row_blocks), static_cast<uint32_t>(turn_blocks)};
    const Rows rows{static_cast<uint32_t>(items), divisor_of(static_cast<uint32_t>(groups)),
                    divisor_of(static_cast<uint32_t>(a.t.rows_per_seq)), shift_of(a.c.page_size)};
    auto kernel = a.x_bf16 ? (deep == 4 ? cache_append_kernel<4, true> : deep == 2 ? cache_append_kernel<2, true> : cache_append_kernel<1, true>)
                           : (deep == 2 ? cache_append_kernel<2, false> : cache_append_kernel<1, false>);
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, blocks, rows, turns, copies);
    return cudaGetLastError();
}

}  // namespace sel
