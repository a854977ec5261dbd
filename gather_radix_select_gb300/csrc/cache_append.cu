// cache_append.cu -- new rows appended to a paged cache at their positions, rotated on the way, and the same tokens'
// queries rotated alike, in one launch.
//
// A pair (u, v) of the run [first, first + rot) becomes (u cos - v sin, v cos + u sin), with the cosine and sine of
// the token's position and the pair's index out of a table.  Both products and their sum are rounded to fp32, each
// once (no fused multiply-add: the bits do not depend on which of the pair's values is formed where), the result once
// more to what it is held in.
//
// The first CTAs take the rows, the others the queries.  Rows go by runs of 128 elements as in cache_write_kernel; a
// lane that holds 8 elements of a rotated run whose pairs lie half the run apart loads the 8 partners too (they are
// in L1 or on their way there: the other lanes' own).  Queries go by units: 8 elements that stay as they are, or 16
// that make 8 pairs, so that whoever reads a value is who writes it and queries can be rotated where they are.
#include <cstdint>

#include "cache_internal.h"
#include "cache_rows.cuh"

namespace sel {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;  // units of queries a thread takes, all of their loads under way at once

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

__device__ __forceinline__ void append_rows(const CacheAppendArgs &a, uint32_t runs, int runs_shift, uint32_t items)
{
    const uint32_t lane = threadIdx.x & (kWriteLanes - 1);
    const unsigned half = 0xffffu << (threadIdx.x & 16);  // this run's lanes of the warp
    const uint32_t item = (blockIdx.x * kThreads + threadIdx.x) / kWriteLanes;
    if (item >= items) return;
    const uint32_t token = quotient(item, runs, runs_shift), run = item - token * runs;
    const uint32_t e = run * kCacheGroup + lane * 8;
    const bool in = e < a.c.d;
    const int64_t pos = position_of(a, token);
    const int at = static_cast<int>(e) - a.first;  // place in the rotated run
    const bool turn = in && at >= 0 && at < a.rot;
    const bool apart = turn && !a.interleaved, second = at >= a.rot / 2;  // pairs half the run apart
    float v[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i] = 0.0f;
    if (in) load8(a.x, a.x_bf16 != 0, token * a.x_stride + e, v);
    if (apart) load8(a.x, a.x_bf16 != 0, token * a.x_stride + e + (second ? -(a.rot / 2) : a.rot / 2), w);
    if (pos < 0) return;
    const int64_t seq = token / static_cast<uint32_t>(a.t.rows_per_seq);  // (tokens are below 2^31)
    int64_t page, place;
    if (pos >= a.rot_rows || !find_row(a.c, a.t, seq, pos, page, place)) {
        if (lane == 0 && run == 0 && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
        return;
    }
    if (turn) {
        const float *cos = a.rotation + pos * a.rot_stride, *sin = cos + a.rot / 2;
        float c[8], s[8];
        if (apart) {
            const int j = second ? at - a.rot / 2 : at;
            load8f(cos + j, c);
            load8f(sin + j, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = second ? turned_second(w[i], v[i], c[i], s[i]) : turned_first(v[i], w[i], c[i], s[i]);
        } else {
            *reinterpret_cast<float4 *>(c) = __ldg(reinterpret_cast<const float4 *>(cos + at / 2));
            *reinterpret_cast<float4 *>(s) = __ldg(reinterpret_cast<const float4 *>(sin + at / 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[2 * i], y = v[2 * i + 1];
                v[2 * i] = turned_first(x, y, c[i], s[i]);
                v[2 * i + 1] = turned_second(x, y, c[i], s[i]);
            }
        }
    }
    store_run(a.c, page, place, run, e, lane, half, in, v);
}

__device__ __forceinline__ void store8(uint16_t *to, const float v[8])
{
    __nv_bfloat162 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<uint4 *>(o);
}

// per_token: units of a token's queries, by_head: of one head's, the rotated ones first.
__device__ __forceinline__ void turn_queries(const CacheAppendArgs &a, uint32_t block, Divisor per_token, Divisor by_head)
{
    const int64_t first = static_cast<int64_t>(block) * (kThreads * kUnits), total = a.tokens * per_token.d;
    const int64_t token0 = first / per_token.d;
    const uint32_t in_token = static_cast<uint32_t>(first - token0 * per_token.d) + threadIdx.x;
    const int pairs = a.rot / 16;
    float u[kUnits][8], v[kUnits][8];
    int64_t token[kUnits], to[kUnits];
    int unit[kUnits], second[kUnits];  // second: elements from a unit's first 8 to its other 8; 0: there are none
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t n = in_token + i * kThreads;
        const uint32_t t = divide(n, per_token), r = n - t * per_token.d, head = divide(r, by_head);
        const int un = static_cast<int>(r - head * by_head.d);
        token[i] = token0 + t;
        unit[i] = un;
        second[i] = un >= pairs ? 0 : a.interleaved ? 8 : a.rot / 2;
        // (units past the rotated ones pass over them)
        const int e = un < pairs ? a.first + un * (a.interleaved ? 16 : 8)
                                 : (un - pairs) * 8 + ((un - pairs) * 8 >= a.first ? a.rot : 0);
        to[i] = (token[i] * a.h + head) * a.c.d + e;
        if (first + threadIdx.x + i * kThreads >= total) {
            unit[i] = -1;
            continue;
        }
        const int64_t from = token[i] * a.q_row_stride + head * a.q_head_stride + e;
        load8(a.q, a.q_bf16 != 0, from, u[i]);
        if (second[i]) load8(a.q, a.q_bf16 != 0, from + second[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (unit[i] < 0) continue;
        if (second[i]) {
            const int64_t pos = position_of(a, token[i]);
            if (pos >= 0 && pos < a.rot_rows) {
                const float *cos = a.rotation + pos * a.rot_stride + unit[i] * 8;
                float c[8], s[8];
                load8f(cos, c);
                load8f(cos + a.rot / 2, s);
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = u[i][2 * j], y = u[i][2 * j + 1], z = v[i][2 * j], w = v[i][2 * j + 1];
                        u[i][2 * j] = turned_first(x, y, c[j], s[j]);
                        u[i][2 * j + 1] = turned_second(x, y, c[j], s[j]);
                        v[i][2 * j] = turned_first(z, w, c[4 + j], s[4 + j]);
                        v[i][2 * j + 1] = turned_second(z, w, c[4 + j], s[4 + j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x = u[i][j], y = v[i][j];
                        u[i][j] = turned_first(x, y, c[j], s[j]);
                        v[i][j] = turned_second(x, y, c[j], s[j]);
                    }
                }
            }
            store8(a.q_out + to[i] + second[i], v[i]);
        }
        store8(a.q_out + to[i], u[i]);
    }
}

__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheAppendArgs a, uint32_t row_blocks,
                                                                uint32_t runs, int runs_shift, uint32_t items,
                                                                Divisor per_token, Divisor by_head)
{
    if (blockIdx.x < row_blocks)
        append_rows(a, runs, runs_shift, items);
    else
        turn_queries(a, blockIdx.x - row_blocks, per_token, by_head);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t s)
{
    const int64_t runs = (a.c.d + kCacheGroup - 1) / kCacheGroup;
    const int64_t items = a.tokens * runs, row_blocks = (items * kWriteLanes + kThreads - 1) / kThreads;
    // rotated where they are, the queries' other elements stay
    const int64_t by_head = a.rot / 16 + (a.q_out == a.q ? 0 : (a.c.d - a.rot) / 8), per_token = a.q ? a.h * by_head : 0;
    const int64_t q_blocks = (a.tokens * per_token + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (items > 0x7fffffffLL / kWriteLanes || per_token > (int64_t{1} << 30) || row_blocks + q_blocks > 0x7fffffffLL)
        return cudaErrorInvalidValue;
    cache_append_kernel<<<static_cast<unsigned>(row_blocks + q_blocks), kThreads, 0, s>>>(
        a, static_cast<uint32_t>(row_blocks), static_cast<uint32_t>(runs), shift_of(runs), static_cast<uint32_t>(items),
        divisor_of(static_cast<uint32_t>(per_token > 0 ? per_token : 1)), divisor_of(static_cast<uint32_t>(by_head > 0 ? by_head : 1)));
    return cudaGetLastError();
}

}  // namespace sel
