// cache.cu -- rows of a paged key cache: written (quantised) at their slots, read back at positions.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"
#include "cache_rows.cuh"

namespace sel {
namespace {

constexpr int kWriteThreads = 128;
constexpr int kGatherPairs = 128; // positions handled by one CTA at most

// One run of 128 elements of one token by 16 lanes.  The elements are on their way while the slot is read.
// To 8 bits no unit is near its limit (42% of the issue slots over the kernel's time, 20% of the DRAM bandwidth):
// each of the many short CTAs is a chain of loads, shuffles and conversions.  Divisions by powers of two are
// shifts and the magnitudes a floating-point maximum.  16384 rows of 512 to 8 bits take 10.2 us a call for 25 MB,
// 6.8 us one after the other in a graph; 100001 rows of 128 fp32 to bf16 14.4 us and 8.2 us for 77 MB.  32 rows,
// 1.8 us in a graph, are two loads one after the other.
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheWriteArgs a, uint32_t runs, int runs_shift,
                                                                    int page_shift, uint32_t items)
{
    const uint32_t lane = threadIdx.x & (kWriteLanes - 1);
    const unsigned half = 0xffffu << (threadIdx.x & 16);  // this run's lanes of the warp
    const uint32_t item = (blockIdx.x * kWriteThreads + threadIdx.x) / kWriteLanes;
    if (item >= items) return;
    const uint32_t token = quotient(item, runs, runs_shift), run = item - token * runs;
    const uint32_t e = run * kCacheGroup + lane * 8;
    const bool in = e < a.c.d;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (in) load8(a.x, a.x_bf16 != 0, token * a.x_stride + e, v);
    const int64_t slot = a.slots_i64 ? __ldg(static_cast<const int64_t *>(a.slots) + token)
                                     : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(a.slots) + token));
    if (slot < 0) return;
    int64_t page, place;
    if (((slot | a.c.page_size) >> 32) == 0) {  // the common case, without the 64-bit division
        const uint32_t s = static_cast<uint32_t>(slot), ps = static_cast<uint32_t>(a.c.page_size);
        const uint32_t q = quotient(s, ps, page_shift);
        page = q;
        place = s - q * ps;
    } else {
        page = slot / a.c.page_size;
        place = slot - page * a.c.page_size;
    }
    if (page >= a.c.pages) {
        if (lane == 0 && run == 0 && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
        return;
    }
    store_run(a.c, page, place, run, e, lane, half, in, v);
}

// 8 codes times their scale, rounded to bf16 (exact for powers of two).
__device__ __forceinline__ uint4 decode8(uint2 codes, float scale)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = ((i & 2 ? codes.y : codes.x) >> (16 * (i & 1))) & 0xffffu;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        w[i] = *reinterpret_cast<const uint32_t *>(&o);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per run of positions, of whatever rows: their cache rows are found once, then copied 16 output
// bytes a lane, four vectors under way at a time.  (By runs within a row short lists left most of a CTA idle:
// 26334 rows x 7 positions of 256 took 45.5 us, now 19.  8 CTAs an SM: with the 36 registers that
// 8-bit rows take unbounded, 16 x 512 positions would be more than one wave, 7.5 against 6.3 us.)
// The output's bytes bound it: 4096 rows x 512 positions of 128 elements (537 MB out, the cache's rows from L2)
// take 78 us, 6.9 TB/s; 1024 x 512 positions of 8-bit rows of 512 (as many bytes out) 83.5 us.
template <bool FP8>
__global__ void __launch_bounds__(kGatherThreads, 8) cache_gather_kernel(const CacheGatherArgs a)
{
    __shared__ int64_t s_row[kGatherPairs];    // element offset of the cache row, -1: none
    __shared__ int64_t s_scale[kGatherPairs];
    const int64_t total = a.rows * a.n, first = static_cast<int64_t>(blockIdx.x) * a.pairs;
    const int np = static_cast<int>(total - first < a.pairs ? total - first : a.pairs);
    for (int i = threadIdx.x; i < np; i += kGatherThreads) {
        const int64_t at_i = first + i;
        int64_t row, seq;
        if (total >> 32 == 0) {  // the common case, without the 64-bit divisions
            row = static_cast<uint32_t>(at_i) / static_cast<uint32_t>(a.n);
            seq = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.t.rows_per_seq);
        } else {
            row = at_i / a.n;
            seq = row / a.t.rows_per_seq;
        }
        const int64_t off = row * a.idx_row_stride + (at_i - row * a.n);
        int64_t p = a.idx_i64 ? static_cast<const int64_t *>(a.idx)[off]
                              : static_cast<int64_t>(static_cast<const int32_t *>(a.idx)[off]);
        p = p < 0 ? 0 : p;
        int64_t page, place;
        int64_t at = -1;
        if (find_row(a.c, a.t, seq, p, page, place)) {
            at = page * a.c.page_stride + place * a.c.row_stride;
            if (FP8) s_scale[i] = page * a.c.scale_page_stride + place * a.c.scale_row_stride;
        } else if (a.err_flag) {
            atomicCAS(a.err_flag, 0, kCacheInval);
        }
        s_row[i] = at;
    }
    __syncthreads();
    const int vpr = static_cast<int>(a.c.d >> 3);
    const int vsh = (vpr & (vpr - 1)) == 0 ? __ffs(vpr) - 1 : -1;
    uint4 *out = reinterpret_cast<uint4 *>(a.out + first * a.c.d);
    const int vecs = np * vpr;
    constexpr int U = 4;
    for (int t0 = threadIdx.x; t0 < vecs; t0 += U * kGatherThreads) {
        uint4 v[U];
        float sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * kGatherThreads;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 0.0f;
            if (t < vecs) {
                const int jj = vsh >= 0 ? (t >> vsh) : t / vpr;
                const int c = t - jj * vpr;
                const int64_t r = s_row[jj];
                if (r >= 0) {
                    if (FP8) {
                        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.c.data) + r) + c);
                        v[u].x = w.x;
                        v[u].y = w.y;
                        sc[u] = __ldg(a.c.scales + s_scale[jj] + (c >> 4));
                    } else {
                        v[u] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.c.data) + r) + c);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * kGatherThreads;
            if (t < vecs) __stcs(out + t, FP8 ? decode8(make_uint2(v[u].x, v[u].y), sc[u]) : v[u]);
        }
    }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t s)
{
    const int64_t runs = (a.c.d + kCacheGroup - 1) / kCacheGroup;
    const int64_t items = a.tokens * runs, grid = (items * kWriteLanes + kWriteThreads - 1) / kWriteThreads;
    if (grid <= 0) return cudaSuccess;
    if (items > 0x7fffffffLL / kWriteLanes) return cudaErrorInvalidValue;
    cache_write_kernel<<<static_cast<unsigned>(grid), kWriteThreads, 0, s>>>(
        a, static_cast<uint32_t>(runs), shift_of(runs), shift_of(a.c.page_size), static_cast<uint32_t>(items));
    return cudaGetLastError();
}

cudaError_t launch_cache_gather(const CacheGatherArgs &a_in, cudaStream_t s)
{
    CacheGatherArgs a = a_in;
    // few positions: fewer a CTA, down to 8, so that there are 4 CTAs for every SM (16 rows x 512 positions of 512
    // elements: 6.3 us, with 128 positions a CTA 10.4)
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 1;
    const int64_t total = a.rows * a.n;
    int64_t pairs = kGatherPairs;
    while (pairs > 8 && (total + pairs - 1) / pairs < 4 * sms) pairs /= 2;
    a.pairs = static_cast<int32_t>(pairs);
    const int64_t grid = (total + pairs - 1) / pairs;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.c.scales)
        cache_gather_kernel<true><<<static_cast<unsigned>(grid), kGatherThreads, 0, s>>>(a);
    else
        cache_gather_kernel<false><<<static_cast<unsigned>(grid), kGatherThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sel
