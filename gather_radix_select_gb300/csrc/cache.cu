// cache.cu -- rows of a paged key cache: written (quantised) at their slots, read back at positions.
//
// An e4m3 row keeps, for each run of 128 elements, one power of two 2^e and the codes x / 2^e rounded
// to nearest even, with the smallest e >= -126 for which 448 * 2^e >= the run's largest finite
// magnitude.  With that magnitude m * 2^E (1 <= m < 2) and 448 = 1.75 * 2^8, e = E - 8, or E - 7 when
// m > 1.75: integer work on the bits, exact.  A power of two leaves 3 significant bits of the code
// untouched, so the value read back is exact in bf16, and dividing by it rounds nothing.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"

namespace sel {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kWriteLanes = 16;   // lanes of one run of 128 elements, 8 elements each
constexpr int kGatherPairs = 128; // positions of one row handled by one CTA

__device__ __forceinline__ void load8(const void *x, bool bf16, int64_t at, float v[8])
{
    if (bf16) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at));
        const float4 b = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// One run of 128 elements of one token by 16 lanes.
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheWriteArgs a, uint32_t runs)
{
    const uint32_t lane = threadIdx.x & (kWriteLanes - 1);
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * kWriteThreads + threadIdx.x) / kWriteLanes;
    const int64_t token = item / runs;
    const uint32_t run = static_cast<uint32_t>(item - token * runs);
    const unsigned half = 0xffffu << (threadIdx.x & 16);  // this run's lanes of the warp
    if (token >= a.tokens) return;
    const int64_t slot = a.slots_i64 ? static_cast<const int64_t *>(a.slots)[token]
                                     : static_cast<int64_t>(static_cast<const int32_t *>(a.slots)[token]);
    if (slot < 0) return;
    const int64_t page = slot / a.c.page_size, place = slot - page * a.c.page_size;
    if (page >= a.c.pages) {
        if (lane == 0 && run == 0 && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
        return;
    }
    const int64_t e = static_cast<int64_t>(run) * kCacheGroup + lane * 8;
    const bool in = e < a.c.d;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (in) load8(a.x, a.x_bf16 != 0, token * a.x_stride + e, v);
    const int64_t row = page * a.c.page_stride + place * a.c.row_stride;
    if (!a.c.scales) {
        if (in) {
            __nv_bfloat162 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.c.data) + row + e) = *reinterpret_cast<uint4 *>(o);
        }
        return;
    }
    uint32_t top = 0;  // bits of the largest finite magnitude
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __float_as_uint(v[i]) & 0x7fffffffu;
        top = max(top, m < 0x7f800000u ? m : 0u);
    }
#pragma unroll
    for (int s = kWriteLanes / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(half, top, s));
    int power = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    power = max(power, -126);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - power) << 23);
    if (in) {
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            o[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.c.data) + row + e) = make_uint2(o[0], o[1]);
    }
    if (lane == 0)
        a.c.scales[page * a.c.scale_page_stride + place * a.c.scale_row_stride + run] =
            __uint_as_float(static_cast<uint32_t>(power + 127) << 23);
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

// One CTA per run of positions of one row: their cache rows are found once, then copied 16 output
// bytes a lane.
template <bool FP8>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const CacheGatherArgs a)
{
    __shared__ int64_t s_row[kGatherPairs];    // element offset of the cache row, -1: none
    __shared__ int64_t s_scale[kGatherPairs];
    const int64_t row = blockIdx.x / a.ctas_per_row;
    const int64_t j0 = (blockIdx.x - row * a.ctas_per_row) * kGatherPairs;
    const int np = static_cast<int>(a.n - j0 < kGatherPairs ? a.n - j0 : kGatherPairs);
    const int64_t seq = row / a.t.rows_per_seq;
    for (int i = threadIdx.x; i < np; i += kGatherThreads) {
        const int64_t off = row * a.idx_row_stride + j0 + i;
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
    uint4 *out = reinterpret_cast<uint4 *>(a.out + (row * a.n + j0) * a.c.d);
    const int total = np * vpr;
    constexpr int U = 4;
    for (int t0 = threadIdx.x; t0 < total; t0 += U * kGatherThreads) {
        uint4 v[U];
        float sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * kGatherThreads;
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 0.0f;
            if (t < total) {
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
            if (t < total) __stcs(out + t, FP8 ? decode8(make_uint2(v[u].x, v[u].y), sc[u]) : v[u]);
        }
    }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t s)
{
    const int64_t runs = (a.c.d + kCacheGroup - 1) / kCacheGroup;
    const int64_t grid = (a.tokens * runs * kWriteLanes + kWriteThreads - 1) / kWriteThreads;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    cache_write_kernel<<<static_cast<unsigned>(grid), kWriteThreads, 0, s>>>(a, static_cast<uint32_t>(runs));
    return cudaGetLastError();
}

cudaError_t launch_cache_gather(const CacheGatherArgs &a_in, cudaStream_t s)
{
    CacheGatherArgs a = a_in;
    a.ctas_per_row = static_cast<int32_t>((a.n + kGatherPairs - 1) / kGatherPairs);
    const int64_t grid = a.rows * a.ctas_per_row;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.c.scales)
        cache_gather_kernel<true><<<static_cast<unsigned>(grid), kGatherThreads, 0, s>>>(a);
    else
        cache_gather_kernel<false><<<static_cast<unsigned>(grid), kGatherThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sel
