// cache_rows.cuh -- new rows on their way into a paged cache, shared by the kernels that write them (cache.cu,
// cache_append.cu): elements loaded, a run of 128 rounded or quantised and stored.
//
// An e4m3 row keeps, for each run of 128 elements, one power of two 2^e and the codes x / 2^e rounded
// to nearest even, with the smallest e >= -126 for which 448 * 2^e >= the run's largest finite
// magnitude.  With that magnitude m * 2^E (1 <= m < 2) and 448 = 1.75 * 2^8, e = E - 8, or E - 7 when
// m > 1.75: integer work on the bits, exact.  A power of two leaves 3 significant bits of the code
// untouched, so the value read back is exact in bf16, and dividing by it rounds nothing.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"

namespace sel {
namespace {

constexpr int kWriteLanes = 16;   // lanes of one run of 128 elements, 8 elements each

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

// a / b for 32-bit a; shift: log2(b), or -1 when b is no power of two.
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b, int shift) { return shift >= 0 ? a >> shift : a / b; }

// The lane's 8 elements v (from element e of the row, `in`: there are any) of run `run` into place `place` of page
// `page`, by all of the run's lanes of the warp (`half`).
__device__ __forceinline__ void store_run(const CacheRef &c, int64_t page, int64_t place, uint32_t run, uint32_t e,
                                          uint32_t lane, unsigned half, bool in, const float v[8])
{
    const int64_t at = page * c.page_stride + place * c.row_stride + e;
    if (!c.scales) {
        if (in) {
            __nv_bfloat162 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.data) + at) = *reinterpret_cast<uint4 *>(o);
        }
        return;
    }
    // the largest finite magnitude (a maximum passes over NaN; with an infinity it is formed again without)
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
    for (int s = kWriteLanes / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(half, top, s));
    if (isinf(top)) {
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, isinf(v[i]) ? 0.0f : fabsf(v[i]));
#pragma unroll
        for (int s = kWriteLanes / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(half, top, s));
    }
    const uint32_t bits = __float_as_uint(top);
    int power = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
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
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.data) + at) = make_uint2(o[0], o[1]);
    }
    if (lane == 0)
        c.scales[page * c.scale_page_stride + place * c.scale_row_stride + run] =
            __uint_as_float(static_cast<uint32_t>(power + 127) << 23);
}

// log2(n), or -1 when n is no power of two (or 2^32 and more).
inline int shift_of(int64_t n)
{
    int s = 0;
    while (s < 31 && (int64_t{1} << s) < n) ++s;
    return (int64_t{1} << s) == n ? s : -1;
}

}  // namespace
}  // namespace sel
