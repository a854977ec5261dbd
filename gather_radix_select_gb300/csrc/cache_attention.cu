// cache_attention.cu -- attention of new tokens over a paged cache: the plain kernel.
//
// One CTA per (row, head).  Tiles of kTile positions: each thread forms the score of one key row, the
// tile's largest score joins the running maximum, the running sum and accumulators are rescaled by
// exp2(old - new), and each thread then adds its value columns' share.  Everything is in fp32.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"

namespace sel {
namespace {

constexpr int kTile = 256;
constexpr int kMaxD = 512;

__device__ __forceinline__ float elem(const CacheRef &c, int64_t row, int64_t srow, int e)
{
    if (!c.scales)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(c.data)[row + e]) << 16);
    const __nv_fp8_storage_t code = static_cast<const uint8_t *>(c.data)[row + e];
    const float v = __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))) * c.scales[srow + e / kCacheGroup];
    return __bfloat162float(__float2bfloat16_rn(v));
}

__global__ void __launch_bounds__(kTile) attention_plain_kernel(const CacheAttnArgs a)
{
    __shared__ float s_q[kMaxD];
    __shared__ float s_p[kTile];
    __shared__ int64_t s_row[kTile], s_scale[kTile];
    __shared__ float s_red[kTile / 32];
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int head = blockIdx.y;
    const int64_t seq = row / a.t.rows_per_seq;
    const uint16_t *q = a.q + row * a.q_row_stride + head * a.q_head_stride;
    for (int e = t; e < a.d; e += kTile) s_q[e] = __uint_as_float(static_cast<uint32_t>(q[e]) << 16);
    const int64_t cap = a.t.max_pages * a.c.page_size;
    int64_t end = a.end ? a.end[row] : cap;
    end = end < 0 ? 0 : (end > cap ? cap : end);
    const int64_t keys = a.idx ? a.n : end;
    float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int64_t k0 = 0; k0 < keys; k0 += kTile) {
        __syncthreads();
        int64_t pos = -1;
        if (k0 + t < keys) {
            pos = k0 + t;
            if (a.idx) {
                const int64_t off = row * a.idx_row_stride + k0 + t;
                pos = a.idx_i64 ? static_cast<const int64_t *>(a.idx)[off]
                                : static_cast<int64_t>(static_cast<const int32_t *>(a.idx)[off]);
                const bool past = pos >= cap;
                if (past && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
                if (pos >= end) pos = -1;
            }
        }
        int64_t page = 0, place = 0;
        float z = -INFINITY;
        int64_t at = -1, sat = 0;
        if (pos >= 0) {
            if (find_row(a.c, a.t, seq, pos, page, place)) {
                at = page * a.c.page_stride + place * a.c.row_stride;
                sat = page * a.c.scale_page_stride + place * a.c.scale_row_stride;
                float dot = 0.0f;
                for (int e = 0; e < a.d; ++e) dot += s_q[e] * elem(a.c, at, sat, e);
                z = dot * a.scale_log2;
            } else if (a.err_flag) {
                atomicCAS(a.err_flag, 0, kCacheInval);
            }
        }
        s_row[t] = at;
        s_scale[t] = sat;
        float zm = z;
        for (int o = 16; o > 0; o >>= 1) zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, o));
        if ((t & 31) == 0) s_red[t >> 5] = zm;
        __syncthreads();
        float m_new = m;
        for (int w = 0; w < kTile / 32; ++w) m_new = fmaxf(m_new, s_red[w]);
        const float base = m_new == -INFINITY ? 0.0f : m_new;
        const float p = at < 0 ? 0.0f : exp2f(z - base);
        const float f = exp2f(m - base);
        s_p[t] = __bfloat162float(__float2bfloat16_rn(p));
        float ps = p;
        for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        __syncthreads();
        if ((t & 31) == 0) s_red[t >> 5] = ps;
        __syncthreads();
        float sum = 0.0f;
        for (int w = 0; w < kTile / 32; ++w) sum += s_red[w];
        l = l * f + sum;
        m = m_new;
        for (int i = 0; i < 2; ++i) {
            const int e = t + i * kTile;
            if (e >= a.dv) continue;
            float o = acc[i] * f;
            for (int k = 0; k < kTile; ++k)
                if (s_row[k] >= 0) o += s_p[k] * elem(a.c, s_row[k], s_scale[k], e);
            acc[i] = o;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t o = (row * a.h + head) * a.dv;
    for (int i = 0; i < 2; ++i) {
        const int e = t + i * kTile;
        if (e < a.dv) reinterpret_cast<__nv_bfloat16 *>(a.out)[o + e] = __float2bfloat16_rn(acc[i] * inv);
    }
    if (t == 0 && a.lse) a.lse[row * a.h + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t cache_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, bool) { return 0; }

cudaError_t launch_cache_attention(const CacheAttnArgs &a, cudaStream_t s)
{
    if (a.rows > 0x7fffffffLL || a.h > 65535) return cudaErrorInvalidValue;
    attention_plain_kernel<<<dim3(static_cast<unsigned>(a.rows), static_cast<unsigned>(a.h)), kTile, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sel
