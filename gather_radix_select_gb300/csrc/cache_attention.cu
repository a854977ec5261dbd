// cache_attention.cu -- attention of new tokens over a paged cache, on the fifth-generation tensor cores.
//
// For the columns n = (row, head) of one CTA and a tile of 128 positions with rows K:
//     S^T = K Q^T            [128 positions x 64 columns]
//     P^T = exp2(S^T * scale - ref)
//     O^T += K[:, :dv]^T P^T [dv x 64 columns]
// Positions are the M dimension of the first product and heads its N dimension, so a single token with
// few heads wastes no part of the 128-row instruction, a thread of the softmax holds one position, and
// the value is the key tile itself, read with the other dimension contiguous: each cache row is staged
// once and used for both products.
//
// The sum of exponentials needs no maximum, only a reference that keeps exp2 in range.  `ref` is the
// column's largest score when it was last set; while no score exceeds it by more than 2^8 the tile is
// taken with one vote.  Else the columns' maxima are formed across the positions and the sums and
// accumulators are rescaled.  Sums are kept per thread (its positions) and joined at the end.
//
// A CTA stays on its SM and takes one unit of work (rows x heads x a part of the positions) after the
// other; its 20 warps are 8 of softmax (two groups of 4: 32 columns each), one that issues the products,
// one that looks up the next unit, 8 that stage queries and rows, the rows in chunks of 128 columns by 128
// positions in a ring.  A chunk is released when its part
// of the second product is done, so the next tile's rows arrive while the rest of the product runs.
//
// Few rows over long contexts are split into parts of the positions, whose sums and accumulators a
// second kernel joins in a fixed order.
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"
#include "tcgen05.cuh"

namespace sel {
namespace {

constexpr int kCols = 64;                  // (row, head) columns of a CTA
constexpr int kTile = 128;                 // positions of a tile
constexpr int kChunkBytes = kTile * 256;   // 128 positions x 128 columns of bf16
constexpr int kHalfBytes = kChunkBytes / 2;  // 64 columns: one 128-byte line a position
constexpr int kQHalf = kCols * 128;        // 64 query columns x 64 elements
constexpr int kPBytes = kTile * 128;       // P^T: 128 positions x 64 columns
constexpr int kSoftWarps = 8, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftWarps;           // its group of 4 warps holds two that work:
constexpr int kUnitWarp = kMmaWarp + 1;        // the one that issues and the one that looks up what is next
constexpr int kLoadWarp0 = kSoftWarps + 4;
constexpr int kThreads = (kLoadWarp0 + kLoadWarps) * 32;
// Registers a thread after the roles part, out of the 640 x 96 of the launch:
// 256 x 136 + 128 x 48 + 256 x 80 = 61440.
constexpr int kSoftRegs = 136, kMmaRegs = 48, kLoadRegs = 80;
constexpr int kMaxRing = 5;
constexpr int kValidSlots = 16;            // tiles whose validity bits are kept (more than the ring holds)
constexpr int kMaxSplit = 64;
constexpr float kRefSlack = 8.0f;          // log2: how far a score may exceed its column's reference
constexpr long long kWaitCycles = 4000000000LL;  // about 2 s
constexpr uint32_t kSuspend = 1000;
constexpr int32_t kTimeout = 5;            // SEL_ETIMEOUT

template <int C>
struct Cfg {
    static constexpr int ring = C <= 1 ? 5 : 4;          // chunks staged
    static constexpr int pbufs = C <= 2 ? 2 : 1;
    static constexpr bool ahead = ring >= 2 * C;         // the next tile's scores before this one's values
    static constexpr int q_off = ring * kChunkBytes;
    static constexpr int p_off = q_off + C * 2 * kQHalf;
    static constexpr int misc_off = p_off + pbufs * kPBytes;
};

// What a CTA works on next, made by one warp ahead of the others.
struct Unit {
    int64_t row0, seq;
    int64_t keys;            // positions, or list entries up to the last valid one
    int64_t list_end;        // exclusive end of the listed positions
    int rows, head0, heads;  // rows and heads of its columns: column = row * heads + head
    int part;
    int lo, n;               // first tile and tiles
    int min_end, max_end;    // of its rows
    alignas(16) int end[kCols];  // exclusive end of each column's row, 0 for unused columns
    __device__ __forceinline__ int cols() const { return rows * heads; }
};

struct Misc {
    uint64_t full[kMaxRing], empty[kMaxRing], s_full[2], s_empty[2], p_full[2], pv_done[2], q_full, q_empty;
    uint64_t unit_full[2], unit_empty[2];
    uint32_t tmem;
    int abort;
    alignas(16) float ref[kCols];  // read 16 bytes at a time
    alignas(16) float factor[kCols];
    alignas(16) float inv[kCols];
    alignas(16) float wmax[4][kCols];
    alignas(16) float lsum[4][kCols];
    alignas(16) uint32_t valid[kValidSlots][4];  // bit k of word w: position 32 w + k of the tile has a cache row
    alignas(16) Unit unit[2];
};
static_assert(offsetof(Misc, ref) % 16 == 0 && offsetof(Misc, factor) % 16 == 0 && offsetof(Misc, valid) % 16 == 0 &&
                  offsetof(Misc, unit) % 16 == 0, "");

struct Plan {
    int rows_per_tile;   // T
    int heads_per_tile;  // heads of a head block
    int head_blocks;
    int64_t tiles_per_seq;
    int64_t items;       // CTAs of one part
    int parts;
};

struct Kargs {
    CacheAttnArgs a;
    Plan p;
    float *part_o;   // [rows * h][parts][dv]
    float2 *part_ml; // [rows * h][parts]: reference (log2), sum
};

struct Waiter {
    volatile int *abort;
    int32_t *err;
    // Waits until the phase of `parity` has completed.  After about 2 s without that, or once another
    // thread gave up, it returns all the same: every loop has a fixed count, so the CTA ends, with
    // SEL_ETIMEOUT in err_flag.
    __device__ __forceinline__ void operator()(uint64_t *bar, int parity) const
    {
        if (!mbar_try_wait(bar, static_cast<uint32_t>(parity), kSuspend)) slow(bar, parity);
        __syncwarp();  // (whole warps wait: none of their lanes falls behind by a phase)
    }
    __device__ __forceinline__ void slow(uint64_t *bar, int parity) const
    {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, static_cast<uint32_t>(parity), kSuspend)) {
            if (*abort) return;
            if (clock64() - t0 > kWaitCycles) {
                *abort = 1;
                if (err) atomicCAS(err, 0, kTimeout);
                return;
            }
        }
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The position in entry j of a row's list, or -1 when it stands for none.
__device__ __forceinline__ int64_t listed(const CacheAttnArgs &a, int64_t row, int64_t j, int64_t end, int64_t cap)
{
    const int64_t off = row * a.idx_row_stride + j;
    const int64_t p = a.idx_i64 ? static_cast<const int64_t *>(a.idx)[off]
                                : static_cast<int64_t>(static_cast<const int32_t *>(a.idx)[off]);
    if (p >= cap && a.err_flag) atomicCAS(a.err_flag, 0, kCacheInval);
    return p < end ? p : -1;
}

// One warp: unit u of the call.
__device__ __forceinline__ void make_unit(const Kargs &k, int64_t u, Unit *w, int lane)
{
    const int64_t cap = k.a.t.max_pages * k.a.c.page_size;
    // the last rows first: in a causal chunk they have the most positions
    const int64_t item = k.p.items - 1 - u / k.p.parts;
    const int part = static_cast<int>(u % k.p.parts);
    const int64_t tile = item / k.p.head_blocks;
    const int hb = static_cast<int>(item - tile * k.p.head_blocks);
    const int64_t seq = tile / k.p.tiles_per_seq;
    const int64_t in_seq = (tile - seq * k.p.tiles_per_seq) * k.p.rows_per_tile;
    const int64_t row0 = seq * k.a.t.rows_per_seq + in_seq;
    const int64_t left = k.a.t.rows_per_seq - in_seq;
    const int rows = static_cast<int>(left < k.p.rows_per_tile ? left : k.p.rows_per_tile);
    const int head0 = hb * k.p.heads_per_tile;
    const int heads = min(k.p.heads_per_tile, k.a.h - head0);
    int least = 0x7fffffff, most = 0;
#pragma unroll
    for (int i = 0; i < kCols / 32; ++i) {
        const int col = i * 32 + lane;
        int e = 0;
        if (col < rows * heads) {
            const int64_t v = k.a.end ? k.a.end[row0 + col / heads] : cap;
            e = static_cast<int>(v < 0 ? 0 : (v > cap ? cap : v));
            least = min(least, e);
            most = max(most, e);
        }
        w->end[col] = e;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    int64_t keys = most;
    if (k.a.idx) {  // one row: its list up to the last entry that counts
        int last = 0;
#pragma unroll 4
        for (int j = lane; j < k.a.n; j += 32)
            if (listed(k.a, row0, j, most, cap) >= 0) last = j + 1;
        keys = __reduce_max_sync(0xffffffffu, last);
    }
    if (lane == 0) {
        const int64_t tiles = (keys + kTile - 1) / kTile;
        w->row0 = row0;
        w->seq = seq;
        w->keys = keys;
        w->list_end = most;
        w->rows = rows;
        w->head0 = head0;
        w->heads = heads;
        w->part = part;
        w->lo = static_cast<int>(tiles * part / k.p.parts);
        w->n = static_cast<int>(tiles * (part + 1) / k.p.parts) - w->lo;
        w->min_end = least;
        w->max_end = most;
    }
}

// ------------------------------------------------------------------------------------ staging rows
// Warp lw of 8 stages positions 16 lw .. 16 lw + 15 of each tile.
struct Loader {
    const Kargs &k;
    Misc *m;
    const Unit *w;
    int64_t cap;
    int lane, lw;
    int stage, phase;  // of the ring; a fresh barrier's phase of parity 1 counts as completed
    int tile;          // tiles staged so far

    struct Rows {
        int64_t row, scale;  // element offsets of the lane's position (lane mod 16); row -1: none
    };

    // Of tile i of the unit.
    __device__ __forceinline__ Rows find(int i) const
    {
        Rows r{-1, 0};
        const int64_t j = static_cast<int64_t>(w->lo + i) * kTile + lw * 16 + (lane & 15);
        if (i < w->n && j < w->keys) {
            const int64_t pos = k.a.idx ? listed(k.a, w->row0, j, w->list_end, cap) : j;
            int64_t page, place;
            if (pos >= 0) {
                if (find_row(k.a.c, k.a.t, w->seq, pos, page, place)) {
                    r.row = page * k.a.c.page_stride + place * k.a.c.row_stride;
                    r.scale = page * k.a.c.scale_page_stride + place * k.a.c.scale_row_stride;
                } else if (k.a.err_flag) {
                    atomicCAS(k.a.err_flag, 0, kCacheInval);
                }
            }
        }
        return r;
    }

    // This warp's 16 validity bits of the next tile.
    __device__ __forceinline__ void note(const Rows &r)
    {
        const uint32_t bits = __ballot_sync(0xffffffffu, r.row >= 0) & 0xffffu;
        if (lane == 0)
            reinterpret_cast<uint16_t *>(m->valid[tile & (kValidSlots - 1)])[lw] = static_cast<uint16_t>(bits);
        ++tile;
    }

    // The unit's queries by all 256 threads; unused columns and elements past d are zeros.
    template <int C>
    __device__ __forceinline__ void queries(unsigned char *q) const
    {
        const int vec = lane & 15, heads = w->heads, cols = w->cols();
        const uint32_t to = smem_addr(q) + (vec >> 3) * kQHalf;
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i) {
            const int col = (i * kLoadWarps + lw) * 2 + (lane >> 4);
            const int row = col / heads;
            const uint16_t *src = k.a.q + (w->row0 + row) * k.a.q_row_stride +
                                  static_cast<int64_t>(w->head0 + col - row * heads) * k.a.q_head_stride;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = c * 128 + vec * 8;
                const bool ok = col < cols && e < k.a.d;
                cp_async16(to + c * 2 * kQHalf + col * 128 + (((vec & 7) ^ (col & 7)) << 4), ok ? src + e : k.a.q,
                           ok ? 16u : 0u);
            }
        }
        cp_async_arrive(&m->q_full);
    }
};

template <int C>
__device__ __forceinline__ void load_bf16(Loader &l, const Waiter &wait, unsigned char *ring)
{
    constexpr int R = Cfg<C>::ring;
    Misc *m = l.m;
    const uint16_t *data = static_cast<const uint16_t *>(l.k.a.c.data);
    const int vec = l.lane & 15, d = l.k.a.d, n = l.w->n;
    const int line0 = l.lw * 16 + (l.lane >> 4);
    const uint32_t to = smem_addr(ring) + (vec >> 3) * kHalfBytes + line0 * 128;
    Loader::Rows next = l.find(0);
    for (int it = 0; it < n; ++it) {
        const Loader::Rows cur = next;
        l.note(cur);
        next = l.find(it + 1);
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            wait(&m->empty[l.stage], l.phase);
            const uint32_t base = to + l.stage * kChunkBytes;
            const int e = c * 128 + vec * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = __shfl_sync(0xffffffffu, cur.row, 2 * i + (l.lane >> 4));
                const bool ok = e < d && row >= 0;
                cp_async16(base + i * 256 + (((vec & 7) ^ ((line0 + 2 * i) & 7)) << 4), data + (ok ? row + e : 0),
                           ok ? 16u : 0u);
            }
            cp_async_arrive(&m->full[l.stage]);
            if (++l.stage == R) l.stage = 0, l.phase ^= 1;
        }
    }
}

// 16 codes times their scale -> 16 bf16 in two 16-byte units.
__device__ __forceinline__ void decode16(uint4 codes, float scale, uint4 &a, uint4 &b)
{
    const uint32_t in[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>((in[i >> 1] >> (16 * (i & 1))) & 0xffffu), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        out[i] = pack_bf16(f.x * scale, f.y * scale);
    }
    a = make_uint4(out[0], out[1], out[2], out[3]);
    b = make_uint4(out[4], out[5], out[6], out[7]);
}

struct CodeChunk {
    uint4 codes[4];
    float scale[4];
};

template <int C>
__device__ __forceinline__ void load_fp8(Loader &l, const Waiter &wait, unsigned char *ring)
{
    constexpr int R = Cfg<C>::ring;
    Misc *m = l.m;
    const uint8_t *data = static_cast<const uint8_t *>(l.k.a.c.data);
    const float *scales = l.k.a.c.scales;
    const int vec = l.lane & 7, d = l.k.a.d;
    const int total = l.w->n * C;
    Loader::Rows cur{-1, 0}, next = l.find(0);
    int fetched = 0, fc = 0, ft = 0;  // next chunk to fetch, its column chunk and tile
    auto fetch = [&](CodeChunk &x) {
        if (fetched >= total) return;
        if (fc == 0) {
            cur = next;
            l.note(cur);
            next = l.find(ft + 1);
        }
        const bool in = fc * 128 + vec * 16 < d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 4 * i + (l.lane >> 3);
            const int64_t row = __shfl_sync(0xffffffffu, cur.row, key);
            const int64_t srow = __shfl_sync(0xffffffffu, cur.scale, key);
            x.codes[i] = make_uint4(0u, 0u, 0u, 0u);
            x.scale[i] = 0.0f;
            if (in && row >= 0) {
                x.codes[i] = *reinterpret_cast<const uint4 *>(data + row + fc * 128 + vec * 16);
                x.scale[i] = scales[srow + fc];
            }
        }
        ++fetched;
        if (++fc == C) fc = 0, ++ft;
    };
    auto store = [&](int g, const CodeChunk &x) {
        if (g >= total) return;
        wait(&m->empty[l.stage], l.phase);
        unsigned char *base = ring + l.stage * kChunkBytes + (vec >> 2) * kHalfBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int line = l.lw * 16 + 4 * i + (l.lane >> 3);
            uint4 a, b;
            decode16(x.codes[i], x.scale[i], a, b);
            const int u = (2 * vec) & 7, sw = line & 7;
            // lanes of the second half store their second unit first: the 8 lanes of a line then
            // cover all banks in each of the two stores
            const bool odd = vec >= 4;
            *reinterpret_cast<uint4 *>(base + line * 128 + (((u + odd) ^ sw) << 4)) = odd ? b : a;
            *reinterpret_cast<uint4 *>(base + line * 128 + (((u + !odd) ^ sw) << 4)) = odd ? a : b;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (l.lane == 0) mbar_arrive(&m->full[l.stage]);
        if (++l.stage == R) l.stage = 0, l.phase ^= 1;
    };
    CodeChunk x, y;
    fetch(x);
    fetch(y);
    for (int g = 0; g < total; g += 2) {
        store(g, x);
        fetch(x);
        store(g + 1, y);
        fetch(y);
    }
}

// ------------------------------------------------------------------------------------ issuing products
// One warp, all lanes in step (so that descriptors stay in uniform registers), one of them issuing.
template <int C, bool FP8>
struct Issuer {
    static constexpr int R = Cfg<C>::ring;
    Misc *m;
    const Waiter &wait;
    // descriptors of the ring's first chunk, of the queries and of P; a step adds its offset / 16
    uint64_t ring_k, ring_v, q0, p0;
    uint32_t o_col, s_col;
    int vchunks;
    int s_stage = 0, s_phase = 0, v_stage = 0;
    int s_tile = 0, v_tile = 0;  // tiles issued so far

    __device__ __forceinline__ void scores()
    {
        constexpr uint32_t kScores = umma_idesc(kTile, kCols, false, false);
        const int buf = s_tile & 1;
        wait(&m->s_empty[buf], ((s_tile >> 1) & 1) ^ 1);
        tmem_fence_after();
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            wait(&m->full[s_stage], s_phase);
            if (!FP8) fence_proxy_async_shared();  // the asynchronous copies' arrivals carry no fence of their own
            tmem_fence_after();
            const uint64_t a = ring_k + static_cast<uint32_t>(s_stage * (kChunkBytes / 16));
            const uint64_t b = q0 + static_cast<uint32_t>(c * (2 * kQHalf / 16));
            const uint32_t d = s_col + buf * kCols;
            if (elect_one()) {
                umma_bf16(d, a, b, kScores, c > 0);
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    umma_bf16(d, a + (s >> 2) * (kHalfBytes / 16) + (s & 3) * 2,
                              b + (s >> 2) * (kQHalf / 16) + (s & 3) * 2, kScores, true);
            }
            if (++s_stage == R) s_stage = 0, s_phase ^= 1;
        }
        if (elect_one()) umma_commit(&m->s_full[buf]);
        ++s_tile;
    }

    __device__ __forceinline__ void values(bool first)
    {
        constexpr uint32_t kValues = umma_idesc(128, kCols, true, true);
        const int buf = v_tile & 1;
        wait(&m->p_full[buf], (v_tile >> 1) & 1);
        tmem_fence_after();
        const uint64_t b = p0 + static_cast<uint32_t>((v_tile % Cfg<C>::pbufs) * (kPBytes / 16));
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            if (c < vchunks) {
                const uint64_t a = ring_v + static_cast<uint32_t>(v_stage * (kChunkBytes / 16));
                const uint32_t d = o_col + c * kCols;
                if (elect_one()) {
                    umma_bf16(d, a, b, kValues, !first);
#pragma unroll
                    for (int s = 1; s < kTile / 16; ++s) umma_bf16(d, a + s * 128, b + s * 128, kValues, true);
                }
            }
            if (elect_one()) umma_commit(&m->empty[v_stage]);
            if (++v_stage == R) v_stage = 0;
        }
        if (elect_one()) umma_commit(&m->pv_done[buf]);
        ++v_tile;
    }

    __device__ __forceinline__ void unit(int n, int phase)
    {
        wait(&m->q_full, phase);
        fence_proxy_async_shared();
        scores();
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            if (Cfg<C>::ahead && it + 1 < n) scores();
            if (it + 1 == n && elect_one()) umma_commit(&m->q_empty);
            values(it == 0);
            if (!Cfg<C>::ahead && it + 1 < n) scores();
        }
    }
};

// ------------------------------------------------------------------------------------ softmax
// Sum (or maximum) over the warp's lanes of each of 32 values a lane holds; lane j gets that of value j.
template <bool MAX>
__device__ __forceinline__ float reduce32(float v[32], int lane)
{
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int j = 0; j < s; ++j) {
            const float send = up ? v[j] : v[j + s];
            const float keep = up ? v[j + s] : v[j];
            const float got = __shfl_xor_sync(0xffffffffu, send, s);
            v[j] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    return v[0];
}

template <int C>
__device__ __forceinline__ void softmax_unit(const Kargs &k, const Unit &w, Misc *m, const Waiter &wait,
                                             unsigned char *smem, int &tile, int warp, int lane)
{
    const int wg = warp >> 2, quad = warp & 3, line = quad * 32 + lane;
    const int bar = 1 + wg;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_tm = m->tmem + lanes + wg * 32, s_tm = m->tmem + lanes + C * kCols + wg * 32;
    const int vchunks = (k.a.dv + 127) >> 7;
    const float scale = k.a.scale_log2;
    const float4 *ref4 = reinterpret_cast<const float4 *>(m->ref + wg * 32);
    const int *ends = w.end + wg * 32;
    unsigned char *pbase = smem + Cfg<C>::p_off + line * 128;
    const int lo = w.lo, n = w.n;
    float l[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) l[j] = 0.0f;
    if (quad == 0) m->ref[wg * 32 + lane] = -INFINITY;
    bar_sync(bar, 128);

    for (int it = 0; it < n; ++it, ++tile) {
        const int buf = tile & 1;
        wait(&m->s_full[buf], (tile >> 1) & 1);
        tmem_fence_after();
        uint32_t raw[32];
        tmem_ld32(s_tm + buf * kCols, raw);
        tmem_wait_ld();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->s_empty[buf]);
        const bool valid = (m->valid[tile & (kValidSlots - 1)][quad] >> lane) & 1u;
        const int pos = (lo + it) * kTile + line;
        // a tile some of whose positions are past the end of some, not all, of the CTA's rows
        const bool edges = !k.a.idx && pos - line + kTile > w.min_end && w.min_end < w.max_end;
        bool dirty = false;
        if (edges) {
            // A position that one row attends to and another does not has weight 0 in the other, but
            // 0 * NaN is NaN: a row that is not finite is taken out of the values, and the columns that
            // do attend to it become NaN by their weight.  Such a row makes its score not finite.
            const bool odd = valid && !(fabsf(__uint_as_float(raw[0])) < INFINITY);
            if (bar_any(3, kSoftWarps * 32, odd)) {
                const int stage0 = static_cast<int>((static_cast<int64_t>(tile) * C) % Cfg<C>::ring);
                auto unit16 = [&](int e) {
                    return smem + ((stage0 + (e >> 7)) % Cfg<C>::ring) * kChunkBytes + ((e >> 6) & 1) * kHalfBytes +
                           line * 128 + ((((e >> 3) & 7) ^ (line & 7)) << 4);
                };
                if (odd)
                    for (int e = 0; e < k.a.dv; ++e)
                        dirty |= (reinterpret_cast<const uint16_t *>(unit16(e))[e & 7] & 0x7f80u) == 0x7f80u;
                bar_sync(3, kSoftWarps * 32);
                if (dirty && wg == 0)
                    for (int e = 0; e < k.a.dv; e += 8)
                        *reinterpret_cast<uint4 *>(unit16(e)) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        // x = log2 of the weight before the column's reference is taken off, -inf where masked
        const bool whole = __all_sync(0xffffffffu, valid) && !edges;
        auto masked = [&](float x, int j) { return valid && !(edges && pos >= ends[j]) ? x : -INFINITY; };
        float x[32];
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
            const float4 r = ref4[j4];
            x[4 * j4] = fmaf(__uint_as_float(raw[4 * j4]), scale, -r.x);
            x[4 * j4 + 1] = fmaf(__uint_as_float(raw[4 * j4 + 1]), scale, -r.y);
            x[4 * j4 + 2] = fmaf(__uint_as_float(raw[4 * j4 + 2]), scale, -r.z);
            x[4 * j4 + 3] = fmaf(__uint_as_float(raw[4 * j4 + 3]), scale, -r.w);
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = masked(x[j], j);
        }
        float top = x[0];
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, x[j]);
        // (a column without positions yet has the reference -inf, which any score exceeds)
        if (bar_any(bar, 128, top > kRefSlack)) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = masked(__uint_as_float(raw[j]) * scale, j);
            m->wmax[quad][wg * 32 + lane] = reduce32<true>(x, lane);
            bar_sync(bar, 128);
            if (quad == 0) {
                const int c = wg * 32 + lane;
                const float old = m->ref[c];
                const float now = fmaxf(fmaxf(old, fmaxf(m->wmax[0][c], m->wmax[1][c])), fmaxf(m->wmax[2][c], m->wmax[3][c]));
                m->factor[c] = old == now ? 1.0f : exp2_approx(old - now);
                m->ref[c] = now;
            }
            bar_sync(bar, 128);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float r = m->ref[wg * 32 + j];
                x[j] = masked(fmaf(__uint_as_float(raw[j]), scale, r == -INFINITY ? 0.0f : -r), j);
                l[j] *= m->factor[wg * 32 + j];
            }
            if (it > 0) {
                wait(&m->pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
                tmem_fence_after();
                for (int c = 0; c < vchunks; ++c) {
                    tmem_ld32(o_tm + c * kCols, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        raw[j] = __float_as_uint(__uint_as_float(raw[j]) * m->factor[wg * 32 + j]);
                    tmem_st32(o_tm + c * kCols, raw);
                }
                tmem_wait_st();
            }
        }
        if (dirty) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (pos < ends[j]) x[j] = __int_as_float(0x7fffffff);
        }
        // the buffer of P is free once the product that read it is done
        if (tile >= Cfg<C>::pbufs) {
            const int before = tile - Cfg<C>::pbufs;
            wait(&m->pv_done[before & 1], (before >> 1) & 1);
        }
        unsigned char *prow = pbase + (tile % Cfg<C>::pbufs) * kPBytes;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = u * 8 + i * 2;
                const float p0 = exp2_approx(x[j]), p1 = exp2_approx(x[j + 1]);
                l[j] += p0;
                l[j + 1] += p1;
                out[i] = pack_bf16(p0, p1);
            }
            *reinterpret_cast<uint4 *>(prow + (((wg * 4 + u) ^ (line & 7)) << 4)) =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
        fence_proxy_async_shared();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->p_full[buf]);
    }

    // column sums, in a fixed order
    m->lsum[quad][wg * 32 + lane] = reduce32<false>(l, lane);
    bar_sync(bar, 128);
    const int col = wg * 32 + lane, cols = w.cols();
    const float sum = (m->lsum[0][col] + m->lsum[1][col]) + (m->lsum[2][col] + m->lsum[3][col]);
    const int64_t out_row = (w.row0 + col / w.heads) * k.a.h + w.head0 + col % w.heads;  // of lane's column
    if (quad == 0) {
        m->inv[col] = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (col < cols) {
            if (k.p.parts > 1)
                k.part_ml[out_row * k.p.parts + w.part] = make_float2(m->ref[col], sum);
            else if (k.a.lse)
                k.a.lse[out_row] = sum == 0.0f ? -INFINITY : (m->ref[col] + log2f(sum)) * 0.69314718055994531f;
        }
    }
    bar_sync(bar, 128);
    if (n > 0) {
        wait(&m->pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
        tmem_fence_after();
    }
    if (k.p.parts > 1) {
        // (a part without positions has the sum 0: its accumulators are not read)
        for (int c = 0; n > 0 && c < vchunks; ++c) {
            uint32_t o[32];
            tmem_ld32(o_tm + c * kCols, o);
            tmem_wait_ld();
            const int e = c * 128 + line;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int64_t r = __shfl_sync(0xffffffffu, out_row, j);
                if (wg * 32 + j < cols && e < k.a.dv)
                    k.part_o[(r * k.p.parts + w.part) * k.a.dv + e] = __uint_as_float(o[j]);
            }
        }
        return;
    }
    // the group's 32 columns x 128 elements through its half of a P buffer (free by now), so that whole
    // 16-byte vectors of a column are written
    unsigned char *stage = smem + Cfg<C>::p_off + wg * (kPBytes / 2);
    for (int c = 0; c < vchunks; ++c) {
        uint32_t o[32];
        if (n > 0) {
            tmem_ld32(o_tm + c * kCols, o);
            tmem_wait_ld();
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float v = __uint_as_float(o[j]) * m->inv[wg * 32 + j];
            *reinterpret_cast<__nv_bfloat16 *>(stage + j * 256 + line * 2) = __float2bfloat16_rn(v);
        }
        bar_sync(bar, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = quad * 8 + i * 2 + (lane >> 4), e = c * 128 + (lane & 15) * 8;
            const int64_t r = __shfl_sync(0xffffffffu, out_row, j);
            if (wg * 32 + j < cols && e < k.a.dv)
                __stcs(reinterpret_cast<uint4 *>(k.a.out + r * k.a.dv + e),
                       *reinterpret_cast<const uint4 *>(stage + j * 256 + (lane & 15) * 16));
        }
        bar_sync(bar, 128);
    }
    bar_sync(3, kSoftWarps * 32);  // the next unit's P covers both groups' staging
}

// ------------------------------------------------------------------------------------ the kernel
template <int C, bool FP8>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ Kargs k)
{
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc *m = reinterpret_cast<Misc *>(smem + Cfg<C>::misc_off);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t units = k.p.items * k.p.parts;
    if (t == 0) {
        for (int i = 0; i < Cfg<C>::ring; ++i) {
            mbar_init(&m->full[i], FP8 ? kLoadWarps : kLoadWarps * 32);
            mbar_init(&m->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], kSoftWarps);
            mbar_init(&m->p_full[i], kSoftWarps);
            mbar_init(&m->pv_done[i], 1);
            mbar_init(&m->unit_full[i], 1);
            mbar_init(&m->unit_empty[i], kSoftWarps + 1 + kLoadWarps);
        }
        mbar_init(&m->q_full, kLoadWarps * 32);
        mbar_init(&m->q_empty, 1);
        fence_mbar_init();
        m->abort = 0;
    }
    if (warp == kMmaWarp) tmem_alloc(&m->tmem, 512);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const Waiter wait{&m->abort, k.a.err_flag};
    // unit i of this CTA is in slot i mod 2
    auto take = [&](int i) -> const Unit * {
        wait(&m->unit_full[i & 1], (i >> 1) & 1);
        return &m->unit[i & 1];
    };
    auto give = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->unit_empty[i & 1]);
    };

    if (warp < kSoftWarps) {
        regs_up<kSoftRegs>();
        int tile = 0, i = 0;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++i) {
            softmax_unit<C>(k, *take(i), m, wait, smem, tile, warp, lane);
            give(i);
        }
    } else if (warp < kLoadWarp0) {
        regs_down<kMmaRegs>();
        if (warp == kMmaWarp) {
            Issuer<C, FP8> issue{m, wait};
            issue.ring_k = umma_desc(smem_addr(smem), 16, 1024);
            issue.ring_v = umma_desc(smem_addr(smem), kHalfBytes, 1024);
            issue.q0 = umma_desc(smem_addr(smem + Cfg<C>::q_off), 16, 1024);
            issue.p0 = umma_desc(smem_addr(smem + Cfg<C>::p_off), kHalfBytes, 1024);
            const uint32_t tm = __reduce_max_sync(0xffffffffu, m->tmem);  // (uniform)
            issue.o_col = tm;
            issue.s_col = tm + C * kCols;
            issue.vchunks = (k.a.dv + 127) >> 7;
            int i = 0, loaded = 0;
            for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++i) {
                const int n = __reduce_max_sync(0xffffffffu, take(i)->n);
                if (n > 0) issue.unit(n, loaded++ & 1);
                give(i);
            }
        } else if (warp == kUnitWarp) {
            int i = 0;
            for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++i) {
                wait(&m->unit_empty[i & 1], ((i >> 1) & 1) ^ 1);
                make_unit(k, u, &m->unit[i & 1], lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&m->unit_full[i & 1]);
            }
        }
    } else {
        regs_down<kLoadRegs>();
        Loader l{k, m, nullptr, k.a.t.max_pages * k.a.c.page_size, lane, warp - kLoadWarp0, 0, 1, 0};
        int i = 0, loaded = 0;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++i) {
            l.w = take(i);
            if (l.w->n > 0) {
                wait(&m->q_empty, (loaded++ & 1) ^ 1);
                l.queries<C>(smem + Cfg<C>::q_off);
                if (FP8)
                    load_fp8<C>(l, wait, smem);
                else
                    load_bf16<C>(l, wait, smem);
            }
            give(i);
        }
        cp_async_wait_all();
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(m->tmem, 512);
}

// Joins the parts of each (row, head): out = sum_p 2^(ref_p - max) o_p / sum_p 2^(ref_p - max) sum_p.
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ Kargs k)
{
    const int64_t item = blockIdx.x;
    const int parts = k.p.parts, dv = k.a.dv;
    const float2 *ml = k.part_ml + item * parts;
    float top = -INFINITY;
    for (int p = 0; p < parts; ++p) {
        const float2 v = ml[p];
        if (v.y != 0.0f) top = fmaxf(top, v.x);
    }
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int e = threadIdx.x * 4;
    for (int p = 0; p < parts; ++p) {
        const float2 v = ml[p];
        if (v.y == 0.0f) continue;
        const float f = v.x == top ? 1.0f : exp2_approx(v.x - top);
        sum += f * v.y;
        if (e < dv) {
            const float4 o = *reinterpret_cast<const float4 *>(k.part_o + (item * parts + p) * dv + e);
            acc.x += f * o.x, acc.y += f * o.y, acc.z += f * o.z, acc.w += f * o.w;
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (e < dv)
        *reinterpret_cast<uint2 *>(k.a.out + item * dv + e) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (threadIdx.x == 0 && k.a.lse) k.a.lse[item] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

template <int C, bool FP8>
cudaError_t launch(const Kargs &k, cudaStream_t s)
{
    constexpr size_t smem = Cfg<C>::misc_off + sizeof(Misc);
    static_assert(smem <= 232448, "more than a CTA may use");
    static_assert(smem > 116 * 1024, "one CTA an SM: each takes all of the tensor memory");
    cudaError_t e = cudaFuncSetAttribute(attention_kernel<C, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int64_t units = k.p.items * k.p.parts, sms = device_sm_count();
    attention_kernel<C, FP8><<<static_cast<unsigned>(units < sms ? units : sms), kThreads, smem, s>>>(k);
    return cudaGetLastError();
}

Plan plan_of(int64_t rows, int64_t h, int64_t b, int64_t positions, bool idx_given)
{
    Plan p{};
    const int64_t per = rows / b;
    p.heads_per_tile = static_cast<int>(h < kCols ? h : kCols);
    p.head_blocks = static_cast<int>((h + kCols - 1) / kCols);
    // rows that share a tile share its positions; a row with a list has its own
    const int64_t fit = idx_given ? 1 : kCols / p.heads_per_tile;
    p.rows_per_tile = static_cast<int>(fit < per ? fit : per);
    p.tiles_per_seq = (per + p.rows_per_tile - 1) / p.rows_per_tile;
    p.items = b * p.tiles_per_seq * p.head_blocks;
    // parts: as many as keep the fewest tiles in a row, counting a part's start and end as 1.5 tiles
    const int64_t tiles = (positions + kTile - 1) / kTile;
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 1;
    p.parts = 1;
    double best = 0.0;
    for (int64_t n = 1; n <= kMaxSplit && n <= (tiles > 1 ? tiles : 1); ++n) {
        const int64_t waves = (p.items * n + sms - 1) / sms;
        const double cost = static_cast<double>(waves) * (static_cast<double>((tiles + n - 1) / n) + 1.5) + (n > 1 ? 1.0 : 0.0);
        if (n == 1 || cost < best) {
            best = cost;
            p.parts = static_cast<int>(n);
        }
        if (p.items * n > 2 * sms) break;
    }
    return p;
}

size_t part_bytes(int64_t items, int parts) { return static_cast<size_t>((items * parts * 8 + 255) / 256 * 256); }

}  // namespace

size_t cache_attention_workspace(int64_t rows, int64_t h, int64_t, int64_t dv, int64_t b, int64_t positions,
                                 bool idx_given)
{
    const Plan p = plan_of(rows, h, b, positions, idx_given);
    if (p.parts == 1) return 0;
    return part_bytes(rows * h, p.parts) + static_cast<size_t>(rows * h) * p.parts * dv * 4;
}

cudaError_t launch_cache_attention(const CacheAttnArgs &a, cudaStream_t s)
{
    Kargs k{};
    k.a = a;
    k.p = plan_of(a.rows, a.h, a.rows / a.t.rows_per_seq, a.idx ? a.n : a.t.max_pages * a.c.page_size, a.idx != nullptr);
    if (k.p.parts > 1) {
        k.part_ml = static_cast<float2 *>(a.ws);
        k.part_o = reinterpret_cast<float *>(static_cast<unsigned char *>(a.ws) + part_bytes(a.rows * a.h, k.p.parts));
    }
    const bool fp8 = a.c.scales != nullptr;
    cudaError_t e;
    switch ((a.d + 127) / 128) {
    case 1: e = fp8 ? launch<1, true>(k, s) : launch<1, false>(k, s); break;
    case 2: e = fp8 ? launch<2, true>(k, s) : launch<2, false>(k, s); break;
    case 3: e = fp8 ? launch<3, true>(k, s) : launch<3, false>(k, s); break;
    default: e = fp8 ? launch<4, true>(k, s) : launch<4, false>(k, s); break;
    }
    if (e != cudaSuccess || k.p.parts == 1) return e;
    join_kernel<<<static_cast<unsigned>(a.rows * a.h), 128, 0, s>>>(k);
    return cudaGetLastError();
}

}  // namespace sel
