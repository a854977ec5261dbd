// cache_attention.cu -- attention of new tokens over a paged cache, on the fifth-generation tensor cores.
//
// For the columns n = (row, head) of one CTA and a tile of 128 positions with rows K:
//     S^T = K Q^T            [128 positions x 64 or 128 columns]
//     P^T = exp2(S^T * scale - ref)
//     O^T += K[:, :dv]^T P^T [dv x 64 or 128 columns]
// Positions are the M dimension of the first product and heads its N dimension, so a single token with
// few heads wastes no part of the 128-row instruction, a thread of the softmax holds few positions and
// many columns, and the value is the key tile itself, read with the other dimension contiguous: each cache
// row is staged once and used for both products.
//
// The sum of exponentials needs no maximum, only a reference that keeps exp2 in range.  A column's is set from
// its largest score, with room above; while no weight outgrows it a tile is taken with one vote.  Else
// the columns' maxima are formed across the positions and the sums and accumulators are rescaled.  Scores, sums,
// references and accumulators are fp32; the weights are rounded to bf16 for the second product, whose other
// operand, the value, has no more bits (the sums are of the unrounded weights: the roundings are to
// nearest, 2^-8 of a weight at most).  Sums are kept per thread (its positions) and joined at the end in a fixed order.
//
// A CTA stays on its SM and takes one unit of work (rows x heads x a part of the positions) after the
// other.  Its warps are those of the softmax in groups of 4, one that issues the products, one that looks up
// the next unit, two that stage queries, and those that stage rows, in chunks of 128 elements by 128 positions
// in a ring.  A chunk is released when its part of the second product is done, or after the first where it is
// no part of the value, so the next tile's rows arrive while the rest of the product runs.
//
// Of few rows over long contexts all tiles are shared out evenly among the CTAs, whatever row they are of; what a
// row's parts come to, sums and accumulators, a second kernel joins in a fixed order.
//
// What bounds it.  Of 512 elements one tile fills the ring beside the queries, so a tile's steps follow one
// another: values, the next rows' way in, scores, softmax, 7100 cycles in all (3.4 us at the 2070 MHz of all
// figures here, 108 tiles of the busiest CTA in the 371 us below), of which the products' 64 instructions take
// 3100 at their own rate.  8-bit rows: 10000 cycles a tile (4.8 us, 28 tiles in the 135 us below): each of the two
// sets of warps loads and decodes two chunks one after the other, and the second one's loads start when the
// products have freed its place.  Of 128 .. 192 elements the softmax bounds, against 1800 cycles of products a tile:
// 3700 cycles a tile with the units' starts and ends (103 tiles, 189 us).  And one-off code: what runs once a unit is fetched from far, about 100 cycles for 8 instructions,
// so masks, column maxima and sums are written for few instructions (the last tile's mask took 6300 cycles
// before, the sums 5400).
// Measured (GB300, device time; of the 1891 TFLOP/s and 6772 GB/s that plain products and copies reach):
//   4096 rows x 64 heads over 512 selected rows of 512, bf16   371 us   649 TFLOP/s (34%)
//   4 rows x 64 heads over 204800 positions of 512, bf16       169 us   4940 GB/s (73%)
//   3 x 701 rows x 24 heads, 5000 positions of 192, causal     189 us   689 TFLOP/s (36%)
//   1024 rows x 64 heads over 512 selected 8-bit rows of 512   135 us   507 TFLOP/s (27%)
//   32 rows x 64 heads over <= 16384 positions of 512, 8 bits  119 us   1840 GB/s, 448 TFLOP/s (27%)
//   1 row over 1000 positions of 128                           10.9 us  (in a graph; latency: start, lookups, a tile, join)
// Tried and slower: tiles of 64 positions (45 cycles an instruction of half the work); pairs of CTAs that share
// a row (622 us against 385 then); TMA gathers of 4 rows (75 to 108 cycles for 512 bytes); bf16 rows through
// registers (564 us); the next tile's rows prefetched into L2 (415 us: the copies fill the path already);
// scores and values issued by a warp each (no change); a warp that looks up the rows for the others (448 us).
// (A few per cent either way say little about an idea here: the order of the roles' code alone moves as much.)
#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"
#include "tcgen05.cuh"

namespace sel {
namespace {

constexpr int kMaxCols = 128;              // (row, head) columns of a CTA at most
constexpr int kMaxRing = 5;
constexpr int kValidSlots = 16;            // tiles whose validity bits are kept (more than the ring holds)
constexpr int kNoted = 8;                  // tiles whose validity bits may be under way (the ring holds 5, lookups are 2 ahead)
constexpr int kScan = 32768;               // entries of a list's end that are looked through for its last position
constexpr int kUnits = 4;                  // units known at a time
constexpr int kMaxItems = 512;             // items whose tiles are shared out evenly at most
constexpr int kMaxCtas = 512;              // CTAs that share at most
constexpr int kStart = 1;                  // tiles that an item's start counts for there
// A column's reference is set 2^kHeadroom above its largest weight so far and moves when a weight reaches
// twice the reference.  bf16 has the range of fp32, so the small weights lose nothing by it down to 2^-102 of the
// column's largest (below, they are 0), and that a weight is 2 or more is one bit of its bf16 exponent.
constexpr float kHeadroom = 24.0f;
constexpr float kNoReference = -3.4028235e38f;  // of a column without a score above -inf: any such score outgrows it
constexpr long long kWaitCycles = 4000000000LL;  // about 2 s: no wait of a working kernel takes a thousandth of it
constexpr uint32_t kSuspend = 1000;
constexpr int32_t kTimeout = 5;            // SEL_ETIMEOUT

// C chunks of 128 elements a row, N columns.  Measured tensor rates: 128 x 64 x 16 takes 48.7 cycles
// (66% of the peak: reading the operands from shared memory bounds it), 128 x 128 x 16 takes 64.6 (99%).
// So 128 columns are taken where queries, P and two tiles of rows fit beside one another: rows of up to 192
// elements.
template <int C, int N, bool FP8>
struct Cfg {
    static_assert(N == 64 || N == 128, "");
    static constexpr bool wide = N == 128;
    static constexpr int M = 128;                                   // positions of a tile
    static constexpr int half_bytes = M * 128;                      // a tile's 64 columns: one 128-byte line a position
    static constexpr int chunk_bytes = 2 * half_bytes;
    static constexpr int q_halves = wide && C == 2 ? 3 : 2 * C;     // blocks of 64 elements of a query
    static constexpr int q_half = N * 128;                          // bytes of one
    static constexpr int p_block = M * 128;                         // 64 columns of P^T, a line a position
    static constexpr int p_bytes = N / 64 * p_block;
    // Chunks staged.  Of rows of 129 to 192 elements the first chunk has 3 places and the second, which is half
    // as large and often no part of the value, 2 of its own (`own`): three tiles are under way at a time where
    // a common ring has two.
    static constexpr bool own = wide && C == 2 && !FP8;
    static constexpr int ring = own ? 5 : wide && C == 1 ? 3 : (C == 1 ? 5 : 4);
    static constexpr int ring_bytes = own ? 4 * chunk_bytes : ring * chunk_bytes;
    static constexpr int own0 = 3, own1 = 2;  // places of the first chunk, of the second
    static_assert(!own || own0 + own1 == ring, "");
    static __device__ __forceinline__ int place(int stage) { return stage * chunk_bytes - (own && stage > own0 ? half_bytes : 0); }
    static constexpr int pbufs = C == 1 || (C == 2 && !wide) ? 2 : 1;
    static constexpr bool ahead = ring >= 2 * C;  // the next tile's scores before this one's values
    static constexpr int q_off = ring_bytes;
    static constexpr int p_off = q_off + q_halves * q_half;
    static constexpr int misc_off = p_off + pbufs * p_bytes;
    // Warps: groups of 4 for the softmax, an equal share of the columns each; a group of 4 with the one that
    // issues, the one that looks up what is next and two that stage queries; those that stage rows.
    // 8-bit rows take two sets of the last, which stage every other chunk each, and fewer of the first: the
    // time from a load to the decoded chunk bounds them.
    static constexpr int groups = FP8 && !wide ? 2 : 4;
    static constexpr int cols_per_group = N / groups;
    static constexpr int soft_warps = 4 * groups, mma_warp = soft_warps, unit_warp = soft_warps + 1;
    static constexpr int load_warp0 = soft_warps + 4;
    static constexpr int load_sets = FP8 && !wide ? 2 : 1, set_warps = wide && FP8 ? 4 : 8;
    static constexpr int load_warps = load_sets * set_warps;
    static constexpr int threads = (load_warp0 + load_warps) * 32;
    // Registers a thread after the roles part, of 896 x 72 (768 x 80) at the launch.
    static constexpr int launch_regs = load_warps == 4 ? 80 : 72;
    static constexpr int soft_regs = wide ? (FP8 ? 88 : 96) : FP8 ? 96 : 64;
    static constexpr int mma_regs = wide && !FP8 ? 32 : 40;
    static constexpr int load_regs = wide ? (FP8 ? 88 : 40) : FP8 ? 64 : 96;
    static_assert(ring >= C && ring <= kMaxRing && ring / C + 2 < kNoted && kNoted <= kValidSlots, "");
    static_assert(32 * soft_warps * soft_regs + 128 * mma_regs + 32 * load_warps * load_regs <= threads * launch_regs, "");
};

// What a CTA works on next, made by one warp ahead of the others.
struct Unit {
    int64_t row0, seq;
    int64_t keys;            // positions, or list entries up to the last valid one
    int64_t list_end;        // exclusive end of the listed positions
    int rows, heads;         // of its columns: column = row * heads + head
    int slot;                // where its sums and accumulators go; -1: it is a whole item, its outputs are written
    int lo, n;               // first tile and tiles
    int min_end, max_end;    // of its rows
    alignas(16) int end[kMaxCols];  // exclusive end of each column's row, 0 for unused columns
    alignas(16) int out[kMaxCols];  // row * heads + head of each column
    alignas(16) int64_t q[kMaxCols];  // element offset of each column's query, -1 for unused columns
    __device__ __forceinline__ int cols() const { return rows * heads; }
};

struct Misc {
    uint64_t full[kMaxRing], empty[kMaxRing], s_full[2], s_empty[2], p_full[2], pv_done[2], q_full, q_empty;
    uint64_t noted[kNoted];  // validity bits of a tile: the scores' barriers say nothing of them
    uint64_t unit_full[kUnits], unit_empty[kUnits];
    uint64_t drained;        // every product is done
    uint32_t tmem;
    int abort;
    int units, item0;        // of this CTA: units, and, where tiles are shared out, the first one's item
    int before[kMaxItems + 1];  // tiles of the items before, where tiles are shared out
    alignas(16) float inv[kMaxCols];      // references, then 1 / sum
    alignas(16) float part[4][kMaxCols];  // maxima, then sums, of the four warps of a group
    alignas(16) uint32_t valid[kValidSlots][4];  // bit k of word w: position 32 w + k of the tile has a cache row
    alignas(16) Unit unit[kUnits];
};

struct Plan {
    int cols;            // columns of a CTA: 64 or 128
    int rows_per_tile;   // T
    int heads_per_tile;  // heads of a head block
    int head_blocks;
    int64_t tiles_per_seq;
    int64_t items;       // row tiles x head blocks
    int ctas;
    int split;           // the items' tiles are shared out evenly among the CTAs, and their parts joined
};

struct Kargs {
    CacheAttnArgs a;
    Plan p;
    // Where items are split: of each its first part's slot, and the first and last CTA that have one; a CTA has
    // two slots, its first unit's and its last one's.
    int4 *parts;
    float *part_o;   // [2 ctas][columns][dv]
    float2 *part_ml; // [2 ctas][columns]: reference (log2), sum
    long long wait_cycles;  // after which a wait gives up
};

// Waits that end.  One that has waited for `limit` cycles gives up and says so in `abort`, after which every wait of
// the CTA that is not over by itself gives up too, and in err_flag (SEL_ETIMEOUT).  What follows is this:
//  - a unit's loops have counts of their own and addresses that do not depend on what was waited for, so whoever has
//    a unit ends it, and its results are NaN;
//  - a unit that did not come is not looked at (its fields may be anything): the role leaves.  The softmax's
//    warps, which meet at barriers, leave together, and put NaN where the results of the units left would go;
//  - the unit warp leaves instead of writing over a unit that may be in use;
//  - the tensor memory is freed once the products issued so far are done.
struct Waiter {
    volatile int *abort;
    int32_t *err;
    long long limit;
    // Whether the phase of `parity` has completed; the same for the whole warp.
    __device__ __forceinline__ bool operator()(uint64_t *bar, int parity) const
    {
        const bool over = mbar_try_wait(bar, static_cast<uint32_t>(parity), kSuspend) || slow(bar, parity);
        return __all_sync(0xffffffffu, over);  // (none of the warp's lanes falls behind by a phase)
    }
    __device__ __forceinline__ bool slow(uint64_t *bar, int parity) const
    {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar, static_cast<uint32_t>(parity), kSuspend)) {
            if (*abort) return false;
            if (clock64() - t0 > limit) {
                *abort = 1;
                if (err) atomicCAS(err, 0, kTimeout);
                return false;
            }
        }
        return true;
    }
};

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Entry j of a row's list.
__device__ __forceinline__ int64_t entry(const CacheAttnArgs &a, int64_t row, int64_t j)
{
    const int64_t off = row * a.idx_row_stride + j;
    return a.idx_i64 ? __ldg(static_cast<const int64_t *>(a.idx) + off)
                     : static_cast<int64_t>(__ldg(static_cast<const int32_t *>(a.idx) + off));
}

// What an item is: its rows and heads.
struct Item {
    int64_t row0;
    uint32_t seq;
    int rows, head0, heads;
};
__device__ __forceinline__ Item item_of(const Kargs &k, uint32_t item)  // (no call has 2^31 items)
{
    Item it;
    const uint32_t tile = item / static_cast<uint32_t>(k.p.head_blocks);
    const int hb = static_cast<int>(item - tile * static_cast<uint32_t>(k.p.head_blocks));
    it.seq = tile / static_cast<uint32_t>(k.p.tiles_per_seq);
    const int64_t in_seq = static_cast<int64_t>(tile - it.seq * static_cast<uint32_t>(k.p.tiles_per_seq)) * k.p.rows_per_tile;
    const int64_t left = k.a.t.rows_per_seq - in_seq;
    it.row0 = it.seq * k.a.t.rows_per_seq + in_seq;
    it.rows = static_cast<int>(left < k.p.rows_per_tile ? left : k.p.rows_per_tile);
    it.head0 = hb * k.p.heads_per_tile;
    it.heads = min(k.p.heads_per_tile, k.a.h - it.head0);
    return it;
}

__device__ __forceinline__ int row_end(const Kargs &k, int64_t row)
{
    const int64_t cap = k.a.t.max_pages * k.a.c.page_size;
    const int64_t v = k.a.end ? k.a.end[row] : cap;
    return static_cast<int>(v < 0 ? 0 : (v > cap ? cap : v));
}

// The CTA's share of all tiles, [from, to) in the order of the items; with fewer tiles than CTAs the last have none.
// (The host sees to it that tiles x CTAs stay below 2^31.)
struct Share {
    int from, to, ctas;  // ctas: those that have one
};
__device__ __forceinline__ Share share_of(int all, const Kargs &k)
{
    const int cta = static_cast<int>(blockIdx.x), ctas = min(k.p.ctas, all);
    return cta < ctas ? Share{all * cta / ctas, all * (cta + 1) / ctas, ctas} : Share{all, all, ctas};
}

// What an item counts for there, of which the last row's positions end at `most`.
template <int M>
__device__ __forceinline__ int weight_of(const Kargs &k, int most)
{
    if (k.a.idx && most > 0) most = k.a.n;
    return kStart + most / M + (most % M != 0);
}

// Where the sums and accumulators of the CTA's unit u go, an item's [at, after) of all `all` tiles; -1: nowhere, it is
// the whole item.
__device__ __forceinline__ int slot_of(const Share &s, int u, int at, int after)
{
    return s.from > at || s.to < after ? 2 * static_cast<int>(blockIdx.x) + (u == 0 ? 0 : 1) : -1;
}

// The item's entry for the join, by the CTA that has its start.
__device__ __forceinline__ void note_parts(const Kargs &k, const Share &s, int number, int u, int at, int after, int all)
{
    // (the last CTA whose share starts at or before the item's last tile)
    if (s.from <= at)
        k.parts[number] = make_int4(slot_of(s, u, at, after), static_cast<int>(blockIdx.x), (after * s.ctas - 1) / all, 0);
}

// The item that the CTA's unit u is, or is part of.  (Whole items: the last rows first, in a causal chunk they have
// the most positions.)
__device__ __forceinline__ int item_number(const Kargs &k, const Misc *m, int u)
{
    return k.p.split ? m->item0 + u
                     : static_cast<int>(k.p.items) - 1 - static_cast<int>(blockIdx.x) - u * k.p.ctas;
}

// All threads: this CTA's units.  Where items are split, every CTA counts all items' tiles, an item's start as
// kStart more, and takes an equal share of them.  (Parts of equal size for each row instead took 144 us for 32 rows
// of up to 16384 8-bit positions of 512, whose lengths differ; shares take 119.)
template <int M>
__device__ __forceinline__ void find_units(const Kargs &k, Misc *m, int t, int threads)
{
    const int items = static_cast<int>(k.p.items);
    if (!k.p.split) {
        if (t == 0) m->units = units_of(items, static_cast<int>(blockIdx.x), k.p.ctas);
        return;
    }
    if (items == 1) {  // (counted with the unit: 1.2 us sooner)
        if (t == 0) m->units = 1, m->item0 = 0;
        return;
    }
    for (int i = t; i < items; i += threads) {
        const Item it = item_of(k, static_cast<uint32_t>(i));
        int most = 0;
#pragma unroll 8
        for (int r = 0; r < it.rows; ++r) most = max(most, row_end(k, it.row0 + r));
        m->before[i + 1] = weight_of<M>(k, most);
    }
    if (t == 0) m->before[0] = 0;
    __syncthreads();
    if (t < 32) {
        int sum = 0;
#pragma unroll 1
        for (int i = 0; i < items; i += 32) {
            int v = i + t < items ? m->before[i + t + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (t >= d) v += o;
            }
            v += sum;
            if (i + t < items) m->before[i + t + 1] = v;
            sum = __shfl_sync(0xffffffffu, v, 31);
        }
        __syncwarp();
        const Share s = share_of(sum, k);
        int first = 0, upto = 0;  // items that end before the share, that start before its end
#pragma unroll 1
        for (int i = t; i < items; i += 32) {
            first += m->before[i + 1] <= s.from ? 1 : 0;
            upto += m->before[i] < s.to ? 1 : 0;
        }
        first = __reduce_add_sync(0xffffffffu, first);
        upto = __reduce_add_sync(0xffffffffu, upto);
        const int units = s.from < s.to ? upto - first : 0;
        if (t == 0) {
            m->item0 = first;
            m->units = units;
        }
        // (here, where nothing is waited for: the join reads them whatever becomes of the units)
        for (int u = t; u < units; u += 32) note_parts(k, s, first + u, u, m->before[first + u], m->before[first + u + 1], sum);
    }
}

// One warp: unit u of the CTA.
template <int N, int M>
__device__ __forceinline__ void make_unit(const Kargs &k, const Misc *m, int u, Unit *w, int lane)
{
    const int64_t cap = k.a.t.max_pages * k.a.c.page_size;
    const int number = item_number(k, m, u);
    const Item it = item_of(k, static_cast<uint32_t>(number));
    const int64_t row0 = it.row0;
    const int rows = it.rows, head0 = it.head0, heads = it.heads;
    int least = 0x7fffffff, most = 0;
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
        const int col = i * 32 + lane;
        int e = 0;
        const int row = col / heads;
        const int head = head0 + col - row * heads;
        w->out[col] = static_cast<int>((row0 + row) * k.a.h) + head;
        w->q[col] = col < rows * heads ? (row0 + row) * k.a.q_row_stride + head * k.a.q_head_stride : -1;
        if (col < rows * heads) {
            e = row_end(k, row0 + row);
            least = min(least, e);
            most = max(most, e);
        }
        w->end[col] = e;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    int64_t keys = most;
    if (k.a.idx) {  // one row: its list up to the last entry that counts
        // (from the back: the last entries of most lists count.  kScan entries at most: the other roles wait for
        // the unit meanwhile, and empty tiles before that are no fault.)
        int last = 0;
        const int stop = max(k.a.n - kScan, 0);
        auto counts = [&](int64_t p) {
            if (p >= cap && k.a.err_flag) atomicCAS(k.a.err_flag, 0, kCacheInval);
            return p >= 0 && p < most;
        };
#pragma unroll 1
        for (int hi = k.a.n; hi > stop && !__any_sync(0xffffffffu, last > 0); hi -= 128) {
            int64_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = hi - 128 + i * 32 + lane;
                p[i] = j >= 0 ? entry(k.a, row0, j) : -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (counts(p[i])) last = hi - 128 + i * 32 + lane + 1;
        }
        keys = __reduce_max_sync(0xffffffffu, last);
        if (keys == 0) keys = stop;
    }
    if (lane == 0) {
        const int64_t tiles = (keys + M - 1) / M;
        w->row0 = row0;
        w->seq = it.seq;
        w->keys = keys;
        w->list_end = most;
        w->rows = rows;
        w->heads = heads;
        int lo = 0, hi = static_cast<int>(tiles), slot = -1;
        if (k.p.split) {
            const bool one = k.p.items == 1;
            const int at = one ? 0 : m->before[number], after = one ? weight_of<M>(k, most) : m->before[number + 1];
            const int all = one ? after : m->before[k.p.items];
            const Share s = share_of(all, k);
            lo = max(s.from - at - kStart, 0);
            hi = min(hi, max(min(s.to, after) - at - kStart, 0));
            slot = slot_of(s, u, at, after);
            if (one) note_parts(k, s, number, u, at, after, all);
        }
        w->slot = slot;
        w->lo = lo;
        w->n = max(0, hi - lo);
        w->min_end = least;
        w->max_end = most;
    }
}

// ------------------------------------------------------------------------------------ staging rows
// Loads under a predicate, without a branch; 0 (or `other`) where it is false.
__device__ __forceinline__ uint4 load16_if(const void *p, bool yes)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(yes ? 1 : 0));
    return v;
}
__device__ __forceinline__ float load4_if(const float *p, bool yes, float other)
{
    float v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, %3;\n\t@p ld.global.nc.f32 %0, [%1];\n\t}"
                 : "=&f"(v)
                 : "l"(p), "r"(yes ? 1 : 0), "f"(other));
    return v;
}

// 8-bit codes to bf16.  With a scale that is a power of two below 2^8 and no NaN among the codes
// (decodes_fast), a code's exponent and mantissa bits, put where bf16 has them, are its value times 2^-120
// (subnormal codes give subnormal numbers), and one bf16 product makes that value * scale, rounding only
// where the result is subnormal.  Else by way of fp32.
__device__ __forceinline__ bool decodes_fast(uint4 codes, float scale)
{
    const uint32_t s = __float_as_uint(scale);
    const uint32_t nan = ((codes.x & 0x7f7f7f7fu) + 0x01010101u) | ((codes.y & 0x7f7f7f7fu) + 0x01010101u) |
                         ((codes.z & 0x7f7f7f7fu) + 0x01010101u) | ((codes.w & 0x7f7f7f7fu) + 0x01010101u);
    return ((s & 0x007fffffu) | (nan & 0x80808080u)) == 0 && s - 0x00800000u < (134u << 23);
}

// Codes of a word: two times two bf16.
__device__ __forceinline__ uint2 decode4_fast(uint32_t codes, uint32_t by2)
{
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // bytes to sign-extended halves, shifted to the places of bf16's exponent and mantissa
        uint32_t y;  // (selector digits from 8 repeat the byte's sign; __byte_perm drops that bit)
        asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(codes), "r"(i ? 0xb3a2 : 0x9180));
        y = (y << 4) & 0x87f087f0u;
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&by2));
        out[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ uint2 decode4_exact(uint32_t codes, float scale)
{
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((codes >> (16 * i)) & 0xffffu), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        out[i] = pack_bf16(v.x * scale, v.y * scale);
    }
    return make_uint2(out[0], out[1]);
}

// A walk over the places of the ring, chunk by chunk.
template <typename F>
struct Walk {
    int s0 = 0, p0 = 0, s1 = F::own0, p1 = 0;  // stage and phase; of the second chunk, where it has its own
    __device__ __forceinline__ int stage(int c) const { return F::own && c ? s1 : s0; }
    __device__ __forceinline__ int phase(int c) const { return F::own && c ? p1 : p0; }
    __device__ __forceinline__ void next(int c)
    {
        if (F::own && c) {
            if (++s1 == F::ring) s1 = F::own0, p1 ^= 1;
        } else {
            if (++s0 == (F::own ? F::own0 : F::ring)) s0 = 0, p0 ^= 1;
        }
    }
};

template <int C, int N, bool FP8>
struct Loader {
    using F = Cfg<C, N, FP8>;
    // Warp lw stages positions lw * kPos .. of each tile: lane mod kPos looks one up, and the lanes of a
    // line (16 of 16 bytes of bf16, 8 of 16 codes) keep the rows they copy in registers for the tile.
    static constexpr int kPos = F::M / F::set_warps;  // 16 or 32
    static constexpr int kLanes = FP8 ? 8 : 16;        // lanes of a line
    static constexpr int kVecs = kPos * kLanes / 32;   // lines a lane takes part in
    const Kargs &k;
    Misc *m;
    const Waiter &wait;
    unsigned char *smem;
    int lane, lw;
    const Unit *w = nullptr;
    Walk<F> at_ring;           // (bf16 rows)
    int stage = 0, phase = 1;  // (8-bit rows) a fresh barrier's phase of parity 1 counts as completed
    int tile = 0;              // tiles staged in units before

    struct Rows {
        int64_t row, scale;  // element offsets of the lane's position; row -1: none
    };
    struct Place {
        int page, in_page;  // in_page kNone: no position
    };
    static constexpr int kNone = -1;

    // The lane's row of a tile in three steps, taken a tile apart so that nothing waits for their loads:
    // the position (of tile i of the unit; -1: none), its page, its row.
    __device__ __forceinline__ int64_t position(int i) const
    {
        const int64_t j = static_cast<int64_t>(w->lo + i) * F::M + lw * kPos + (lane & (kPos - 1));
        if (i >= w->n || j >= w->keys) return -1;
        return k.a.idx ? entry(k.a, w->row0, j) : j;
    }
    __device__ __forceinline__ Place page_of(int64_t pos) const
    {
        if (pos < 0) return Place{0, kNone};
        if (pos >= w->list_end) {
            if (k.a.err_flag && pos >= k.a.t.max_pages * k.a.c.page_size) atomicCAS(k.a.err_flag, 0, kCacheInval);
            return Place{0, kNone};
        }
        // (positions are below 2^31, and so is the size of a page where there is a page table)
        const uint32_t p = static_cast<uint32_t>(pos), ps = static_cast<uint32_t>(k.a.c.page_size), col = p / ps;
        return Place{__ldg(k.a.t.table + w->seq * k.a.t.stride + col), static_cast<int>(p - col * ps)};
    }
    __device__ __forceinline__ Rows row_of(Place at) const
    {
        if (at.in_page == kNone) return Rows{-1, 0};
        if (at.page < 0 || at.page >= k.a.c.pages) {
            if (k.a.err_flag) atomicCAS(k.a.err_flag, 0, kCacheInval);
            return Rows{-1, 0};
        }
        return Rows{at.page * k.a.c.page_stride + at.in_page * k.a.c.row_stride,
                    at.page * k.a.c.scale_page_stride + at.in_page * k.a.c.scale_row_stride};
    }

    // This warp's validity bits of tile i of the unit.  (They have a barrier of their own: of the staged chunks only
    // the copies are waited for, which orders no ordinary store before them.)
    __device__ __forceinline__ void note(int i, const Rows &r) const
    {
        const uint32_t bits = __ballot_sync(0xffffffffu, r.row >= 0);
        uint32_t *to = m->valid[(tile + i) & (kValidSlots - 1)];
        if (lane == 0) {
            if (kPos == 32)
                to[lw] = bits;
            else
                reinterpret_cast<uint16_t *>(to)[lw] = static_cast<uint16_t>(bits);
            mbar_arrive(&m->noted[(tile + i) & (kNoted - 1)]);
        }
    }

    // ---- bf16 rows: asynchronous copies, whose completion arrives at the chunk's barrier by itself.  (Waiting
    // for them here instead keeps the warp from filling a chunk that has come free meanwhile.)
    __device__ __forceinline__ void rows_bf16()
    {
        const uint16_t *data = static_cast<const uint16_t *>(k.a.c.data);
        const int vec = lane & 15, d = k.a.d, n = w->n;
        const int line0 = lw * kPos + (lane >> 4);
        const uint32_t to = smem_addr(smem) + (vec >> 3) * F::half_bytes + line0 * 128;
        const int halves = (d + 63) >> 6;
        int64_t pos = position(1);
        Place at = page_of(position(0));
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const Rows cur = row_of(at);
            note(it, cur);
            at = page_of(pos);
            pos = position(it + 2);
            int64_t row[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) row[i] = __shfl_sync(0xffffffffu, cur.row, 2 * i + (lane >> 4));
#pragma unroll 1
            for (int c = 0; c < C; ++c) {
                const int stage = at_ring.stage(c);
                wait(&m->empty[stage], at_ring.phase(c) ^ 1);
                const uint32_t base = to + F::place(stage);
                const int e = c * 128 + vec * 8;
                const bool used = c * 2 + (vec >> 3) < halves;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const bool ok = e < d && row[i] >= 0;
                    if (used)
                        cp_async16(base + i * 256 + (((vec & 7) ^ ((line0 + 2 * i) & 7)) << 4), data + (ok ? row[i] + e : 0),
                                   ok ? 16u : 0u);
                }
                cp_async_arrive(&m->full[stage]);
                at_ring.next(c);
            }
        }
    }

    // ---- 8-bit rows: loaded to registers a group ahead, decoded to bf16 on the way to shared memory.  (Two
    // groups ahead were measured slower, 188 against 157 us for 1024 rows over 512 selected positions of 512;
    // a second set of warps, with chunks of its own, hides the loads instead.)  A lane takes codes 16 v .. of a
    // line's 128 (v = lane mod 8), two units of 16 bytes of bf16; lanes 4 .. 7 of a line, whose units are in its
    // other half, store the second first: without bank conflicts.  A tile's scales are loaded by a line a lane,
    // and passed on.
    static constexpr int kLoads = kVecs < 4 ? kVecs : 4;           // lines of a group
    static constexpr int kGroups = (kVecs + kLoads - 1) / kLoads;  // groups of a chunk
    static constexpr int kScales = kPos == 32 ? C : 1;  // scales of a lane: its line's, or one of its line's chunks
    int chunks = 0;  // staged in units before, by all sets

    __device__ __forceinline__ void rows_codes(int set)
    {
        constexpr int S = F::load_sets, kNext = C < S ? S : 1;  // chunks, tiles from one of the warp's to its next
        const uint8_t *data = static_cast<const uint8_t *>(k.a.c.data);
        const float *scales = k.a.c.scales;
        const int vec = lane & 7, d = k.a.d;
        const int total = w->n * C;
        int g = S == 1 || (chunks & 1) == set ? 0 : 1;  // the warp's next chunk of the unit
        int fc = g % C, ft = g / C, fg = 0;             // of the next group to fetch: chunk of the tile, tile, group
        bool fresh = true;                              // rows of tile ft not looked up yet
        int64_t pos = position(ft + kNext);
        Place at = page_of(position(ft));
        int64_t mine = -1;  // row of the lane's line; -1: none
        float sc[kScales];
        uint4 x[kLoads];
        auto fetch = [&]() {
            if (ft >= w->n) return;
            if (fresh) {
                const Rows cur = row_of(at);
                if (fc == 0) note(ft, cur);
                at = page_of(pos);
                pos = position(ft + 2 * kNext);
                if (kPos == 32) {
#pragma unroll
                    for (int i = 0; i < kScales; ++i) sc[i] = load4_if(scales + cur.scale + i, cur.row >= 0 && i * 128 < d, 1.0f);
                } else {  // (with 16 lines a warp, its chunks of the tile are fc and fc + 2)
                    const int c = fc + 2 * (lane >> 4);
                    sc[0] = load4_if(scales + cur.scale + c, cur.row >= 0 && c * 128 < d, 1.0f);
                }
                mine = cur.row;
                fresh = false;
            }
            const bool in = fc * 128 + vec * 16 < d;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int64_t row = __shfl_sync(0xffffffffu, mine, (fg * kLoads + i) * 4 + (lane >> 3));
                x[i] = load16_if(data + row + fc * 128 + vec * 16, row >= 0 && in);
            }
            if (++fg < kGroups) return;
            fg = 0;
            fc += S;
            if (fc >= C) {
                ft += fc / C;
                fc %= C;
                fresh = true;
            }
        };
        static_assert(!FP8 || kGroups <= 2, "");
        const int line0 = lw * kPos + (lane >> 3), swap = vec >> 2;
        unsigned char *to = smem + (vec >> 2) * F::half_bytes + line0 * 128;
        int c = g % C;  // chunk of the tile
        fetch();
#pragma unroll 1
        for (; g < total; g += S) {
            wait(&m->empty[stage], phase);
#pragma unroll 1
            for (int sg = 0; sg < kGroups; ++sg) {
                unsigned char *base = to + stage * F::chunk_bytes + sg * (kLoads * 4 * 128);
                float scale[kLoads];
                bool fast = true;
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int line = (sg * kLoads + i) * 4 + (lane >> 3);
                    scale[i] = kPos == 32 ? __shfl_sync(0xffffffffu, c == 0 ? sc[0] : sc[kScales - 1], line)
                                          : __shfl_sync(0xffffffffu, sc[0], line + 16 * (c >> 1));
                    fast &= decodes_fast(x[i], scale[i]);
                }
                auto store = [&](int i, uint2 a0, uint2 a1, uint2 b0, uint2 b1) {
                    unsigned char *line = base + i * 512;
                    const int at7 = (line0 + 4 * i) & 7, u = (2 * vec & 7) + swap;
                    *reinterpret_cast<uint4 *>(line + ((u ^ at7) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
                    *reinterpret_cast<uint4 *>(line + (((u ^ 1) ^ at7) << 4)) = make_uint4(b0.x, b0.y, b1.x, b1.y);
                };
                if (fast) {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const uint32_t f = (__float_as_uint(scale[i]) >> 16) + (120u << 7), by2 = f | (f << 16);
                        store(i, decode4_fast(swap ? x[i].z : x[i].x, by2), decode4_fast(swap ? x[i].w : x[i].y, by2),
                              decode4_fast(swap ? x[i].x : x[i].z, by2), decode4_fast(swap ? x[i].y : x[i].w, by2));
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < kLoads; ++i) {
                        uint4 v = x[0];
                        float f = scale[0];
#pragma unroll
                        for (int j = 1; j < kLoads; ++j) {
                            if (i == j) v = x[j], f = scale[j];
                        }
                        if (swap) v = make_uint4(v.z, v.w, v.x, v.y);
                        store(i, decode4_exact(v.x, f), decode4_exact(v.y, f), decode4_exact(v.z, f), decode4_exact(v.w, f));
                    }
                }
                if (sg + 1 < kGroups) fetch();
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->full[stage]);
            stage += S;
            if (stage >= F::ring) stage -= F::ring, phase ^= 1;
            c = (c + S) % C;
            fetch();
        }
        chunks += total;
    }
};

// The queries of a unit by two warps; unused columns and elements past d are zeros.
template <int C, int N, bool FP8>
__device__ __forceinline__ void load_queries(const Kargs &k, const Unit *w, Misc *m, unsigned char *smem, int warp, int lane)
{
    using F = Cfg<C, N, FP8>;
    const int vec = lane & 15;
    const uint32_t to = smem_addr(smem + F::q_off) + (vec >> 3) * F::q_half;
#pragma unroll 4
    for (int i = 0; i < N / 4; ++i) {
        const int col = (i * 2 + warp) * 2 + (lane >> 4);
        const int64_t at = w->q[col];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = c * 128 + vec * 8;
            const bool ok = at >= 0 && e < k.a.d;
            if (c * 2 + (vec >> 3) < F::q_halves)
                cp_async16(to + c * 2 * F::q_half + col * 128 + (((vec & 7) ^ (col & 7)) << 4),
                           k.a.q + (ok ? at + e : 0), ok ? 16u : 0u);
        }
    }
    cp_async_wait_all();
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&m->q_full);
}

// ------------------------------------------------------------------------------------ issuing products
// One warp, all lanes in step, one of them issuing.
template <int C, int N, bool FP8>
struct Issuer {
    using F = Cfg<C, N, FP8>;
    Misc *m;
    const Waiter &wait;
    // descriptors of the ring's first chunk, of the queries and of P; a step adds its offset / 16
    uint64_t ring_k, ring_v, q0, p0;
    uint32_t o_col, s_col;
    int halves, vchunks;  // blocks of 64 elements of a row, of 128 of a value
    Walk<F> s_ring, v_ring;
    int s_tile = 0, v_tile = 0;  // tiles issued so far

    // A tile's scores.
    __device__ __forceinline__ void scores()
    {
        constexpr uint32_t kScores = umma_idesc(F::M, N, false, false);
        const int buf = s_tile & 1;
        const uint32_t d = s_col + buf * N;
        wait(&m->s_empty[buf], ((s_tile >> 1) & 1) ^ 1);
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            const int stage = s_ring.stage(c);
            wait(&m->full[stage], s_ring.phase(c));
            if (!FP8) fence_proxy_async_shared();  // (asynchronous copies arrive without a fence of their own)
            tmem_fence_after();
            const uint64_t a = ring_k + static_cast<uint32_t>(F::place(stage) / 16);
            const uint64_t b = q0 + static_cast<uint32_t>(c * (2 * F::q_half / 16));
            if (elect_one()) {
                umma_bf16(d, a, b, kScores, c > 0);
#pragma unroll
                for (int s = 1; s < 4; ++s) umma_bf16(d, a + s * 2, b + s * 2, kScores, true);
                if (2 * c + 1 < halves) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_bf16(d, a + F::half_bytes / 16 + s * 2, b + F::q_half / 16 + s * 2, kScores, true);
                }
                if (c >= vchunks) umma_commit(&m->empty[stage]);  // (no part of the value: free by then)
            }
            __syncwarp();
            s_ring.next(c);
        }
        if (elect_one()) umma_commit(&m->s_full[buf]);
        ++s_tile;
    }

    __device__ __forceinline__ void values(bool first)
    {
        constexpr uint32_t kValues = umma_idesc(128, N, true, true);
        const int buf = v_tile & 1;
        wait(&m->p_full[buf], (v_tile >> 1) & 1);
        tmem_fence_after();
        const uint64_t b = p0 + static_cast<uint32_t>((v_tile % F::pbufs) * (F::p_bytes / 16));
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            const int stage = v_ring.stage(c);
            const uint64_t a = ring_v + static_cast<uint32_t>(F::place(stage) / 16);
            const uint32_t d = o_col + c * N;
            if (elect_one()) {
                if (c < vchunks) {
                    umma_bf16(d, a, b, kValues, !first);
#pragma unroll
                    for (int s = 1; s < F::M / 16; ++s) umma_bf16(d, a + s * 128, b + s * 128, kValues, true);
                    umma_commit(&m->empty[stage]);
                }
                if (c + 1 == C) umma_commit(&m->pv_done[buf]);
            }
            __syncwarp();
            v_ring.next(c);
        }
        ++v_tile;
    }

    __device__ __forceinline__ void unit(int n, int phase)
    {
        wait(&m->q_full, phase);
        scores();
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            if (F::ahead && it + 1 < n) scores();
            if (it + 1 == n && elect_one()) umma_commit(&m->q_empty);
            values(it == 0);
            if (!F::ahead && it + 1 < n) scores();
        }
    }
};

// ------------------------------------------------------------------------------------ softmax
// Thread t of warp `quad` of a group holds, of a tile's scores, H blocks of 16 positions by the group's
// columns in the layout of tmem_ld: 2 H positions by 2 G columns.
template <int C, int N, bool FP8>
struct Softmax {
    using F = Cfg<C, N, FP8>;
    static constexpr int W = F::cols_per_group, G = W / 8, H = F::M / 64;
    static constexpr int X = 4 * G;  // values of a block of 16 positions
    const Kargs &k;
    Misc *m;
    const Waiter &wait;
    unsigned char *smem;
    int group, quad, lane;
    uint32_t o_tm, s_tm;  // the warp's lanes and the group's columns of the accumulators and scores
    int tile = 0;         // tiles done so far
    float2 neg[G], sum[G];  // of the thread's pairs of columns: minus the reference, sum over its positions

    __device__ __forceinline__ int line(int h, int r) const { return quad * (16 * H) + h * 16 + r * 8 + (lane >> 2); }
    __device__ __forceinline__ int col(int i) const { return group * W + (i >> 1) * 8 + (lane & 3) * 2 + (i & 1); }

    __device__ __forceinline__ void load_scores(float x[H][X], int buf) const
    {
#pragma unroll
        for (int h = 0; h < H; ++h) tmem_ld<G>(s_tm + buf * N + (static_cast<uint32_t>(h * 16) << 16), x[h]);
        tmem_wait_ld();
    }

    // What the thread's positions and columns of a tile are masked by.
    struct Mask {
        bool edges;        // some positions are past the end of some, not all, of the CTA's rows
        uint32_t valid;    // bit 2 h + r: the position has a cache row
        int pos0;          // position of line 0
        const int *ends;
    };
    // Scores that a mask leaves out become the infinity whose weight is 0; those of a cache row that is taken
    // out (`dirty`) and not masked become NaN.
    __device__ __forceinline__ void mask_all(float x[H][X], const Mask &a, uint32_t dirty) const
    {
        const float none = k.a.scale_log2 > 0.0f ? -INFINITY : INFINITY;
        if (dirty) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int i = 0; i < X; ++i)
                    if ((dirty >> (2 * h + ((i >> 1) & 1))) & 1u) x[h][i] = quiet_nan();
        }
        // a position against the ends: its offset from the thread's first, or past every end without a row
        int at[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) at[h][r] = (a.valid >> (2 * h + r)) & 1u ? h * 16 + r * 8 : 0x7fffffff;
        const int first = a.pos0 + line(0, 0);
#pragma unroll
        for (int c = 0; c < 2 * G; ++c) {
            const int end = a.edges ? a.ends[col(c)] - first : 0x7fffffff;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float &v = x[h][(c >> 1) * 4 + r * 2 + (c & 1)];
                    v = at[h][r] >= end ? none : v;
                }
        }
    }

    // The thread's 2 G columns reduced over the 8 lanes that share them: the lane is left with one column, its
    // column own().  (Fewer instructions than a butterfly a column; what runs once a unit waits for them.)
    __device__ __forceinline__ int own() const
    {
        return G == 4 ? ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1)
                      : ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
    }
    template <typename Op>
    __device__ __forceinline__ float over_lanes(float v[2 * G], Op op) const
    {
        static_assert(G == 2 || G == 4, "");
        int n = 2 * G;
#pragma unroll
        for (int s = 16; s >= 4; s >>= 1) {
            if (n > 1) {
                n /= 2;
                const bool up = (lane & s) != 0;
#pragma unroll
                for (int i = 0; i < G; ++i)
                    if (i < n) v[i] = op(up ? v[i + n] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], s));
            } else {
                v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
            }
        }
        return v[0];
    }
    // Of the thread's columns: its own one's value, and each column's from the lane that owns it.
    __device__ __forceinline__ float pick(const float2 v[G]) const
    {
        const int c = own();
        float out = v[0].x;
#pragma unroll
        for (int i = 1; i < 2 * G; ++i) out = c == i ? ((i & 1) ? v[i >> 1].y : v[i >> 1].x) : out;
        return out;
    }
    __device__ __forceinline__ float from_own(float v, int c) const
    {
        return __shfl_sync(0xffffffffu, v, (c << (G == 4 ? 2 : 3)) | (lane & 3));
    }

    // Weights outgrow their columns' references: new references, sums and accumulators brought to them.  (The
    // unit's `first` tile sets the references, there is nothing to bring along.)
    __device__ __forceinline__ void move_references(const float x[H][X], bool first)
    {
        float top[2 * G];
#pragma unroll
        for (int c = 0; c < 2 * G; ++c) {
            top[c] = -INFINITY;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    top[c] = fmaxf(top[c], x[h][(c >> 1) * 4 + r * 2 + (c & 1)] * k.a.scale_log2);
        }
        const int at = col(own());
        m->part[quad][at] = over_lanes(top, [](float a, float b) { return fmaxf(a, b); });
        bar_sync(1 + group, 128);
        const float most = fmaxf(fmaxf(m->part[0][at], m->part[1][at]), fmaxf(m->part[2][at], m->part[3][at]));
        const float was = -pick(neg);
        // (a column without a score above -inf so far, for whatever reason, may still get one: it stays without)
        const float now = most == -INFINITY ? was : fmaxf(was, most + kHeadroom);
#pragma unroll
        for (int g = 0; g < G; ++g) neg[g] = make_float2(-from_own(now, 2 * g), -from_own(now, 2 * g + 1));
        if (first) return;
        const float by = was == now ? 1.0f : exp2_approx(was - now);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            sum[g].x *= from_own(by, 2 * g);
            sum[g].y *= from_own(by, 2 * g + 1);
        }
        wait(&m->pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
        tmem_fence_after();
        const int vchunks = (k.a.dv + 127) >> 7;
#pragma unroll 1
        for (int c = 0; c < 2 * vchunks; ++c) {
            const uint32_t at = o_tm + (c >> 1) * N + (static_cast<uint32_t>((c & 1) * 16) << 16);
            float o[X];
            tmem_ld<G>(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < X; ++i) o[i] *= from_own(by, 2 * (i >> 2) + (i & 1));
            tmem_st<G>(at, o);
        }
        tmem_wait_st();
    }

    // A tile's weights 2^(score * scale - reference), two positions by G pairs of columns a block, as bf16
    // pairs; added to `to`.  Returns whether one is 2 or more (or NaN).
    __device__ __forceinline__ bool weights(const float x[H][X], uint32_t out[H][2 * G], float2 to[G]) const
    {
        const float2 scale = make_float2(k.a.scale_log2, k.a.scale_log2);
        uint32_t any = 0;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 y = fma2(make_float2(x[h][4 * g + 2 * r], x[h][4 * g + 2 * r + 1]), scale, neg[g]);
                    const float2 p = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                    to[g] = add2(to[g], p);
                    out[h][2 * g + r] = pack_bf16(p.x, p.y);
                    any |= out[h][2 * g + r];
                }
        return (any & 0x40004000u) != 0;
    }

    // A position that one row attends to and another does not has weight 0 in the other, but 0 * NaN is
    // NaN: a cache row that is not finite is taken out of the values here (its bit 2 h + r is returned), and
    // the columns that do attend to it become NaN by their weight.  Such a row makes its scores not finite.
    __device__ __forceinline__ uint32_t take_out(const float x[H][X], const Mask &mask) const
    {
        uint32_t dirty = 0;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (((mask.valid >> (2 * h + r)) & 1u) && !(fabsf(x[h][2 * r]) < INFINITY)) dirty |= 1u << (2 * h + r);
        if (!bar_any(5, F::soft_warps * 32, dirty != 0)) return 0;
        // chunk c of the tile: its place in the ring, and how often that was filled before
        auto stage_of = [&](int c) {
            if (!F::own) return static_cast<int>((static_cast<int64_t>(tile) * C + c) % F::ring);
            return c ? F::own0 + tile % F::own1 : tile % F::own0;
        };
        auto fills_of = [&](int c) {
            if (!F::own) return static_cast<int>((static_cast<int64_t>(tile) * C + c) / F::ring);
            return c ? tile / F::own1 : tile / F::own0;
        };
        // (the chunks are read here: the scores' barrier speaks for the products alone)
#pragma unroll 1
        for (int c = 0; c * 128 < k.a.dv; ++c) wait(&m->full[stage_of(c)], fills_of(c) & 1);
        auto unit16 = [&](int at, int e) {
            const int stage = stage_of(e >> 7);
            return smem + F::place(stage) + ((e >> 6) & 1) * F::half_bytes + at * 128 +
                   ((((e >> 3) & 7) ^ (at & 7)) << 4);
        };
#pragma unroll 1
        for (int b = 0; b < 2 * H; ++b) {
            if (!((dirty >> b) & 1u)) continue;
            bool bad = false;
#pragma unroll 1
            for (int e = 0; e < k.a.dv; ++e)
                bad |= (reinterpret_cast<const uint16_t *>(unit16(line(b >> 1, b & 1), e))[e & 7] & 0x7f80u) == 0x7f80u;
            if (!bad) dirty &= ~(1u << b);
        }
        bar_sync(5, F::soft_warps * 32);
#pragma unroll 1
        for (int b = 0; b < 2 * H; ++b)
            if (((dirty >> b) & 1u) && group == 0 && (lane & 3) == 0)
#pragma unroll 1
                for (int e = 0; e < k.a.dv; e += 8)
                    *reinterpret_cast<uint4 *>(unit16(line(b >> 1, b & 1), e)) = make_uint4(0u, 0u, 0u, 0u);
        return dirty;
    }

    __device__ __forceinline__ void tiles(const Unit &w)
    {
        const int n = w.n;
        const uint32_t vshift = line(0, 0) & 31;  // the thread's first position within its word of validity bits
#pragma unroll 1
        for (int it = 0; it < n; ++it, ++tile) {
            const int buf = tile & 1;
            Mask mask;
            mask.pos0 = (w.lo + it) * F::M;
            mask.ends = w.end;
            mask.edges = !k.a.idx && mask.pos0 + F::M > w.min_end && w.min_end < w.max_end;
            wait(&m->noted[tile & (kNoted - 1)], (tile / kNoted) & 1);
            wait(&m->s_full[buf], (tile >> 1) & 1);
            tmem_fence_after();
            const uint4 words = *reinterpret_cast<const uint4 *>(m->valid[tile & (kValidSlots - 1)]);
            float x[H][X];
            load_scores(x, buf);
            const uint32_t word = quad < 2 ? (quad == 0 ? words.x : words.y) : (quad == 2 ? words.z : words.w);
            mask.valid = 0;
#pragma unroll
            for (int b = 0; b < 2 * H; ++b) mask.valid |= ((word >> (vshift + 8 * b)) & 1u) << b;
            const bool whole = word == 0xffffffffu && !mask.edges;
            uint32_t dirty = 0;
            if (!whole) {
                if (mask.edges) dirty = take_out(x, mask);
                mask_all(x, mask, dirty);
            }
            // the first tile sets the references, a later one moves them when a weight outgrows its own
            if (it == 0) move_references(x, true);
            uint32_t out[H][2 * G];
            float2 to[G];
#pragma unroll
            for (int g = 0; g < G; ++g) to[g] = sum[g];
            const bool over = weights(x, out, to);
            if (it > 0 && bar_any(1 + group, 128, over)) {
                load_scores(x, buf);  // (not kept: registers)
                if (!whole) mask_all(x, mask, dirty);
                move_references(x, false);
#pragma unroll
                for (int g = 0; g < G; ++g) to[g] = sum[g];
                weights(x, out, to);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) sum[g] = to[g];
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->s_empty[buf]);
            // the buffer of P is free once the product that read it is done
            if (tile >= F::pbufs) {
                const int before = tile - F::pbufs;
                wait(&m->pv_done[before & 1], (before >> 1) & 1);
            }
            // P^T, four 8 x 8 blocks an instruction: lane i gives the address of line i mod 8 of block i / 8
            const uint32_t p = smem_addr(smem + F::p_off + (tile % F::pbufs) * F::p_bytes + (group * W / 64) * F::p_block);
            const int unit0 = (group * W % 64) / 8;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int g = 0; g < G; g += 2) {
                    const int at = quad * (16 * H) + h * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
                    stmatrix4(p + at * 128 + (((unit0 + g + (lane >> 4)) ^ (at & 7)) << 4), out[h] + 2 * g);
                }
            fence_proxy_async_shared();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->p_full[buf]);
        }
    }

    __device__ __forceinline__ void unit(const Unit &w)
    {
        const int bar = 1 + group, cols = w.cols(), n = w.n;
        auto out_row = [&](int c) { return static_cast<int64_t>(w.out[c]); };
#pragma unroll
        for (int g = 0; g < G; ++g) {
            neg[g] = make_float2(-kNoReference, -kNoReference);
            sum[g] = make_float2(0.0f, 0.0f);
        }
        tiles(w);
        // column sums, in a fixed order
        bar_sync(bar, 128);
        {
            float l[2 * G];
#pragma unroll
            for (int c = 0; c < 2 * G; ++c) l[c] = (c & 1) ? sum[c >> 1].y : sum[c >> 1].x;
            const int at = col(own());
            m->part[quad][at] = over_lanes(l, [](float a, float b) { return a + b; });
            if (quad == 0) m->inv[at] = -pick(neg);
        }
        bar_sync(bar, 128);
        if (quad == 0 && lane < W) {  // a column a lane
            const int at = group * W + lane;
            const float l = (m->part[0][at] + m->part[1][at]) + (m->part[2][at] + m->part[3][at]);
            const float ref = m->inv[at];
            m->inv[at] = l == 0.0f ? 0.0f : 1.0f / l;
            if (at < cols) {
                if (w.slot >= 0)
                    k.part_ml[w.slot * N + at] = make_float2(ref, l);
                else if (k.a.lse)
                    k.a.lse[out_row(at)] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;
            }
        }
        bar_sync(bar, 128);
        if (n > 0) {
            wait(&m->pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
            tmem_fence_after();
        }
        // (the unit's last wait is behind it: one that gave up leaves no result of the unit)
        const bool lost = *wait.abort != 0;
        if (lost && quad == 0 && lane < W && group * W + lane < cols) {
            const int at = group * W + lane;
            if (w.slot >= 0)
                k.part_ml[w.slot * N + at] = make_float2(0.0f, quiet_nan());
            else if (k.a.lse)
                k.a.lse[out_row(at)] = quiet_nan();
        }
        const int vchunks = (k.a.dv + 127) >> 7;
        if (w.slot >= 0) {
            // (a part without positions has the sum 0: its accumulators are not read)
#pragma unroll 1
            for (int b = 0; n > 0 && b < 2 * vchunks; ++b) {
                float o[X];
                tmem_ld<G>(o_tm + (b >> 1) * N + (static_cast<uint32_t>((b & 1) * 16) << 16), o);
                tmem_wait_ld();
                const int e = (b >> 1) * 128 + quad * 32 + (b & 1) * 16 + (lane >> 2);
#pragma unroll
                for (int c = 0; c < 2 * G; ++c) {
                    const int at = col(c);
                    if (at >= cols) continue;
                    float *to = k.part_o + static_cast<int64_t>(w.slot * N + at) * k.a.dv + e;
                    if (e < k.a.dv) to[0] = o[(c >> 1) * 4 + (c & 1)];
                    if (e + 8 < k.a.dv) to[8] = o[(c >> 1) * 4 + 2 + (c & 1)];
                }
            }
            return;
        }
        // A warp's columns x 32 elements through its part of a P buffer (free by now), so that whole 16-byte
        // vectors of a column are written; unit u of column j lies at unit u ^ (j / 2 mod 4).
        unsigned char *stage = smem + F::p_off + (group * 4 + quad) * (W * 64);
        float2 inv[G];
#pragma unroll
        for (int g = 0; g < G; ++g) inv[g] = lost ? make_float2(quiet_nan(), quiet_nan()) : make_float2(m->inv[col(2 * g)], m->inv[col(2 * g + 1)]);
        uint16_t *to[W / 8];  // the vectors this thread writes; null: unused
#pragma unroll
        for (int i = 0; i < W / 8; ++i) {
            const int at = group * W + i * 8 + (lane >> 2);
            to[i] = at < cols ? k.a.out + out_row(at) * k.a.dv + quad * 32 + (lane & 3) * 8 : nullptr;
        }
#pragma unroll 1
        for (int ch = 0; ch < vchunks; ++ch) {
            float o[2][X];
            if (n > 0) {
                tmem_ld<G>(o_tm + ch * N, o[0]);
                tmem_ld<G>(o_tm + ch * N + (16u << 16), o[1]);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 2 * X; ++i) o[i / X][i % X] = 0.0f;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int g = 0; g < G; g += 2) {
                    uint32_t out[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // as P^T's blocks, stored transposed: 8 elements of a column a line
                        const int gg = g + (q >> 1), i = 4 * gg + 2 * (q & 1);
                        out[q] = pack_bf16(o[b][i] * inv[gg].x, o[b][i + 1] * inv[gg].y);
                    }
                    const int j = (g + (lane >> 4)) * 8 + (lane & 7), u = b * 2 + ((lane >> 3) & 1);
                    stmatrix4_trans(smem_addr(stage) + j * 64 + ((u ^ ((j >> 1) & 3)) << 4), out);
                }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < W / 8; ++i) {
                const int j = i * 8 + (lane >> 2), u = lane & 3;
                if (to[i] && ch * 128 + quad * 32 + u * 8 < k.a.dv)
                    __stcs(reinterpret_cast<uint4 *>(to[i] + ch * 128),
                           *reinterpret_cast<const uint4 *>(stage + j * 64 + ((u ^ ((j >> 1) & 3)) << 4)));
            }
            __syncwarp();
        }
    }

    // The units from `u` on have not come: NaN where their results would go.
    __device__ __forceinline__ void give_up(int u, int units) const
    {
        constexpr int kThreads = F::soft_warps * 32;
        const int t = (group * 4 + quad) * 32 + lane;
#pragma unroll 1
        for (; u < units; ++u) {
            const Item it = item_of(k, static_cast<uint32_t>(item_number(k, m, u)));
#pragma unroll 1
            for (int r = 0; r < it.rows; ++r) {
                const int64_t first = (it.row0 + r) * k.a.h + it.head0;
#pragma unroll 1
                for (int i = t; i < it.heads * k.a.dv; i += kThreads) k.a.out[first * k.a.dv + i] = 0x7fff;
#pragma unroll 1
                for (int i = t; k.a.lse && i < it.heads; i += kThreads) k.a.lse[first + i] = quiet_nan();
            }
#pragma unroll 1
            for (int i = t; k.p.split && i < N; i += kThreads)
                k.part_ml[(2 * static_cast<int>(blockIdx.x) + (u == 0 ? 0 : 1)) * N + i] = make_float2(0.0f, quiet_nan());
        }
    }
};

// ------------------------------------------------------------------------------------ the kernel
template <int C, int N, bool FP8>
__global__ void __launch_bounds__(Cfg<C, N, FP8>::threads, 1) attention_kernel(const __grid_constant__ Kargs k)
{
    using F = Cfg<C, N, FP8>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc *m = reinterpret_cast<Misc *>(smem + F::misc_off);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (t == 0) {
        for (int i = 0; i < F::ring; ++i) {
            mbar_init(&m->full[i], FP8 ? F::set_warps : F::load_warps * 32);
            mbar_init(&m->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], F::soft_warps);
            mbar_init(&m->p_full[i], F::soft_warps);
            mbar_init(&m->pv_done[i], 1);
        }
        for (int i = 0; i < kNoted; ++i) mbar_init(&m->noted[i], F::set_warps);
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&m->unit_full[i], 1);
            mbar_init(&m->unit_empty[i], F::soft_warps + 3 + F::load_warps);
        }
        mbar_init(&m->q_full, 2);
        mbar_init(&m->q_empty, 1);
        mbar_init(&m->drained, 1);
        fence_mbar_init();
        m->abort = 0;
    }
    if (warp == F::mma_warp) tmem_alloc(&m->tmem, 512);
    find_units<F::M>(k, m, t, F::threads);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const Waiter wait{&m->abort, k.a.err_flag, k.wait_cycles};
    const int units = m->units;
    // unit i of this CTA is in slot i mod kUnits; null: it did not come
    auto take = [&](int i) -> const Unit * {
        return wait(&m->unit_full[i % kUnits], (i / kUnits) & 1) ? &m->unit[i % kUnits] : nullptr;
    };
    auto give = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->unit_empty[i % kUnits]);
    };

    if (warp >= F::load_warp0) {
        regs_to<F::load_regs, (F::load_regs > F::launch_regs)>();
        const int set = (warp - F::load_warp0) / F::set_warps;
        Loader<C, N, FP8> load{k, m, wait, smem, lane, (warp - F::load_warp0) % F::set_warps};
        load.stage = set;  // (sets take the stages in turn)
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
            load.w = take(i);
            if (!load.w) break;
            if (load.w->n > 0) {
                if (FP8)
                    load.rows_codes(set);
                else
                    load.rows_bf16();
                load.tile += load.w->n;
            }
            give(i);
        }
        cp_async_wait_all();
    } else if (warp < F::soft_warps) {
        regs_to<F::soft_regs, (F::soft_regs > F::launch_regs)>();
        const int group = warp >> 2, quad = warp & 3;
        const uint32_t at = m->tmem + (static_cast<uint32_t>(quad * 32) << 16) + group * F::cols_per_group;
        Softmax<C, N, FP8> soft{k, m, wait, smem, group, quad, lane, at, at + C * N};
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
            const Unit *w = take(i);
            // (also: the unit's P covers what every warp staged for the one before)
            if (bar_any(5, F::soft_warps * 32, w == nullptr)) {
                soft.give_up(i, units);
                break;
            }
            soft.unit(*w);
            give(i);
        }
    } else {
        regs_to<F::mma_regs, false>();
        if (warp == F::mma_warp) {
            Issuer<C, N, FP8> issue{m, wait};
            issue.ring_k = umma_desc(smem_addr(smem), 16, 1024);
            issue.ring_v = umma_desc(smem_addr(smem), F::half_bytes, 1024);
            issue.q0 = umma_desc(smem_addr(smem + F::q_off), 16, 1024);
            issue.p0 = umma_desc(smem_addr(smem + F::p_off), F::p_block, 1024);
            const uint32_t tm = __reduce_max_sync(0xffffffffu, m->tmem);  // (uniform)
            issue.o_col = tm;
            issue.s_col = tm + C * N;
            issue.halves = (k.a.d + 63) >> 6;
            issue.vchunks = (k.a.dv + 127) >> 7;
            int loaded = 0;
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                const Unit *w = take(i);
                if (!w) break;
                const int n = __reduce_max_sync(0xffffffffu, w->n);
                if (n > 0) issue.unit(n, loaded++ & 1);
                give(i);
            }
            // no product is under way when the tensor memory is freed.  (This wait has the whole limit, whoever gave up.)
            if (elect_one()) umma_commit(&m->drained);
            int none = 0;
            Waiter{&none, k.a.err_flag, kWaitCycles}(&m->drained, 0);
        } else if (warp == F::unit_warp) {
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                if (!wait(&m->unit_empty[i % kUnits], ((i / kUnits) & 1) ^ 1)) break;
                make_unit<N, F::M>(k, m, i, &m->unit[i % kUnits], lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&m->unit_full[i % kUnits]);
            }
        } else {
            int loaded = 0;
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                const Unit *w = take(i);
                if (!w) break;
                if (w->n > 0) {
                    wait(&m->q_empty, (loaded++ & 1) ^ 1);
                    load_queries<C, N, FP8>(k, w, m, smem, warp - F::unit_warp - 1, lane);
                }
                give(i);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == F::mma_warp) tmem_dealloc(m->tmem, 512);
}

// Joins the parts of each column: out = sum_p 2^(ref_p - max) o_p / sum_p 2^(ref_p - max) sum_p.  A CTA a
// column; `V` threads have 4 elements of a part each, and the CTA's groups of as many take every groups-th part, so
// that few loads follow one another: their latency bounds it (4 rows x 64 heads of 512 over 204800 positions, 39
// parts a column: 178 us with one group of 128 threads, 169.5 with four).  Launched ahead of the first kernel's end.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Kargs k, int V)
{
    __shared__ float2 part[kMaxCtas];  // reference and sum, then factor and sum, of each part
    __shared__ float4 partial[kJoinThreads];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: until the parts are there
    const int N = k.p.cols, dv = k.a.dv, t = threadIdx.x, lane = t & 31;
    const uint32_t item = blockIdx.x / static_cast<uint32_t>(N);
    const int col = static_cast<int>(blockIdx.x - item * static_cast<uint32_t>(N));
    const int4 at = k.parts[item];
    if (at.x < 0) return;  // a whole one
    const Item it = item_of(k, item);
    if (col >= it.rows * it.heads) return;
    auto slot = [&](int p) { return static_cast<int64_t>(p == 0 ? at.x : 2 * (at.y + p)) * N + col; };
    const int parts = at.z - at.y + 1;
    for (int p = t; p < parts; p += blockDim.x) part[p] = k.part_ml[slot(p)];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;  // (each warp for itself, in the same order)
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, part[p].y != 0.0f ? part[p].x : -INFINITY);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    auto factor = [&](float2 v) { return v.y == 0.0f ? 0.0f : v.x == top ? 1.0f : exp2_approx(v.x - top); };
    for (int p = lane; p < parts; p += 32) sum += factor(part[p]) * part[p].y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const int groups = blockDim.x / V, group = t / V, e = (t - group * V) * 4;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int p = group; p < parts; p += groups) {
        const float2 v = part[p];
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // (a part whose sum is 0 has written no accumulators)
        if (e < dv && v.y != 0.0f) o = *reinterpret_cast<const float4 *>(k.part_o + slot(p) * dv + e);
        const float f = factor(v);
        acc.x += f * o.x, acc.y += f * o.y, acc.z += f * o.z, acc.w += f * o.w;
    }
    if (groups > 1) {
        partial[t] = acc;
        __syncthreads();
        if (group > 0) return;
        for (int g = 1; g < groups; ++g) {
            const float4 o = partial[g * V + t];
            acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
        }
    }
    const int row = col / it.heads;
    const int64_t out = (it.row0 + row) * k.a.h + it.head0 + col - row * it.heads;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (e < dv)
        *reinterpret_cast<uint2 *>(k.a.out + out * dv + e) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (t == 0 && k.a.lse) k.a.lse[out] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

// The current device's SMs, asked for once a device.
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 64) return device_sm_count();
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) known[dev].store(n = device_sm_count(), std::memory_order_relaxed);
    return n;
}

template <int C, int N, bool FP8>
cudaError_t launch(const Kargs &k, cudaStream_t s)
{
    using F = Cfg<C, N, FP8>;
    constexpr size_t smem = F::misc_off + sizeof(Misc);
    static_assert(smem <= 232448, "more than a CTA may use");
    static_assert(smem > 116 * 1024, "one CTA an SM: each takes all of the tensor memory");
    static_assert(N * 256 <= F::pbufs * F::p_bytes, "outputs are staged where P was");
    // the attribute is set once on each device (a device past the mask's 64: on each call)
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(attention_kernel<C, N, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    attention_kernel<C, N, FP8><<<static_cast<unsigned>(k.p.ctas), F::threads, smem, s>>>(k);
    return cudaGetLastError();
}

template <int C, int N>
cudaError_t launch(const Kargs &k, cudaStream_t s)
{
    return k.a.c.scales ? launch<C, N, true>(k, s) : launch<C, N, false>(k, s);
}

Plan plan_of(int64_t rows, int64_t h, int64_t d, int64_t b, int64_t positions, bool idx_given)
{
    Plan p{};
    const int64_t per = rows / b;
    // 128 columns where the kernel has them and rows and heads fill more than 64
    const int64_t cols = d <= 192 && (idx_given ? h : h * per) > 64 ? 128 : 64;
    p.cols = static_cast<int>(cols);
    p.heads_per_tile = static_cast<int>(h < cols ? h : cols);
    p.head_blocks = static_cast<int>((h + cols - 1) / cols);
    // rows that share a tile share its positions; a row with a list has its own
    const int64_t fit = idx_given ? 1 : cols / p.heads_per_tile;
    p.rows_per_tile = static_cast<int>(fit < per ? fit : per);
    p.tiles_per_seq = (per + p.rows_per_tile - 1) / p.rows_per_tile;
    p.items = b * p.tiles_per_seq * p.head_blocks;
    // Few items: their tiles are shared out, where that leaves the fewest tiles in a row, counting a part's start
    // and end as 1.5 tiles and the join as 1.
    const int64_t tiles = positions > 128 ? (positions + 127) / 128 : 1;
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    const int64_t waves = (p.items + sms - 1) / sms;
    const double whole = static_cast<double>(waves) * (static_cast<double>(tiles) + 1.5);
    const int64_t all = p.items * (tiles + kStart), most = sms < kMaxCtas ? sms : kMaxCtas, ctas = all < most ? all : most;
    const double shared = static_cast<double>((all + ctas - 1) / ctas) + 1.5 + 1.0;
    p.split = p.items <= kMaxItems && p.items < 2 * sms && all < 0x7fffffff / (sms + 1) && shared < whole;
    p.ctas = static_cast<int>(p.split ? ctas : p.items < sms ? p.items : sms);
    return p;
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }
size_t parts_bytes(const Plan &p) { return rounded(static_cast<size_t>(p.items) * sizeof(int4)); }
size_t ml_bytes(const Plan &p) { return rounded(static_cast<size_t>(2) * p.ctas * p.cols * sizeof(float2)); }

}  // namespace

size_t cache_attention_workspace(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b, int64_t positions,
                                 bool idx_given)
{
    const Plan p = plan_of(rows, h, d, b, positions, idx_given);
    if (!p.split) return 0;
    return parts_bytes(p) + ml_bytes(p) + static_cast<size_t>(2) * p.ctas * p.cols * dv * sizeof(float);
}

static std::atomic<long long> g_wait_cycles{kWaitCycles};

void set_cache_wait_cycles(long long cycles)
{
    g_wait_cycles.store(cycles < 0 ? kWaitCycles : cycles, std::memory_order_relaxed);
}

cudaError_t launch_cache_attention(const CacheAttnArgs &a, cudaStream_t s)
{
    Kargs k{};
    k.a = a;
    k.wait_cycles = g_wait_cycles.load(std::memory_order_relaxed);
    k.p = plan_of(a.rows, a.h, a.d, a.rows / a.t.rows_per_seq, a.idx ? a.n : a.t.max_pages * a.c.page_size, a.idx != nullptr);
    if (k.p.split) {
        unsigned char *ws = static_cast<unsigned char *>(a.ws);
        k.parts = reinterpret_cast<int4 *>(ws);
        k.part_ml = reinterpret_cast<float2 *>(ws + parts_bytes(k.p));
        k.part_o = reinterpret_cast<float *>(ws + parts_bytes(k.p) + ml_bytes(k.p));
    }
    cudaError_t e;
    if (k.p.cols == 128)
        e = a.d <= 128 ? launch<1, 128>(k, s) : launch<2, 128>(k, s);
    else if (a.d <= 256)
        e = a.d <= 128 ? launch<1, 64>(k, s) : launch<2, 64>(k, s);
    else
        e = a.d <= 384 ? launch<3, 64>(k, s) : launch<4, 64>(k, s);
    if (e != cudaSuccess || !k.p.split) return e;
    // groups for half of the parts that a column has, as long as all threads are resident at once (2048 columns of
    // 6 parts: 119 us with the first kernel by one group, 121 by two, 127 by four)
    int vecs = 32;
    while (vecs * 4 < a.dv) vecs *= 2;
    const int64_t columns = k.p.items * k.p.cols, parts = (k.p.ctas + k.p.items) / k.p.items, sms = sm_count();
    int threads = vecs;
    while (threads < kJoinThreads && threads / vecs * 2 < parts && columns * threads * 2 <= 2048 * sms) threads *= 2;
    cudaLaunchConfig_t at = {};
    at.gridDim = dim3(static_cast<unsigned>(k.p.items * k.p.cols));
    at.blockDim = dim3(static_cast<unsigned>(threads));
    at.stream = s;
    cudaLaunchAttribute ahead;
    ahead.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ahead.val.programmaticStreamSerializationAllowed = 1;
    at.attrs = &ahead;
    at.numAttrs = 1;
    return cudaLaunchKernelEx(&at, join_kernel, k, vecs);
}

}  // namespace sel
