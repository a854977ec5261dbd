// cache_attention.cu -- attention over a paged cache: which layout a call takes, how its work is shared out, and the
// join of the parts (the kernel is in cache_attention.cuh).
#include "cache_attention.cuh"

namespace sel {
namespace {

// Joins the parts of each column: out = sum_p 2^(ref_p - max) o_p / sum_p 2^(ref_p - max) sum_p.  A CTA a
// column; `V` threads have 4 elements of a part each, and the CTA's groups of as many take every groups-th part, so
// that few loads follow one another: their latency bounds it (4 rows x 64 heads of 512 over 204800 positions, 39
// parts a column: 178 us with one group of 128 threads, 169.5 with four).  Launched ahead of the first kernel's end.
// SHARED: a column's parts are those of the shared prefix, then those of its sequence's own positions.
constexpr int kJoinThreads = 512;
template <bool SHARED>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Kargs k, int V)
{
    __shared__ float2 part[kMaxCtas + 1];  // (two items share a CTA at most)
    // reference and sum, then factor and sum, of each part
    __shared__ float4 partial[kJoinThreads];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched ahead: until the parts are there
    const int N = k.p.cols, dv = k.a.dv, t = threadIdx.x, lane = t & 31;
    int64_t out;              // row * heads + head
    int4 at[SHARED ? 2 : 1];  // of each item: its first part's slot (-1: it is a whole one), its first CTA and last
    int col[SHARED ? 2 : 1], count[SHARED ? 2 : 1];
    if (SHARED) {
        out = blockIdx.x;
        const uint32_t h = static_cast<uint32_t>(k.a.h), row = blockIdx.x / h, head = blockIdx.x - row * h;
        const uint32_t seq = row / static_cast<uint32_t>(k.a.t.rows_per_seq);
        const uint32_t in_seq = row - seq * static_cast<uint32_t>(k.a.t.rows_per_seq);
        const uint32_t rows[2] = {static_cast<uint32_t>(k.p.prefix_rows), static_cast<uint32_t>(k.p.rows_per_tile)};
        const uint32_t in[2] = {row, in_seq};  // the rows before it of those dealt out in tiles
        const uint32_t first[2] = {0, static_cast<uint32_t>(k.p.prefix_items) + seq * static_cast<uint32_t>(k.p.tiles_per_seq)};
#pragma unroll
        for (int i = 0; i < (SHARED ? 2 : 1); ++i) {
            const uint32_t tile = in[i] / rows[i];
            col[i] = static_cast<int>((in[i] - tile * rows[i]) * h + head);
            at[i] = k.p.split ? k.parts[first[i] + tile] : make_int4(-1, 0, 0, 0);
            count[i] = at[i].x < 0 ? 1 : at[i].z - at[i].y + 1;
        }
    } else {
        const uint32_t item = blockIdx.x / static_cast<uint32_t>(N);
        col[0] = static_cast<int>(blockIdx.x - item * static_cast<uint32_t>(N));
        at[0] = k.parts[item];
        if (at[0].x < 0) return;  // a whole one
        const Item it = item_of<false>(k, item);
        if (col[0] >= it.rows * it.heads) return;
        count[0] = at[0].z - at[0].y + 1;
        const int row = col[0] / it.heads;
        out = (it.row0 + row) * k.a.h + it.head0 + col[0] - row * it.heads;
    }
    auto slot_in = [&](int i, int p) {
        if (SHARED && at[i].x < 0) return k.whole0 + i * (k.a.rows * k.a.h) + out;
        return static_cast<int64_t>(p == 0 ? at[i].x : 2 * (at[i].y + p)) * N + col[i];
    };
    auto slot = [&](int p) { return SHARED && p >= count[0] ? slot_in(SHARED ? 1 : 0, p - count[0]) : slot_in(0, p); };
    const int parts = SHARED ? count[0] + count[SHARED ? 1 : 0] : count[0];
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

Plan plan_of(int64_t rows, int64_t h, int64_t d, int64_t b, int64_t positions, bool idx_given, int64_t sms)
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
    const int64_t waves = (p.items + sms - 1) / sms;
    const double whole = static_cast<double>(waves) * (static_cast<double>(tiles) + 1.5);
    const int64_t all = p.items * (tiles + kStart), most = sms < kMaxCtas ? sms : kMaxCtas, ctas = all < most ? all : most;
    const double shared = static_cast<double>((all + ctas - 1) / ctas) + 1.5 + 1.0;
    p.split = p.items <= kMaxItems && p.items < 2 * sms && all < 0x7fffffff / (sms + 1) && shared < whole;
    p.ctas = static_cast<int>(p.split ? ctas : p.items < sms ? p.items : sms);
    return p;
}

// The same under a window: `reach` positions at most are visible to a row, and fewer than rows_per_tile more to the rows
// of a tile where their ends follow one another.  (Where they do not, an item may be as long as the page table, whose
// tiles have to be countable all the same.)
Plan plan_window(int64_t rows, int64_t h, int64_t d, int64_t b, int64_t positions, int64_t reach, int64_t sms)
{
    Plan p = plan_of(rows, h, d, b, positions, false, sms);
    const int64_t most = reach + p.rows_per_tile - 1;
    if (most >= positions) return p;
    p = plan_of(rows, h, d, b, most, false, sms);
    if (p.split && p.items * (positions / 128 + 1 + kStartRanges) >= 0x7fffffff / (sms + 1)) {
        p.split = 0;
        p.ctas = static_cast<int>(p.items < sms ? p.items : sms);
    }
    return p;
}

// With a shared prefix: the rows of all sequences attend to it by tiles of their own, where a sequence's rows do not
// fill a tile by themselves, and where that makes less of the work, counted as in plan_of (there a part's or an
// item's start, here the join is always taken).  Else prefix_items is 0, and every sequence reads its own page table.
Plan plan_shared(int64_t rows, int64_t h, int64_t d, int64_t b, int64_t positions, int64_t shared, int64_t sms)
{
    const Plan plain = plan_of(rows, h, d, b, positions, false, sms);
    const int64_t per = rows / b, prefix = shared < positions ? shared : positions;
    const int64_t cols = d <= 192 && h * rows > 64 ? 128 : 64;
    if (prefix <= 0 || b < 2 || h * per >= cols) return plain;
    Plan p{};
    p.cols = static_cast<int>(cols);
    p.heads_per_tile = static_cast<int>(h);
    p.head_blocks = 1;
    p.rows_per_tile = static_cast<int>(per);  // (all of a sequence's fit)
    p.tiles_per_seq = 1;
    p.prefix_rows = static_cast<int>(cols / h < rows ? cols / h : rows);
    p.prefix_items = (rows + p.prefix_rows - 1) / p.prefix_rows;
    p.items = p.prefix_items + b;
    const int64_t most = sms < kMaxCtas ? sms : kMaxCtas;
    const int64_t own = (positions - prefix + 127) / 128;
    const int64_t all = p.prefix_items * ((prefix + 127) / 128 + kStartRanges) + b * (own + kStartRanges);
    p.split = p.items <= kMaxItems && all < 0x7fffffff / (sms + 1);
    p.ctas = static_cast<int>(p.split ? (all < most ? all : most) : p.items < sms ? p.items : sms);
    const int64_t counted = all - p.items * (kStartRanges - kStart);  // (a start counts for both alike)
    const double grouped = static_cast<double>((counted + sms - 1) / sms) + 1.5 + 1.0;
    const int64_t tiles = (positions + 127) / 128, waves = (plain.items + sms - 1) / sms;
    const double apart = plain.split ? static_cast<double>((plain.items * (tiles + kStart) + plain.ctas - 1) / plain.ctas) + 1.5 + 1.0
                                     : static_cast<double>(waves) * (static_cast<double>(tiles) + 1.5);
    return grouped < apart ? p : plain;
}

Plan plan_for(int64_t rows, int64_t h, int64_t d, int64_t b, int64_t positions, bool idx_given, const Seen &seen)
{
    const int64_t known = sm_count(), sms = known > 0 ? known : 1;
    if (seen.window > 0) return plan_window(rows, h, d, b, positions, int64_t{seen.window} + seen.sinks, sms);
    if (seen.shared > 0) return plan_shared(rows, h, d, b, positions, seen.shared, sms);
    return plan_of(rows, h, d, b, positions, idx_given, sms);
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }
size_t parts_bytes(const Plan &p) { return rounded(static_cast<size_t>(p.items) * sizeof(int4)); }
// The parts of an item each CTA's two slots have columns for, and behind them those of whole items (shared prefix).
size_t slot_columns(const Plan &p) { return p.split ? static_cast<size_t>(2) * p.ctas * p.cols : 0; }
size_t part_columns(const Plan &p, int64_t rows, int64_t h)
{
    return slot_columns(p) + (p.prefix_items > 0 ? static_cast<size_t>(2) * rows * h : 0);
}

}  // namespace

size_t cache_attention_workspace(int64_t rows, int64_t h, int64_t d, int64_t dv, int64_t b, int64_t positions,
                                 bool idx_given, const Seen &seen)
{
    const Plan p = plan_for(rows, h, d, b, positions, idx_given, seen);
    if (!p.split && p.prefix_items == 0) return 0;
    const size_t columns = part_columns(p, rows, h);
    return parts_bytes(p) + rounded(columns * sizeof(float2)) + columns * dv * sizeof(float);
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
    k.p = plan_for(a.rows, a.h, a.d, a.rows / a.t.rows_per_seq, a.idx ? a.n : a.t.max_pages * a.c.page_size, a.idx != nullptr,
                   a.seen);
    const bool grouped = k.p.prefix_items > 0;
    if (k.p.split || grouped) {
        unsigned char *ws = static_cast<unsigned char *>(a.ws);
        k.parts = reinterpret_cast<int4 *>(ws);
        k.part_ml = reinterpret_cast<float2 *>(ws + parts_bytes(k.p));
        k.part_o = reinterpret_cast<float *>(ws + parts_bytes(k.p) + rounded(part_columns(k.p, a.rows, a.h) * sizeof(float2)));
        k.whole0 = static_cast<int64_t>(slot_columns(k.p));
    }
    const cudaError_t e = grouped || a.seen.window > 0 ? launch_attention_ranges(k, s) : launch_layout<false>(k, s);
    if (e != cudaSuccess || !(k.p.split || grouped)) return e;
    // groups for half of the parts that a column has, as long as all threads are resident at once (2048 columns of
    // 6 parts: 119 us with the first kernel by one group, 121 by two, 127 by four)
    int vecs = 32;
    while (vecs * 4 < a.dv) vecs *= 2;
    const int64_t columns = grouped ? a.rows * a.h : k.p.items * k.p.cols;
    // (of a shared prefix's items, which are cut most, as many as all CTAs come to)
    const int64_t cut = grouped ? k.p.prefix_items : k.p.items, parts = k.p.split ? (k.p.ctas + cut) / cut : 2, sms = sm_count();
    int threads = vecs;
    while (threads < kJoinThreads && threads / vecs * 2 < parts && columns * threads * 2 <= 2048 * sms) threads *= 2;
    cudaLaunchConfig_t at = {};
    at.gridDim = dim3(static_cast<unsigned>(columns));
    at.blockDim = dim3(static_cast<unsigned>(threads));
    at.stream = s;
    cudaLaunchAttribute ahead;
    ahead.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ahead.val.programmaticStreamSerializationAllowed = 1;
    at.attrs = &ahead;
    at.numAttrs = 1;
    return cudaLaunchKernelEx(&at, grouped ? join_kernel<true> : join_kernel<false>, k, vecs);
}

}  // namespace sel
