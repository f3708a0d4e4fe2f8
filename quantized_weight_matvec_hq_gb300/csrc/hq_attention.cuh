// hq_attention.cuh -- how the attention of a batch is divided among blocks.
//
// An item is a tile of a request's query rows on one key/value head: up to `tokens` neighbouring tokens with all heads
// of the group, or, where a group has more heads than a tile has rows, one token with a part of them.  The positions that an item
// sees are cut into units of 2^unit_shift; the units of all items, one after another, are dealt to the blocks in equal
// contiguous ranges.  Lengths are known on the device only, so every block finds its range itself.
// An item that one block has whole is finished there; of the others each block leaves a partial result (its maximum, sum
// and weighted sum), and the combine kernel joins them.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "hq_cache.cuh"

namespace hq {

struct AttnArgs {
    CacheView c;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    int dtype;                          // of q and out: HQ_DT_*
    int n_heads, group;                 // heads, and those that share a key/value head
    int tokens, part_heads, parts;      // of a tile: tokens, heads of a group, and tiles a group takes
    int inv_heads;                      // 2^16 / part_heads, rounded up: quotients of numbers below 128
    int causal;
    float scale;
    long long window;                   // 0: none
    float *partial;                     // [2 blocks][rows][head_dim]
    float2 *stat;                       // [2 blocks][rows]: maximum and sum of a partial result
    struct Join *joins;                 // [blocks]
    int unit_shift, blocks;
    long long most_units;               // an item can have
};

// sum of floor((a i + b) / 2^shift) for i < n; a, b >= 0, a n below 2^31 (the Euclidean recursion; behind its first step
// everything fits 32 bits, whose divisions are a fraction of the 64-bit ones')
__device__ __forceinline__ long long floor_sum(long long n, int shift, long long a, long long b) {
    if (n <= 0) return 0;
    unsigned m = 1u << shift;
    long long s = (n - 1) * n / 2 * (a >> shift) + n * (b >> shift);
    unsigned x = (unsigned)a & (m - 1), y = (unsigned)b & (m - 1), top = x * (unsigned)n + y;
    while (top >= m) {
        const unsigned k = top / m;                         // the next sum: k terms, of slope m over x
        y = top % m;
        s += (long long)(k - 1) * k / 2 * (m / x) + (long long)k * (y / x);
        const unsigned slope = m % x;
        y %= x;
        top = slope * k + y;
        m = x;
        x = slope;
    }
    return s;
}

// sum of floor(max(0, c + tokens j) / 2^shift) for j < n
__device__ __forceinline__ long long unit_sum(int n, long long c, int tokens, int shift) {
    if (n <= 0) return 0;
    if (n == 1) return c > 0 ? c >> shift : 0;
    const long long skip = c < 0 ? (-c + tokens - 1) / tokens : 0;
    return floor_sum(n - skip, shift, tokens, c + skip * tokens);
}

// Positions [lo, hi) that a token sees.
struct Range { int lo, hi; };
__device__ __forceinline__ Range seen_by(const AttnArgs &a, const Request &q, int token) {
    const int at = q.length - q.n + token;
    Range s;
    s.hi = a.causal ? max(at + 1, 0) : q.length;
    s.lo = a.window > 0 && a.window <= at ? at + 1 - (int)a.window : 0;
    return s;
}

__device__ __forceinline__ int tiles_of(const AttnArgs &a, const Request &q) { return (q.n + a.tokens - 1) / a.tokens; }

// Units of the tiles before tile j, on one head and part.  A tile sees what its first token's window begins with up to its
// last token's position; it has at least one unit, so that rows that see nothing are written too.
__device__ __forceinline__ long long units_before(const AttnArgs &a, const Request &q, int j) {
    if (j == 0) return 0;
    if (!a.causal) return (long long)j * max(1, (q.length + (1 << a.unit_shift) - 1) >> a.unit_shift);
    const int base = q.length - q.n, n = tiles_of(a, q);
    long long u = j;                                        // 1 + floor((last position) / unit) each
    u += unit_sum(j - (j == n), (long long)base + a.tokens - 1, a.tokens, a.unit_shift);
    if (j == n && q.length > 0) u += (q.length - 1) >> a.unit_shift;
    if (a.window > 0) u -= unit_sum(j, (long long)base + 1 - a.window, a.tokens, a.unit_shift);
    return u;
}

__device__ __forceinline__ long long request_units(const AttnArgs &a, const Request &q) {
    return q.n == 0 ? 0 : units_before(a, q, tiles_of(a, q)) * a.c.n_kv_heads * a.parts;
}

// A block's way through the units: the request that it is at.
struct Walk {
    long long start, next;              // units before the request, and up to its end
    int r;                              // that request
    Request q;
};

// The item of a unit, and which of its units that is.
struct Item {
    int tile, kv_head, part;            // of a request
    long long first;                    // its first unit
    int units, unit;                    // how many it has, and which one it is
};

// A block's part of an item: `take` units from `unit` on.  What the producer warp tells the consumers.
struct Part {
    Request q;
    Item item;
    int take, slot;                     // 0: no more; where the partial result goes, or -1: the whole item
    int begin;                          // the position of its first unit
    Range span;                         // positions of it that some row sees
    int all_lo, all_hi;                 // every row sees [all_lo, all_hi) of them
};
// What the combine kernel is told: the item that begins in a block (with its first unit, or with the block's) and goes on
// past its end, in which of the block's two partial results it begins, and the last block that has one.
struct Join {
    Request q;
    Item item;
    int valid, slot, last;
};

struct WalkShared {
    long long warp_sum[32];
    Walk walk;
};

// Inclusive scan over the THREADS threads that call (the block, or a warp); every thread gets their sum.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long &sum, WalkShared &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += w;
    }
    if constexpr (THREADS == 32) {
        sum = __shfl_sync(0xffffffffu, v, 31);
        return v;
    } else {
        __syncthreads();
        if (lane == 31) s.warp_sum[warp] = v;
        __syncthreads();
        sum = 0;
        long long before = 0;
        for (int i = 0; i < THREADS / 32; ++i) {
            if (i < warp) before += s.warp_sum[i];
            sum += s.warp_sum[i];
        }
        return v + before;
    }
}

// Takes the walk to the request with unit x, looking from request r0 on, which begins at unit `start`.  The whole
// block calls it, or (THREADS 32) one warp; x is below the batch's units.
template <int THREADS>
__device__ __forceinline__ void walk_to(const AttnArgs &a, long long x, int r0, long long start, WalkShared &s) {
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    for (long long i = r0; i < a.c.n_req; i += THREADS) {
        const long long r = i + tid;
        Request q = {0, 0, 0, false};
        if (r < a.c.n_req) q = request_of(a.c, (int)r);
        const long long u = request_units(a, q);
        long long sum;
        const long long upto = start + block_scan<THREADS>(u, sum, s);
        if (x >= upto - u && x < upto) {
            s.walk.r = (int)r;
            s.walk.start = upto - u;
            s.walk.next = upto;
            s.walk.q = q;
        }
        start += sum;
        if (x < start) break;
    }
    if (THREADS == 32) __syncwarp(); else __syncthreads();
}

// a / b for a >= 0, b > 0: in 32 bits where they fit, a fraction of the instructions.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The first unit of block `b`.  Fewer units than blocks go to as many blocks.
__device__ __forceinline__ long long first_unit(const AttnArgs &a, long long total, int b) {
    const long long n = min((long long)a.blocks, total);
    return b >= n ? total : quotient(total * b, n);
}

// The block that has a unit.
__device__ __forceinline__ int block_of(const AttnArgs &a, long long total, long long unit) {
    const long long n = min((long long)a.blocks, total);
    return (int)quotient((unit + 1) * n - 1, total);
}

// This block's units [x0, end) of the batch's `total`, and the walk at the first one's request.  The whole block calls it.
template <int THREADS>
__device__ __forceinline__ void deal(const AttnArgs &a, long long &total, long long &x0, long long &end, WalkShared &s) {
    if (threadIdx.x == 0) a.joins[blockIdx.x].valid = 0;
    long long mine = 0;
    Request q = {0, 0, 0, false};
    for (int r = threadIdx.x; r < a.c.n_req; r += THREADS) {
        q = request_of(a.c, r);
        if (q.bad && blockIdx.x == 0) atomicOr(a.c.fault, kFaultCache);
        mine += request_units(a, q);
    }
    const long long upto = block_scan<THREADS>(mine, total, s);
    x0 = first_unit(a, total, blockIdx.x);
    end = first_unit(a, total, blockIdx.x + 1);
    if (x0 >= end) return;
    if (a.c.n_req > THREADS) {
        walk_to<THREADS>(a, x0, 0, 0, s);
        return;
    }
    if (x0 >= upto - mine && x0 < upto) {                   // a request a thread: its own
        s.walk.r = threadIdx.x;
        s.walk.start = upto - mine;
        s.walk.next = upto;
        s.walk.q = q;
    }
    __syncthreads();
}

// The whole warp calls it, all lanes for the same unit: each step of the search looks at 32 tiles.
__device__ __forceinline__ Item item_at(const AttnArgs &a, const Walk &w, long long x) {
    const long long local = x - w.start;
    const int heads = a.c.n_kv_heads * a.parts, lane = threadIdx.x & 31;
    int lo = 0, n = tiles_of(a, w.q);                       // the last tile with units_before * heads <= local is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, at < n && units_before(a, w.q, lo + at) * heads <= local);
        const int k = 31 - __clz(m);                        // (lane 0 always is)
        lo += k * step;
        n = min(step, n - k * step);
    }
    const long long before = units_before(a, w.q, lo);
    Item it;
    it.tile = lo;
    it.units = (int)(units_before(a, w.q, lo + 1) - before);
    const long long rest = local - before * heads;
    const int h = (int)quotient(rest, it.units);
    it.kv_head = h / a.parts;
    it.part = h % a.parts;
    it.unit = (int)(rest - (long long)h * it.units);
    it.first = x - it.unit;
    return it;
}

// The part at unit x of a block with units [x0, end), into shared memory; and the block's join, if that is it.  A whole warp.
__device__ __forceinline__ void tell_part(const AttnArgs &a, const Walk &w, long long x, long long x0, long long end, long long total,
                                          Part &p) {
    const Item it = item_at(a, w, x);
    if ((threadIdx.x & 31) == 0) {
        const int take = (int)min((long long)(it.units - it.unit), end - x);
        const int slot = take == it.units ? -1 : 2 * (int)blockIdx.x + (x == x0 ? 0 : 1);
        const int t0 = it.tile * a.tokens, t1 = min(t0 + a.tokens, w.q.n) - 1;
        const Range first = seen_by(a, w.q, t0), last = seen_by(a, w.q, t1);
        const int begin = ((first.lo >> a.unit_shift) + it.unit) << a.unit_shift;
        p.q = w.q;
        p.item = it;
        p.take = take;
        p.slot = slot;
        p.begin = begin;
        p.span = {first.lo, min(begin + (take << a.unit_shift), last.hi)};
        p.all_lo = last.lo;
        p.all_hi = first.hi;
        if (it.unit + take < it.units && it.first >= x0) {
            Join &j = a.joins[blockIdx.x];
            j.q = w.q;
            j.item = it;
            j.slot = slot;
            j.last = block_of(a, total, it.first + it.units - 1);
            j.valid = 1;
        }
    }
    __syncwarp();
}

// Row i of an item is token tile * tokens + i / part_heads of the request, and of its group head part * part_heads + i % part_heads.
__device__ __forceinline__ bool row_of(const AttnArgs &a, const Request &q, const Item &it, int i, int &token, int &head) {
    const int t = i * a.inv_heads >> 16;                    // i / part_heads
    token = it.tile * a.tokens + t;
    const int h = it.part * a.part_heads + i - t * a.part_heads;
    head = it.kv_head * a.group + h;
    return i < a.tokens * a.part_heads && token < q.n && h < a.group;
}

// 8 neighbouring elements of a token's row of type WIDE ? fp32 : a.dtype.
template <bool WIDE>
__device__ __forceinline__ void load_row8(const AttnArgs &a, long long at, float (&v)[8]) {
    if (WIDE) load8(static_cast<const float *>(a.q) + at, v);
    else if (a.dtype == HQ_DT_F16) load8(static_cast<const __half *>(a.q) + at, v);
    else load8(static_cast<const __nv_bfloat16 *>(a.q) + at, v);
}
template <bool WIDE>
__device__ __forceinline__ void store_row8(const AttnArgs &a, long long at, const float (&v)[8]) {
    if (WIDE) store8(static_cast<float *>(a.out) + at, v);
    else if (a.dtype == HQ_DT_F16) store8(static_cast<__half *>(a.out) + at, v);
    else store8(static_cast<__nv_bfloat16 *>(a.out) + at, v);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ host side

// Blocks of a launch: those that fit a multiprocessor, by the registers that a thread needs (few rows, of 5 warps each: 4 blocks 96, 3: 128,
// 2: 168), or the shared memory (tiles).  At most kSms times that: the workspace holds two partial results of each.
constexpr int kSms = 152;
constexpr int stream_blocks(bool wide, int dim, int rows) {
    return rows == 8 ? (dim == 256 ? 2 : wide && dim == 128 ? 3 : 4) : dim == 64 && !wide ? 3 : 2;
}
constexpr int tile_blocks(int dim) { return dim == 256 ? 1 : 2; }

// Allows a kernel its shared memory, once a device.
template <class K>
hq_status allow_smem(K kern, int bytes, std::atomic<bool> (&done)[64]) {
    int d = 0;
    cudaGetDevice(&d);
    if (d >= 0 && d < 64 && done[d].load(std::memory_order_acquire)) return HQ_OK;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    if (d >= 0 && d < 64) done[d].store(true, std::memory_order_release);
    return HQ_OK;
}

template <class K, class... A>
hq_status launch_blocks(K kern, dim3 grid, int threads, int smem, cudaStream_t stream, const char *what, const A &... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "%s launch: %s", what, cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

// A window of at least the positions that a request can have hides none of them: it is no window.  (Windows of any size are
// allowed, and the sums of units are for those below 2^30.)
inline long long window_of(long long window, const CacheView &c) { return window < c.table_width << c.page_shift ? window : 0; }

// Tiles of `rows` query rows, units of 2^unit_shift positions, no more blocks than there can be units, and the workspace.
inline void deal_rows(AttnArgs &a, int rows, int dim, int unit_shift, int blocks) {
    a.tokens = a.group <= rows ? rows / a.group : 1;
    a.part_heads = a.group <= rows ? a.group : rows;
    a.parts = (a.group + a.part_heads - 1) / a.part_heads;
    a.inv_heads = (65536 + a.part_heads - 1) / a.part_heads;
    a.unit_shift = unit_shift;
    const long long tiles = std::min(a.c.n_tokens, a.c.n_tokens / a.tokens + a.c.n_req);
    a.most_units = ((a.c.table_width << a.c.page_shift) + (1 << unit_shift) - 1) >> unit_shift;
    const double most = (double)tiles * a.c.n_kv_heads * a.parts * a.most_units;
    a.blocks = blocks;
    if (most < a.blocks) a.blocks = (int)most;
    a.stat = reinterpret_cast<float2 *>(a.partial + 2ll * a.blocks * rows * dim);
    a.joins = reinterpret_cast<Join *>(a.stat + 2ll * a.blocks * rows);
}

// Joins partial results, where there can be any: 16-bit tokens, tiles of `rows`.
hq_status run_attention_combine(const AttnArgs &a, int rows, int dim, cudaStream_t stream);
// The kernel for many rows, 16-bit tokens.
hq_status run_attention_tile(const AttnArgs &a, int fmt, int dim, int num_sms, cudaStream_t stream);

}  // namespace hq
