// hq_matmul.cu -- products of many tokens with quantized weights on the tensor
// cores: grouped by expert, or shared with an adapter per request.
//
//   y[s][i] = sum_j w[m(s)][i][j] x[s][j],  w = d q (Q8_0) or d (n - 8) (Q4_0)
//
// A prepare kernel lays the call out, then one persistent kernel multiplies:
//  * The weights are the M operand (128 rows of W a tile) and the tokens the N
//    operand (16 to 192 a tile), so ragged groups of tokens cost what they are.
//  * Raw blocks come by TMA (256 columns of 128 rows a chunk).  Four groups of four warps
//    decode a quarter (64 columns) each to 16-bit floats, a row a thread, and store them to TMEM, from where
//    the tensor core reads them.  (Through shared memory, decoded weights were written and read
//    at 256 of the about 440 to 880 cycles of its bandwidth that 64 columns took, and it was the limit.)
//    Each scheduler has a warp of every group, so that the groups' loads, waits and arithmetic overlap.
//  * Tokens come by TMA, an expert's tokens next to each other (the prepare kernel sorts them).  Every CTA fetches its own:
//    no load writes to more than one CTA, since x may lie in memory that is not this GPU's (neighbouring row tiles that shared
//    their loads gained 1 to 2 %: grouped, 4096 tokens 252 -> 247 us; 2011 tokens with adapters 139 -> 136 us).
//  * Adapters are further columns of the same product: a tile's distinct adapters' B, side by side, times each token's
//    u = A x at its own adapter's place and zero elsewhere.
//  * Accumulators live in TMEM, two of them, so a tile's outputs are formed while the next one is
//    multiplied.
//  * Few tiles: a cluster splits the columns and joins its partial sums in a
//    fixed order through distributed shared memory.
//
// What bounds it.  Few tokens: the weights' bytes (1560 cycles a chunk and CTA at 6.8 TB/s) against about 1700
// cycles that a chunk takes through decode; 128 experts x 1536 x 2048 of which 40 slots choose 35 or so: 28 us for 118 MB.
// Many tokens: the round of barriers between the copies, the decode warps and the one thread that issues the products, about
// 2300 cycles a chunk, whatever the tile holds (192 tokens are 1536 cycles of products); so tiles are as large as TMEM lets
// them be.  4096 tokens, 8 of 128 experts, 1536 x 2048: 194 us, 1.06 PFLOP/s in this kernel.  f32: three
// products for one, 120 us at 131 tokens, 8 of 128 experts.
//
// Numbers.  A decoded weight is d q rounded to f16 (11 bits, where bf16 would keep 8), scaled by a power of two per
// matrix so that its largest weight is just below 1/2: what is smaller than 2^-13 of that is rounded to
// multiples of 2^-24 of 1, and its block's offset (-128 d or -8 d) as well.  (That range is what a decode with one multiply-add for
// two weights takes: the quant is a
// subnormal f16.)  Tokens of
// bf16 become f16 exactly, scaled by a power of two per token (what lies 2^-29 below a
// token's largest element is rounded to 2^-39 of it).  f32 tokens and weights are two
// f16 terms each (22 bits, weights scaled to just below 2^14) and three products; sums of 256 columns leave the
// tensor core, whose adds may truncate, and are added in fp32 to the running
// sum, with the two small products in an accumulator of their own.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <stddef.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "hq_internal.h"
#include "hq_tc.cuh"

namespace hq {
namespace {

// ------------------------------------------------------------------ shared with the host

constexpr int kTileRows = 128;
constexpr int kMaxTokens = 192;             // tokens of a tile: two accumulators and four operand slots are 512 columns
constexpr int kMaxTokensSplit = 48;         // f32: twice the operands
constexpr int kSlotCols = 32;               // TMEM columns of a decoded quarter (f32: of each term)
constexpr int kDecodeWarps = 16;
// Warps of a block: outputs (one or two for each quarter of the rows), decode, and one each for the weights' copies,
// the tokens' copies and the products.
template <bool SPLIT> struct Roles {
    static constexpr int kSides = SPLIT ? 1 : 2, kEpi = 4 * kSides, kW = kEpi + kDecodeWarps, kX = kW + 1, kMma = kX + 1;
    static constexpr int kThreads = 32 * (kMma + 1);
};
constexpr int kPrepThreads = 512;
constexpr int kMaxRaw = 4, kMaxX = 8;
constexpr int kBoxes = 5;                   // boxes of 16, 32, 64, 128 and tile_n tokens

template <int FMT> struct Fmt;
template <> struct Fmt<8> { static constexpr int kChunk = 272, kVecs = 5; };   // bytes of 8 blocks; 16-byte units a quarter touches
template <> struct Fmt<4> { static constexpr int kChunk = 144, kVecs = 3; };

// Virtual ranks of an adapter quarter: u is two bf16 terms (16 bits) of 32 ranks, or three (f32) of 16.
template <bool SPLIT> struct Ext { static constexpr int kRanks = SPLIT ? 16 : 32, kTerms = SPLIT ? 3 : 2; };

// One tile of tokens of one expert: sorted slots [start, start + n).
struct TileRec { int mat, start, n, w_exp; };

// What the kernel's warps keep in registers: they copy it, since what a pointer is taken from (the tensor maps) is read again
// after every inline statement, a constant-cache access each time.
struct Sizes {
    const int32_t *w_exp;
    const int32_t *x_exp;           // [sorted slots], or NULL: 0
    const int32_t *order;           // sorted slot -> slot, or NULL: the same
    const TileRec *tiles;           // or NULL: one matrix
    const int32_t *n_tiles;         // device count (grouped)
    // adapters: of each tile its distinct ones, of each token the place of its own among them (-1:
    // none, -2: an id out of range)
    const int32_t *tile_count, *tile_list, *place;
    const uint16_t *B;
    const float *u;                 // [n_tokens][rank]
    void *y;
    uint32_t *fault;
    long long rows;
    int n_tokens, n_tt, n_items, n_rt, n_chunks;
    int tile_n, raw_slots, x_slots, x_k, deep, ksplit, step, tmem_cols;    // x_slots slots of x_k (1, 2 or 4) times 64 columns of tokens
    int epilogue, rank, stream_w;
    int early;                      // one matrix's weights may be copied before the wait for the kernel before
    uint32_t off_raw, off_red;
};

struct TcArgs {
    CUtensorMap map_w, map_x[kBoxes], map_lo[kBoxes];
    Sizes z;
};

// A tile's columns: output slot, scale (a power of two; NaN for a bad adapter id), its exponent, the adapter's place; and the
// tile's adapters.
struct Columns {
    alignas(16) int slot[kMaxTokens];
    alignas(16) float scale[kMaxTokens];
    int list[kMaxTokens];
    int16_t e[kMaxTokens], place[kMaxTokens];
};

struct Meta {
    uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw], x_full[kMaxX], x_empty[kMaxX], full[4], empty[4];
    uint64_t acc_full[2], acc_empty[2], columns_full[2], red_full, red_empty, done;
    uint32_t tmem;
    // wide: number of the last (even, odd) item with a column whose scale is no float; odd: with an infinity or NaN in B
    int abort, wide[2], odd[2];
    Columns columns[2];             // of this item and the next
};

constexpr int kOffX = 7168;                 // shared memory: the barriers and a tile's columns, tokens, raw blocks, joined sums
static_assert(sizeof(Meta) <= kOffX && kOffX % 1024 == 0 && offsetof(Meta, columns) % 16 == 0, "the head of shared memory");

struct Item { int mat, rt, start, n, w_exp, count; };

// Work items, tiles of rows times tiles of tokens, in the order a CTA takes every step-th of.  Grouped: an expert's row
// tiles follow one another (inner), so that its weights are read again from L2 if it has several tiles of tokens; one
// matrix: a row tile's token tiles follow one another.
struct Cursor {
    int outer, inner;
    __device__ __forceinline__ void next(const Sizes &a, const Cursor &step) {
        const int count = a.tiles ? a.n_rt : a.n_tt;
        outer += step.outer;
        inner += step.inner;
        if (inner >= count) { inner -= count; ++outer; }
    }
};

__device__ __forceinline__ Cursor cursor_at(const Sizes &a, int w) {
    const int count = a.tiles ? a.n_rt : a.n_tt;
    return Cursor{w / count, w % count};
}

__device__ __forceinline__ Item get_item(const Sizes &a, const Cursor &c) {
    Item t;
    if (a.tiles) {
        const TileRec r = a.tiles[c.outer];
        t.rt = c.inner;
        t.mat = r.mat;
        t.start = r.start;
        t.n = r.n;
        t.w_exp = r.w_exp;
        t.count = 0;
    } else {
        t.mat = 0;
        t.rt = c.outer;
        t.start = c.inner * a.tile_n;
        t.n = min(a.tile_n, a.n_tokens - t.start);
        t.w_exp = *a.w_exp;
        t.count = a.tile_count ? a.tile_count[c.inner] : 0;
    }
    return t;
}

// Adapter quarters of a tile: this CTA's share of them.  They go through the pipeline as
// chunks of four; the last one may hold fewer.
template <bool SPLIT>
__device__ __forceinline__ int2 ext_range(const Sizes &a, const Item &t, int rank) {
    const int all = (t.count * a.rank + Ext<SPLIT>::kRanks - 1) / Ext<SPLIT>::kRanks;
    return make_int2(all * rank / a.ksplit, all * (rank + 1) / a.ksplit);
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// The box that fetches a tile of n tokens, and its rows.
__device__ __forceinline__ int box_of(const Sizes &a, int n) {
    const int b = n <= 16 ? 0 : n <= 32 ? 1 : n <= 64 ? 2 : n <= 128 ? 3 : 4;
    return a.tiles && 16 << b < a.tile_n ? b : kBoxes - 1;
}
__device__ __forceinline__ int box_rows(const Sizes &a, int b) { return b == kBoxes - 1 ? a.tile_n : 16 << b; }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// ------------------------------------------------------------------ decode

// A shared-memory load that stays before the barrier operations that follow it.
__device__ __forceinline__ void ld_shared_volatile(uint32_t addr, uint32_t *v) {
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// Block B (32 columns) of the two of one row's quarter, pairs of columns: `w` holds the 16-byte units that the quarter touches, block 0 begins at
// word I0.  The byte u = q + 128 (Q8_0) in the low bits of a half is the subnormal u 2^-24, and
// one multiply-add gives u 2^-24 (d 2^24) - 128 d, rounded once: both factors and the offset are exact.  Q4_0: the byte
// 16 n, n 2^-20 (d 2^20) - 8 d; d 2^24 or d 2^20 is then below 2^16 (d: scaled as the weights are).
// f32: the byte goes into the mantissa of 1024 instead, 1024 + bias is subtracted exactly, and the product with d is
// rounded to f16 and its rest, which a multiply-add gives exactly.
template <int FMT, bool SPLIT, int I0, int B>
__device__ __forceinline__ void decode_block(const uint32_t *w, float wscale, uint32_t (&hi)[16], uint32_t (&lo)[SPLIT ? 16 : 1]) {
    constexpr int kWords = FMT == 8 ? 8 : 4;
    const __half2 bias = FMT == 8 ? __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480))    // 1152
                                  : __half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));   // 1032
    const uint32_t dw = B == 0 ? w[I0] & 0xffffu : w[I0 + kWords] >> 16;
    const float df = __half2float(__ushort_as_half((unsigned short)dw)) * wscale;
    const __half2 d = __half2half2(__float2half_rn(SPLIT ? df : df * (FMT == 8 ? 16777216.f : 1048576.f)));
    const __half2 off = __half2half2(__float2half_rn(df * (FMT == 8 ? -128.f : -8.f)));
#pragma unroll
    for (int h = 0; h < 8; ++h) {                       // four columns
        const int j = FMT == 8 ? h : h & 3;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            // block 0 begins in the middle of a word, block 1 does not: a pair is the upper or the lower half of one
            uint32_t v = w[B == 0 ? I0 + j + p : I0 + kWords + 1 + j];
            if constexpr (FMT == 8) v ^= 0x80808080u;
            else if constexpr (SPLIT) v = (h < 4 ? v : v >> 4) & 0x0f0f0f0fu;
            else v = (h < 4 ? v << 4 : v) & 0xf0f0f0f0u;
            const uint32_t u = prmt(v, SPLIT ? 0x64646464u : 0u, (p == 0) == (B == 0) ? 0x4342u : 0x4140u);
            const __half2 n = *reinterpret_cast<const __half2 *>(&u);
            if constexpr (SPLIT) {
                const __half2 s = __hsub2(n, bias), r = __hmul2(s, d), l = __hfma2(s, d, __hneg2(r));
                hi[2 * h + p] = *reinterpret_cast<const uint32_t *>(&r);
                lo[2 * h + p] = *reinterpret_cast<const uint32_t *>(&l);
            } else {
                const __half2 r = __hfma2(n, d, off);
                hi[2 * h + p] = *reinterpret_cast<const uint32_t *>(&r);
            }
        }
    }
}

// The exponent that scales a matrix's decoded weights (see above), from the one kept beside it.
template <bool SPLIT> __device__ __forceinline__ int decode_exp(int w_exp) { return SPLIT ? w_exp : w_exp + 15; }

// ------------------------------------------------------------------ outputs

__device__ __forceinline__ void store_elem(void *y, long long i, int dtype, float v) {
    if (dtype == HQ_DT_F32) static_cast<float *>(y)[i] = v;
    else if (dtype == HQ_DT_F16) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

// z / (1 + e^-z).  fp32 outputs: the accurate power and the hardware's reciprocal (within an ulp), together within 2^-20 of it
// wherever e^-z is a float (z above -88.7; 0 below).  16-bit outputs: the approximate power as well, within
// 2^-21 (1 + |z| / 4) of it, 0 below z = -87.  (f32, 600 tokens, 8 of 128 experts, 1536 x 2048: 270 us, 258 us with that one.)
template <int OT>
__device__ __forceinline__ float silu(float z) {
    if constexpr (OT == HQ_DT_F32) {
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-z)));
        return z * r;
    } else {
        return __fdividef(z, 1.f + __expf(-z));
    }
}

template <int OT>
__device__ __forceinline__ void store_out(void *y, float v) {
    if constexpr (OT == HQ_DT_F32) *static_cast<float *>(y) = v;
    else if constexpr (OT == HQ_DT_F16) *static_cast<__half *>(y) = __float2half_rn(v);
    else *static_cast<__nv_bfloat16 *>(y) = __float2bfloat16_rn(v);
}

// The 8 columns from c0 of one output row (its sums in v): scales, SwiGLU with the neighbouring lane's row, store.
// `out` is the row's place in output row 0 and `pitch` the elements of an output row; `live`: the row exists.
template <int OT>
__device__ __forceinline__ void finish(const Columns *m, bool swiglu, bool wide, int c0, int n, bool live, char *out, uint32_t pitch, float (&v)[8]) {
    constexpr int kOut = OT == HQ_DT_F32 ? 4 : 2;
    const float4 *sp = reinterpret_cast<const float4 *>(m->scale + c0);
    const int4 *op = reinterpret_cast<const int4 *>(m->slot + c0);
    const float4 s0 = sp[0], s1 = sp[1];
    const int4 o0 = op[0], o1 = op[1];
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    const int slot[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s[j];
    if (wide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = m->e[c0 + j];
            v[j] *= pow2(e - max(-126, min(127, e)));
        }
    }
    if (swiglu) {
        // even lanes hold gate rows, odd lanes up rows: each finishes every other token
        const bool odd = threadIdx.x & 1;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const float h = silu<OT>(odd ? got : v[j]) * (odd ? v[j + 1] : got);
            if (live && c0 + j + (odd ? 1 : 0) < n) store_out<OT>(out + (uint64_t)(uint32_t)(odd ? slot[j + 1] : slot[j]) * pitch * kOut, h);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (live && c0 + j < n) store_out<OT>(out + (uint64_t)(uint32_t)slot[j] * pitch * kOut, v[j]);
}

// ------------------------------------------------------------------ adapter quarters

// The next bf16 terms of v0 and v1, which they lose.  Any but the last is kept finite: an infinity (or a finite value that rounds to
// one) would leave a NaN behind, while as the last term it stays what it is.
template <bool LAST>
__device__ __forceinline__ uint32_t take_term(float &v0, float &v1) {
    uint32_t h;
    if constexpr (LAST) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v1), "f"(v0));
    else asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v1), "f"(v0));
    v0 -= __uint_as_float(h << 16);
    v1 -= __uint_as_float(h & 0xffff0000u);
    return h;
}

// Virtual ranks [v0, v0 + kRanks) of one row of the tile's adapters' B, packed in pairs.
template <bool SPLIT>
__device__ __forceinline__ void load_b(const Sizes &a, const int *list, int total, int v0, long long row, uint32_t (&b)[16]) {
    constexpr int R = Ext<SPLIT>::kRanks;
    if ((a.rank & 7) == 0) {
#pragma unroll
        for (int k = 0; k < R; k += 8) {
            uint4 w = make_uint4(0, 0, 0, 0);
            const int v = v0 + k;
            if (v < total) {
                const uint16_t *p = a.B + ((long long)list[v / a.rank] * a.rows + row) * a.rank + v % a.rank;
                if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) w = *reinterpret_cast<const uint4 *>(p);
                else
                    w = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                                   p[6] | (uint32_t)p[7] << 16);
            }
            b[k / 2] = w.x; b[k / 2 + 1] = w.y; b[k / 2 + 2] = w.z; b[k / 2 + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < R; k += 2) {
            uint32_t w = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int v = v0 + k + h;
                if (v < total) w |= (uint32_t)a.B[((long long)list[v / a.rank] * a.rows + row) * a.rank + v % a.rank] << (16 * h);
            }
            b[k / 2] = w;
        }
    }
}

// In the product, an infinity or NaN of B would meet the zeros of other adapters' tokens and spoil them: its exponent loses a
// bit there (whether there was one), and add_odd_b adds what it stands for to its own adapter's tokens.
__device__ __forceinline__ bool take_odd_b(uint32_t (&b)[16]) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) any = __vmaxu2(any, b[i] & 0x7fff7fffu);
    if ((any & 0xffffu) < 0x7f80u && any >> 16 < 0x7f80u) return false;
    // an exponent of ones carries into the sign's place
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] &= ~((((b[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 1);
    return true;
}

// The terms of B's infinities and NaN to 8 columns of one output row, over this CTA's virtual ranks.
template <bool SPLIT>
__device__ __forceinline__ void add_odd_b(const Sizes &a, const Columns *m, const Item &t, int rank, long long row, int c0, float (&v)[8]) {
    const int2 ext = ext_range<SPLIT>(a, t, rank);
    const int lo = ext.x * Ext<SPLIT>::kRanks, hi = ext.y * Ext<SPLIT>::kRanks;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const int place = c0 + j < t.n ? m->place[c0 + j] : -1;
        float s = 0.f;
        if (place >= 0 && row < a.rows) {
            const uint16_t *b = a.B + ((long long)m->list[place] * a.rows + row) * a.rank;
            const float *u = a.u + (long long)(t.start + c0 + j) * a.rank;
#pragma unroll 1
            for (int k = max(0, lo - place * a.rank); k < min(a.rank, hi - place * a.rank); ++k) {
                const float f = __uint_as_float((uint32_t)b[k] << 16);
                if (!(fabsf(f) < INFINITY)) s += f * u[k];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += i == j ? s : 0.f;
    }
    __syncwarp();
}

// Row `c` of the token operand: u of the token's own adapter at its virtual ranks, as bf16 terms side by side, zero elsewhere.
template <bool SPLIT>
__device__ __forceinline__ void store_u(const Sizes &a, const Columns *m, const Item &t, int v0, int c, uint8_t *dst) {
    constexpr int R = Ext<SPLIT>::kRanks, T = Ext<SPLIT>::kTerms;
    const int place = c < t.n ? m->place[c] : -1;
    const int lo = place * a.rank - v0;                     // virtual rank v0 + k is rank k - lo of the adapter
    const bool any = place >= 0 && lo < R && lo + a.rank > 0;
    const int e = -m->e[c];
    const float s1 = pow2(e / 2), s2 = pow2(e - e / 2);
    uint8_t *line = dst + c * 128;
    const float *u = a.u + (long long)(t.start + c) * a.rank - lo;
    const bool four = ((a.rank | lo) & 3) == 0;
#pragma unroll
    for (int k0 = 0; k0 < R; k0 += 8) {
        float f[8];
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            const int k = k0 + h;
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
            if (any) {
                if (four) {
                    if (k >= lo && k < lo + a.rank) q = *reinterpret_cast<const float4 *>(u + k);
                } else {
                    if (k >= lo && k < lo + a.rank) q.x = u[k];
                    if (k + 1 >= lo && k + 1 < lo + a.rank) q.y = u[k + 1];
                    if (k + 2 >= lo && k + 2 < lo + a.rank) q.z = u[k + 2];
                    if (k + 3 >= lo && k + 3 < lo + a.rank) q.w = u[k + 3];
                }
            }
            f[h] = q.x * s1 * s2; f[h + 1] = q.y * s1 * s2; f[h + 2] = q.z * s1 * s2; f[h + 3] = q.w * s1 * s2;
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = i + 1 < T ? take_term<false>(f[2 * k], f[2 * k + 1]) : take_term<true>(f[2 * k], f[2 * k + 1]);
            *reinterpret_cast<uint4 *>(line + (((i * R + k0) / 8 ^ (c & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------ the kernel

// The products, as the head of the file describes and measures them; bound by the weights' bytes and their decode at few
// tokens, by the round of barriers of a chunk at many.  One CTA a multiprocessor, 27 warps (f32: 23) of fixed roles.
template <int FMT, bool SPLIT, int OT>
__global__ void __launch_bounds__(Roles<SPLIT>::kThreads, 1) matmul_tc_kernel(const __grid_constant__ TcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Meta *m = reinterpret_cast<Meta *>(smem);
    const Sizes z = a.z;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int kTerms = SPLIT ? 2 : 1, kSides = Roles<SPLIT>::kSides;
    constexpr int kEpiWarps = Roles<SPLIT>::kEpi, kWarpW = Roles<SPLIT>::kW, kWarpX = Roles<SPLIT>::kX, kWarpMma = Roles<SPLIT>::kMma;
    constexpr int kChunkBytes = kTileRows * Fmt<FMT>::kChunk;
    // a cluster shares an item's columns
    const int rank = z.ksplit > 1 ? (int)cluster_ctarank() : 0;
    const uint32_t x_base = smem_u32(smem) + kOffX, raw_base = smem_u32(smem) + z.off_raw;
    const uint32_t x_lo = z.x_k * z.tile_n * 128, x_slot = kTerms * x_lo;     // bytes to the low terms, of a slot
    volatile int *abort = &m->abort;
    uint32_t *fault = z.fault;

    // (after a time-out a list may be read that is not this tile's: whatever is there is an adapter)
    if (threadIdx.x < 2 * kMaxTokens) m->columns[threadIdx.x / kMaxTokens].list[threadIdx.x % kMaxTokens] = 0;
    if (threadIdx.x == 0) {
        m->abort = 0;
        for (int i = 0; i < z.raw_slots; ++i) { mbar_init(smem_u32(&m->raw_full[i]), 1); mbar_init(smem_u32(&m->raw_empty[i]), kDecodeWarps); }
        for (int i = 0; i < z.x_slots; ++i) { mbar_init(smem_u32(&m->x_full[i]), 1); mbar_init(smem_u32(&m->x_empty[i]), 1); }
        for (int i = 0; i < 4; ++i) { mbar_init(smem_u32(&m->full[i]), z.deep ? kDecodeWarps : 4); mbar_init(smem_u32(&m->empty[i]), 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&m->acc_full[i]), 1); mbar_init(smem_u32(&m->acc_empty[i]), kEpiWarps); }
        m->wide[0] = m->wide[1] = m->odd[0] = m->odd[1] = 0;
        mbar_init(smem_u32(&m->done), 1);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&m->columns_full[i]), kEpiWarps);
        mbar_init(smem_u32(&m->red_full), (uint32_t)max(1, (z.ksplit - 1) * kEpiWarps));
        mbar_init(smem_u32(&m->red_empty), (uint32_t)max(1, (z.ksplit - 1) * kEpiWarps));
        fence_mbar_init();
    }
    if (warp == kWarpMma) tmem_alloc(smem_u32(&m->tmem), (uint32_t)z.tmem_cols);
    tc_fence_before();
    if (z.ksplit > 1) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&m->tmem;
    // TMEM: two buffers of accumulators, (f32) the running sums, then the operand slots
    const uint32_t half = (SPLIT ? 2 : 1) * z.tile_n, run = 2 * half, slots = run + (SPLIT ? z.tile_n : 0);
    griddep_launch_dependents();

    const int first = (int)cluster_id(), step = z.step;
    const int c_lo = (int)((long long)z.n_chunks * rank / z.ksplit);
    const int c_hi = (int)((long long)z.n_chunks * (rank + 1) / z.ksplit);
    const Cursor stride = cursor_at(z, step);
    Cursor at = cursor_at(z, min(first, z.n_items - 1));
    // One matrix's weights may be fetched before the prepare kernel is done, since that lets this one start only after its own
    // wait for whatever comes before it in the stream, which may have written them.  Everything else waits for the prepare
    // kernel, and where there is none (f16 without adapters) so do the weights.
    if (!z.early || warp != kWarpW) griddep_wait();
    Item t = {};
    if (z.tiles || warp != kWarpW) t = get_item(z, at);
    const int n_items = z.tiles ? *z.n_tiles * z.n_rt : z.n_items;

    if (warp == kWarpW) {
        if (elect_one()) {
            const uint64_t pol = z.stream_w ? l2_evict_first_policy() : l2_evict_normal_policy();
            uint32_t s = 0, ph = 1, it = 0;
            bool ok = true;
            for (int w = first; w < n_items && ok; w += step) {
                const int row0 = z.tiles ? (int)((long long)t.mat * z.rows + (long long)t.rt * kTileRows) : at.outer * kTileRows;
                at.next(z, stride);
                if (z.tiles && w + step < n_items) t = get_item(z, at);
                for (int c = c_lo; c < c_hi; ++c, ++it) {
                    // past the first slots the wait is for this kernel's own warps, which wait for the prepare kernel
                    if (z.early && it == (uint32_t)z.raw_slots) griddep_wait();
                    ok = tc_wait(smem_u32(&m->raw_empty[s]), ph, abort, fault);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&m->raw_full[s]);
                    mbar_arrive_expect_tx(bar, kChunkBytes);
                    tma_load_2d(raw_base + s * kChunkBytes, &a.map_w, c * (Fmt<FMT>::kChunk / 2), row0, bar, pol);
                    if (++s == (uint32_t)z.raw_slots) { s = 0; ph ^= 1; }
                }
            }
            // copies in flight end before the block's memory is given back
            for (uint32_t k = it > (uint32_t)z.raw_slots ? it - z.raw_slots : 0; !ok && k < it; ++k)
                for (int tries = 0; tries < 1 << 8 && !mbar_try_wait(smem_u32(&m->raw_full[k % z.raw_slots]), (k / z.raw_slots) & 1); ++tries) {}
        }
        __syncwarp();
    } else if (warp == kWarpX) {
        if (elect_one()) {
            const uint64_t pol = l2_evict_normal_policy();
            uint32_t it = 0, s = 0, ph = 1;
            bool ok = true, free = false;                   // free: the next slot is known to be
            for (int w = first; w < n_items && ok; w += step) {
                const Item cur = t;
                at.next(z, stride);
                if (w + step < n_items) t = get_item(z, at);
                const int box = box_of(z, cur.n);
                const int2 ext = ext_range<SPLIT>(z, cur, rank);
                const uint32_t bytes = kTerms * z.x_k * box_rows(z, box) * 128;
                // the adapter chunks come first
#pragma unroll 1
                for (int k = 4 * (c_lo - (ext.y - ext.x + 3) / 4); k < 4 * c_hi; k += z.x_k, ++it) {
                    const uint32_t bar = smem_u32(&m->x_full[s]), dst = x_base + s * x_slot;
                    ok = free || tc_wait(smem_u32(&m->x_empty[s]), ph, abort, fault);
                    if (!ok) break;
                    if (++s == (uint32_t)z.x_slots) { s = 0; ph ^= 1; }
                    free = tc_test(smem_u32(&m->x_empty[s]), ph);
                    if (k >= 4 * c_lo) {
                        mbar_arrive_expect_tx(bar, bytes);
                        tma_load_3d(dst, &a.map_x[box], 0, cur.start, k, bar, pol);
                        if constexpr (SPLIT) tma_load_3d(dst + x_lo, &a.map_lo[box], 0, cur.start, k, bar, pol);
                    } else {
                        mbar_arrive(bar);                   // the decode warps fill an adapter chunk
                    }
                }
            }
            // copies in flight end before the block's memory is given back
            for (uint32_t k = it > (uint32_t)z.x_slots ? it - z.x_slots : 0; !ok && k < it; ++k)
                for (int tries = 0; tries < 1 << 8 && !mbar_try_wait(smem_u32(&m->x_full[k % z.x_slots]), (k / z.x_slots) & 1); ++tries) {}
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        if (elect_one()) {
            // chunk number, token slot and its parity, number of the accumulator
            uint32_t it = 0, xs = 0, xp = 0, acc = 0;
            const uint64_t desc_x = tc_desc_sw128(x_base);
            const uint32_t x_units = x_slot >> 4, lo_units = x_lo >> 4;
            // the products of one quarter: 64 columns of weights, or the terms of u times an adapter quarter
            auto quarter = [&](uint32_t d, uint32_t ta, uint64_t db, uint32_t idesc, bool add) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    tc_mma(d, ta + 8 * j, db + 2 * j, idesc, add || j);
                    if constexpr (SPLIT) {
                        tc_mma(d + z.tile_n, ta + 8 * j, db + lo_units + 2 * j, idesc, add || j);
                        tc_mma(d + z.tile_n, ta + kSlotCols + 8 * j, db + 2 * j, idesc, true);
                    }
                }
            };
            auto next_x = [&]() {
                tc_commit(smem_u32(&m->x_empty[xs]));
                if (++xs == (uint32_t)z.x_slots) { xs = 0; xp ^= 1; }
            };
            // A wait costs hundreds of cycles even if there is nothing to wait for (the question queues behind the other
            // warps' shared-memory accesses): the next stage's barriers are asked about before this one's products are
            // issued, and waited for only if the answer was no.
            bool x_ready = false, w_ready = false;
            auto wait_x = [&]() {
                tc_wait_go(x_ready, smem_u32(&m->x_full[xs]), xp, abort, fault);
                x_ready = false;
            };
            auto wait_w = [&](uint32_t bar, uint32_t par) {
                tc_wait_go(w_ready, smem_u32(&m->full[bar]), par, abort, fault);
                w_ready = false;
            };
            auto ask_x = [&]() {
                const bool wrap = xs + 1 == (uint32_t)z.x_slots;
                x_ready = tc_test(smem_u32(&m->x_full[wrap ? 0 : xs + 1]), xp ^ (wrap ? 1u : 0u));
            };
            auto ask_w = [&](uint32_t bar, uint32_t par) { w_ready = tc_test(smem_u32(&m->full[bar]), par); };
            for (int w = first; w < n_items && !*abort; w += step) {
                const Item cur = t;
                at.next(z, stride);
                if (w + step < n_items) t = get_item(z, at);
                const int n16 = round16(cur.n);
                const uint32_t idesc = tc_idesc(n16, false);
                const uint32_t kb_step = (uint32_t)(box_rows(z, box_of(z, cur.n)) * 128) >> 4;
                const int2 ext = ext_range<SPLIT>(z, cur, rank);
                bool add = false;                           // to the accumulator, or start it
                // adapter chunks, ahead of the weights' (which are on their way meanwhile)
                if (ext.x < ext.y) {
                    tc_wait_go(false, smem_u32(&m->acc_empty[acc & 1]), ((acc >> 1) & 1) ^ 1, abort, fault);
                    const uint32_t d = tmem + (acc & 1) * half, idesc_b = tc_idesc(n16, true);
                    for (int e = ext.x; e < ext.y; e += 4, ++it) {
                        const uint32_t buf = z.deep ? it & 1 : 0, par = z.deep ? (it >> 1) & 1 : it & 1;
                        uint32_t ta = tmem + slots + buf * 4 * kSlotCols;
                        uint64_t db = 0;
#pragma unroll 1
                        for (int q = 0; q < 4; ++q, ta += kTerms * kSlotCols, db += kb_step) {
                            if ((q & (z.x_k - 1)) == 0) {
                                wait_x();
                                db = desc_x + (uint64_t)(xs * x_units);
                            }
                            if (!z.deep || q == 0) wait_w(buf + q, par);
                            tc_fence_after();
                            if (e + q < ext.y) {
                                // the terms of u times the same columns of B
                                constexpr int kPer = Ext<SPLIT>::kRanks / 16;
#pragma unroll
                                for (int j = 0; j < kPer * Ext<SPLIT>::kTerms; ++j)
                                    tc_mma(d, ta + 8 * (j % kPer), db + 2 * j, idesc_b, add || j);
                                add = true;
                            }
                            if (!z.deep || q == 3) tc_commit(smem_u32(&m->empty[z.deep ? buf : q]));
                            if ((q & (z.x_k - 1)) == z.x_k - 1) next_x();
                        }
                    }
                    if (SPLIT) {                            // an accumulator of their own: they have no small products
                        tc_commit(smem_u32(&m->acc_full[acc & 1]));
                        ++acc;
                        add = false;
                    }
                }
                for (int c = c_lo; c < c_hi; ++c, ++it) {
                    if (!add) tc_wait_go(false, smem_u32(&m->acc_empty[acc & 1]), ((acc >> 1) & 1) ^ 1, abort, fault);
                    const uint32_t d = tmem + (acc & 1) * half;
                    if (z.deep) {
                        // two buffers of four quarters, a barrier each; the chunk's tokens are one to four stages
                        const uint32_t buf = it & 1, ta = tmem + slots + buf * 4 * kSlotCols;
                        wait_w(buf, (it >> 1) & 1);
                        wait_x();
                        tc_fence_after();
                        ask_x();
                        ask_w(buf ^ 1, ((it + 1) >> 1) & 1);
                        uint64_t db = desc_x + (uint64_t)(xs * x_units);
                        quarter(d, ta, db, idesc, add);
#pragma unroll
                        for (int q = 1; q < 4; ++q) {
                            if ((q & (z.x_k - 1)) == 0) {
                                next_x();
                                wait_x();
                                ask_x();
                                db = desc_x + (uint64_t)(xs * x_units);
                            } else {
                                db += kb_step;
                            }
                            quarter(d, ta + q * kSlotCols, db, idesc, true);
                        }
                        tc_commit(smem_u32(&m->empty[buf]));
                        next_x();
                    } else {
                        // one buffer, a barrier a quarter
                        uint64_t db = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if ((q & (z.x_k - 1)) == 0) {
                                wait_x();
                                db = desc_x + (uint64_t)(xs * x_units);
                            } else {
                                db += kb_step;
                            }
                            wait_w(q, it & 1);
                            tc_fence_after();
                            if ((q & (z.x_k - 1)) == z.x_k - 1) ask_x();
                            ask_w((q + 1) & 3, (it + (q == 3 ? 1 : 0)) & 1);
                            quarter(d, tmem + slots + q * kTerms * kSlotCols, db, idesc, add || q);
                            tc_commit(smem_u32(&m->empty[q]));
                            if ((q & (z.x_k - 1)) == z.x_k - 1) next_x();
                        }
                    }
                    add = true;
                    if (SPLIT || c + 1 == c_hi) {
                        tc_commit(smem_u32(&m->acc_full[acc & 1]));
                        ++acc;
                        add = false;
                    }
                }
            }
            // every product ends before TMEM is given back
            tc_commit(smem_u32(&m->done));
            for (int tries = 0; tries < 1 << 20 && !mbar_try_wait(smem_u32(&m->done), 0); ++tries) {}
        }
        __syncwarp();
    } else if (warp >= kEpiWarps) {
        const int g = (warp - kEpiWarps) >> 2, row = (warp & 3) * 32 + lane;
        constexpr int kUnit = FMT == 8 ? 64 : 32;           // quarter q begins within the 16-byte unit at q * kUnit bytes
        const uint32_t src = raw_base + row * Fmt<FMT>::kChunk;
        const uint32_t lane_base = tmem + slots + ((uint32_t)((warp & 3) * 32) << 16);
        // raw slot and its parity, chunk number, item number
        uint32_t s = 0, ph = 0, it = 0, item = ~0u;
        uint32_t v[4 * Fmt<FMT>::kVecs];                    // words 0 to 4 kVecs - 1, of which quarter g begins at g
        auto fetch = [&]() {
#pragma unroll
            for (int i = 0; i < Fmt<FMT>::kVecs; ++i)
                ld_shared_volatile(src + s * kChunkBytes + g * kUnit + 16 * i, v + 4 * i);
        };
        if (first < n_items) {
            tc_wait_go(false, smem_u32(&m->raw_full[0]), 0, abort, fault);
            fetch();
        }
        for (int w = first; w < n_items && !__any_sync(0xffffffffu, *abort); w += step) {
            ++item;
            const Item cur = t;
            at.next(z, stride);
            if (w + step < n_items) t = get_item(z, at);
            if (cur.count) {
                // adapter chunks: group g has their quarter g
                const int2 ext = ext_range<SPLIT>(z, cur, rank);
                if (!__all_sync(0xffffffffu, tc_wait(smem_u32(&m->columns_full[item & 1]), (item >> 1) & 1, abort, fault))) break;
                const int total = cur.count * z.rank;
                const long long r = min((long long)cur.rt * kTileRows + row, z.rows - 1);
                for (int e = ext.x + g; e < (ext.y - ext.x + 3) / 4 * 4 + ext.x; e += 4, ++it) {
                    const uint32_t bar = z.deep ? it & 1 : g, par = z.deep ? (it >> 1) & 1 : it & 1;
                    const uint32_t dst = lane_base + (z.deep ? (it & 1) * 4 * kSlotCols : 0) + g * kTerms * kSlotCols;
                    uint32_t b[16] = {};
                    if (e < ext.y) {
                        load_b<SPLIT>(z, m->columns[item & 1].list, total, e * Ext<SPLIT>::kRanks, r, b);
                        if (take_odd_b(b)) *(volatile int *)&m->odd[item & 1] = (int)item + 1;
                    }
                    // the token stage that quarter g of this chunk falls on
                    const uint32_t xi = (it * 4 + g) / z.x_k, sx = xi % z.x_slots;
                    tc_wait_go(false, smem_u32(&m->empty[bar]), par ^ 1, abort, fault);
                    tc_wait_go(false, smem_u32(&m->x_empty[sx]), ((xi / z.x_slots) & 1) ^ 1, abort, fault);
                    __syncwarp();
                    tc_fence_after();
                    if (e < ext.y) {
                        tmem_st16(dst, b);
                        uint8_t *x = smem + kOffX + sx * x_slot + (g & (z.x_k - 1)) * z.tile_n * 128;
                        for (int c = row; c < round16(cur.n); c += kTileRows) store_u<SPLIT>(z, &m->columns[item & 1], cur, e * Ext<SPLIT>::kRanks, c, x);
                        fence_proxy_async_shared();
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m->full[bar]));
                }
            }
            const float wscale = pow2(-decode_exp<SPLIT>(cur.w_exp));
            for (int c = c_lo; c < c_hi; ++c, ++it) {
                const bool more = c + 1 < c_hi || w + step < n_items;
                const uint32_t bar = z.deep ? it & 1 : g, par = z.deep ? (it >> 1) & 1 : it & 1, here = s;
                const uint32_t dst = lane_base + (z.deep ? (it & 1) * 4 * kSlotCols : 0) + g * kTerms * kSlotCols;
                if (++s == (uint32_t)z.raw_slots) { s = 0; ph ^= 1; }
                // asked about now, while this quarter is decoded: the slot it goes to and the next raw chunk
                const bool free = tc_test(smem_u32(&m->empty[bar]), par ^ 1), ready = tc_test(smem_u32(&m->raw_full[s]), ph);
                auto decode = [&](auto block, uint32_t (&hi)[16], uint32_t (&lo)[SPLIT ? 16 : 1]) {
                    constexpr int B = decltype(block)::value;
                    if (g == 0) decode_block<FMT, SPLIT, 0, B>(v, wscale, hi, lo);
                    else if (g == 1) decode_block<FMT, SPLIT, 1, B>(v, wscale, hi, lo);
                    else if (g == 2) decode_block<FMT, SPLIT, 2, B>(v, wscale, hi, lo);
                    else decode_block<FMT, SPLIT, 3, B>(v, wscale, hi, lo);
                };
                // (f32: half of it ahead, for the registers)
                uint32_t hi[16], lo[SPLIT ? 16 : 1], rest[16];
                decode(std::integral_constant<int, 0>(), hi, lo);
                if constexpr (!SPLIT) decode(std::integral_constant<int, 1>(), rest, lo);
                tc_wait_go(free, smem_u32(&m->empty[bar]), par ^ 1, abort, fault);
                __syncwarp();
                tc_fence_after();
                const bool early = __all_sync(0xffffffffu, ready) && more;
                tmem_st16(dst, hi);
                if constexpr (SPLIT) {
                    tmem_st16(dst + kSlotCols, lo);
                    decode(std::integral_constant<int, 1>(), rest, lo);
                    tmem_st16(dst + kSlotCols + 16, lo);
                }
                tmem_st16(dst + 16, rest);
                if (early) fetch();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                // Only now, with every value decoded, does the raw buffer go back to the copy engine: an arrival does
                // not wait for loads in flight, and overtakes them when the load unit is busy.
                if (lane == 0) {
                    mbar_arrive(smem_u32(&m->full[bar]));
                    mbar_arrive(smem_u32(&m->raw_empty[here]));
                }
                if (more && !early) {
                    tc_wait_go(false, smem_u32(&m->raw_full[s]), ph, abort, fault);
                    fetch();
                }
            }
        }
    } else {
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int side = warp >> 2;                         // of the two warps of these rows
        float *red = reinterpret_cast<float *>(smem + z.off_red);
        const uint32_t red_addr = smem_u32(red);
        const int my_row = (warp & 3) * 32 + lane;
        constexpr int kOut = OT == HQ_DT_F32 ? 4 : 2;
        const bool swiglu = z.epilogue == HQ_MOE_EPI_SWIGLU;
        const uint32_t pitch = (uint32_t)(swiglu ? z.rows / 2 : z.rows);
        uint32_t acc = 0, item = 0;
        bool ok = true;
        // An item's columns, a thread each: loaded a whole item before they are stored, and its tile an item before that.
        struct Column { int slot, e, place, list; } col = {};
        auto load = [&](const Item &c) {
            const int k = c.start + min((int)threadIdx.x, c.n - 1);
            if (threadIdx.x >= round16(c.n)) return;
            col.e = decode_exp<SPLIT>(c.w_exp) + (z.x_exp ? z.x_exp[k] : 0);
            col.place = z.place ? z.place[k] : -1;
            col.slot = z.order ? z.order[k] : k;
            if (threadIdx.x < c.count) col.list = z.tile_list[c.start + threadIdx.x];
        };
        // To where the decode warps and, after the next named barrier, these warps read them.
        auto store = [&](const Item &c, uint32_t i) {
            Columns *to = &m->columns[i & 1];
            const int j = threadIdx.x, near = max(-126, min(127, col.e));
            if (j < round16(c.n)) {
                to->slot[j] = col.slot;
                to->scale[j] = col.place == -2 ? __int_as_float(0x7fc00000) : pow2(near);
                to->e[j] = (int16_t)col.e;
                to->place[j] = (int16_t)col.place;
                if (col.e != near) m->wide[i & 1] = (int)i + 1;
                if (j < c.count) to->list[j] = col.list;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&m->columns_full[i & 1]));
        };
        Item next_t = {}, after = {};
        if (first < n_items) {
            load(t);
            store(t, 0);
        }
        auto ahead = [&](int w) -> Item {                   // the item after the cursor's, if it is one
            at.next(z, stride);
            return w < n_items ? get_item(z, at) : Item{};
        };
        next_t = ahead(first + step);
        if (first + step < n_items) load(next_t);
        after = ahead(first + 2 * step);
        for (int w = first; w < n_items; w += step, ++item) {
            // the warps leave together, the last tile's columns are read and this one's stored
            if (!named_barrier_and(1, 32 * kEpiWarps, ok)) break;
            const Item cur = t;
            const bool wide = *(volatile int *)&m->wide[item & 1] == (int)item + 1;
            t = next_t;
            if (w + step < n_items) store(t, item + 1);
            next_t = after;
            if (w + 2 * step < n_items) load(next_t);
            after = ahead(w + 3 * step);
            const int n8 = round16(cur.n) / 8;
            const long long row = (long long)cur.rt * kTileRows + my_row;
            char *out = static_cast<char *>(z.y) + (swiglu ? row / 2 : row) * kOut;
            const int ks = z.ksplit;
            uint32_t base = lane_base + run;                // where the tile's sums are
            if constexpr (SPLIT) {
                // Each chunk's sums (and the adapters') leave the accumulator for the running sums.
                const int2 ext = ext_range<SPLIT>(z, cur, rank);
                const int own = ext.x < ext.y ? 1 : 0, rounds = c_hi - c_lo + own;    // the adapters' round is the first
                for (int i = 0; i < rounds; ++i, ++acc) {
                    ok = __all_sync(0xffffffffu, tc_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t from = lane_base + (acc & 1) * half;
#pragma unroll 1
                    for (int g = side; g < n8; g += kSides) {
                        float v[8], x[8], r[8];
                        tmem_ld8(from + 8 * g, v);
                        // (loaded whether they count or not: registers on their way may not be moved, as where branches join)
                        tmem_ld8(from + z.tile_n + 8 * g, x);       // the small products
                        tmem_ld8(base + 8 * g, r);
                        tmem_wait_ld(v);
                        tmem_wait_ld(x);
                        tmem_wait_ld(r);
                        if (i >= own) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] += x[j];
                        }
                        if (i > 0) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] += r[j];
                        }
                        tmem_st8(base + 8 * g, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m->acc_empty[acc & 1]));
                }
                if (!ok) continue;
            } else {
                ok = __all_sync(0xffffffffu, tc_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault));
                if (!ok) continue;
                tc_fence_after();
                base = lane_base + (acc & 1) * half;
            }
            if (*(volatile int *)&m->odd[item & 1] == (int)item + 1) {
#pragma unroll 1
                for (int g = side; g < n8; g += kSides) {
                    float v[8];
                    tmem_ld8(base + 8 * g, v);
                    tmem_wait_ld(v);
                    add_odd_b<SPLIT>(z, &m->columns[item & 1], cur, rank, row, 8 * g, v);
                    tmem_st8(base + 8 * g, v);
                }
                tmem_wait_st();
            }
            if (ks == 1) {
                // 8 columns at a time, the next ones (at the end, these again) on their way meanwhile
                float v[8], next[8];
                tmem_ld8(base + 8 * side, next);
                tmem_wait_ld(next);
#pragma unroll 1
                for (int g = side; g < n8; g += kSides) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = next[j];
                    tmem_ld8(base + 8 * (g + kSides < n8 ? g + kSides : g), next);
                    finish<OT>(&m->columns[item & 1], swiglu, wide, 8 * g, cur.n, row < z.rows, out, pitch, v);
                    tmem_wait_ld(next);
                }
            } else {
                // group g of 8 columns is finished by rank (g / 2) % ks, which receives the other ranks' sums
                const int per = (z.tile_n / 16 + ks - 1) / ks * 2;
                if (item > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&m->red_empty), (item - 1) & 1, abort, fault));
                    if (!ok) continue;
                }
#pragma unroll 1
                for (int g = side; g < n8; g += kSides) {
                    const int to = (g >> 1) % ks;
                    if (to == rank) continue;
                    float v[8];
                    tmem_ld8(base + 8 * g, v);
                    tmem_wait_ld(v);
                    const int from = rank - (rank > to ? 1 : 0), at = (g >> 1) / ks * 2 + (g & 1);
                    const uint32_t dst = map_shared_rank(red_addr + (uint32_t)(((from * per + at) * 8 * kTileRows + my_row) * 4), (uint32_t)to);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_cluster_f32(dst + j * (kTileRows * 4), v[j]);
                }
                __syncwarp();
                if (lane < ks && lane != rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_full), (uint32_t)lane));
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&m->red_full), item & 1, abort, fault));
                if (!ok) continue;
#pragma unroll 1
                for (int g = side; g < n8; g += kSides) {
                    if ((g >> 1) % ks != rank) continue;
                    float v[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    tmem_ld8(base + 8 * g, v);
                    tmem_wait_ld(v);
                    const int at = (g >> 1) / ks * 2 + (g & 1);
#pragma unroll 1
                    for (int r = 0; r < ks; ++r) {
                        if (r == rank) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] += v[j];
                        } else {
                            const float *src = red + ((r - (r > rank ? 1 : 0)) * per + at) * 8 * kTileRows + my_row;
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] += src[j * kTileRows];
                        }
                    }
                    finish<OT>(&m->columns[item & 1], swiglu, wide, 8 * g, cur.n, row < z.rows, out, pitch, o);
                }
                __syncwarp();
                if (lane < ks && lane != rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_empty), (uint32_t)lane));
            }
            if constexpr (!SPLIT) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&m->acc_empty[acc & 1]));
                ++acc;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (z.ksplit > 1) cluster_sync();
    if (warp == kWarpMma) tmem_dealloc(tmem, (uint32_t)z.tmem_cols);
}

// ------------------------------------------------------------------ prepare

constexpr int kWindow = 128;            // tokens whose adapters are looked at together
constexpr int kSelfPlan = 1024;         // slots up to which every block finds its own places (one launch less)

struct PrepArgs {
    const void *x;
    int dtype;
    long long cols;
    int x_rows, copies;             // each row of x goes to `copies` slots
    __half *hi, *lo;                // lo: f32 only
    int32_t *x_exp;                 // NULL for f16: copied as it is
    int row_threads, pack_blocks;
    // grouping
    const int32_t *ids;
    const int32_t *w_exp;
    int n_slots, n_mats, tile_n, plan_blocks;
    int32_t *order, *pos, *n_tiles; // pos[slot]: its sorted place (plan kernel), or NULL: found here
    TileRec *tiles;
    void *y;                        // rows of slots whose id is out of range get NaN
    long long y_cols;
    int y_dtype;
    // adapters
    const int32_t *adapter_ids;
    const uint16_t *A;
    const float *scales;
    long long n_adapters;
    int n_tokens, rank, list_blocks, down_tokens, down_turns, down_split;
    int32_t *tile_count, *tile_list, *place;
    float *u;
    uint32_t *fault;
};

// Sum of `v` over the threads before this one, and over all of them.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int *red, int *all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    const int part = lane < THREADS / 32 ? red[lane] : 0;
    int sum = part;
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    *all = __shfl_sync(0xffffffffu, sum, 31);
    return __shfl_sync(0xffffffffu, sum - part, warp) + inc - v;
}

// Counts the experts' slots, cuts each expert's slots into tiles of tokens, and (PLACE) gives every slot its
// place.  The order within an expert is whatever the counters give; an output does not depend on it.  A cluster shares the
// slots: each block counts its own, and reads the others' counts.
template <int THREADS, bool PLACE>
__device__ void plan_slots(const PrepArgs &a, int *count, int blocks, int rank) {
    __shared__ int red[32];
    constexpr int U = 4;                                    // loads in flight
    const int lo = (int)((long long)a.n_slots * rank / blocks), hi = (int)((long long)a.n_slots * (rank + 1) / blocks);
    for (int e = threadIdx.x; e < a.n_mats; e += THREADS) count[e] = 0;
    __syncthreads();
    for (int s0 = lo; s0 < hi; s0 += U * THREADS) {
        int e[U];
#pragma unroll
        for (int i = 0; i < U; ++i) { const int s = s0 + i * THREADS + threadIdx.x; e[i] = s < hi ? a.ids[s] : -1; }
#pragma unroll
        for (int i = 0; i < U; ++i) if (e[i] >= 0 && e[i] < a.n_mats) atomicAdd(&count[e[i]], 1);
    }
    if (blocks > 1) cluster_sync(); else __syncthreads();
    int base_n = 0, base_t = 0;
    int *first = count + a.n_mats;                          // places of this block's slots (the counts are still read by others)
    for (int e0 = 0; e0 < a.n_mats; e0 += THREADS) {
        const int e = e0 + threadIdx.x;
        int n = 0, before = 0;
        if (e < a.n_mats) {
            if (blocks == 1) n = count[e];
            else
                for (int r = 0; r < blocks; ++r) {
                    const int c = ld_shared_cluster_s32(map_shared_rank(smem_u32(&count[e]), (uint32_t)r));
                    n += c;
                    before += r < rank ? c : 0;
                }
        }
        int size = 0, nt = 0;
        if (n) {
            nt = (n + a.tile_n - 1) / a.tile_n;
            size = round16((n + nt - 1) / nt);
            nt = (n + size - 1) / size;
        }
        int all_n, all_t;
        const int at = base_n + block_scan<THREADS>(n, red, &all_n);
        const int tile = base_t + block_scan<THREADS>(nt, red, &all_t);
        if (rank == 0) {
            const int we = n ? a.w_exp[e] : 0;
            for (int i = 0; i < nt; ++i) a.tiles[tile + i] = TileRec{e, at + i * size, min(size, n - i * size), we};
        }
        if (PLACE && e < a.n_mats) first[e] = at + before;
        base_n += all_n;
        base_t += all_t;
    }
    if (rank == 0 && threadIdx.x == 0) *a.n_tiles = base_t;
    if constexpr (PLACE) {
        __syncthreads();
        for (int s0 = lo; s0 < hi; s0 += U * THREADS) {
            int e[U];
#pragma unroll
            for (int i = 0; i < U; ++i) { const int s = s0 + i * THREADS + threadIdx.x; e[i] = s < hi ? a.ids[s] : -1; }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool ok = e[i] >= 0 && e[i] < a.n_mats;
                const int at = ok ? atomicAdd(&first[e[i]], 1) : -1, s = s0 + i * THREADS + threadIdx.x;
                if (s < hi) {
                    a.pos[s] = at;
                    if (ok) a.order[at] = s;
                    else atomicOr(a.fault, kFaultExpertId);
                }
            }
        }
    }
    if (blocks > 1) cluster_sync();
}

// One block or a cluster of eight, bound by its chain of counter updates: 8 us at 4136 slots, 9 us at 32768.
__global__ void __launch_bounds__(1024) plan_kernel(PrepArgs a) {
    extern __shared__ int count[];                          // [2][n_mats]
    griddep_launch_dependents();
    griddep_wait();
    plan_slots<1024, true>(a, count, (int)gridDim.x, gridDim.x > 1 ? (int)cluster_ctarank() : 0);
}

// max over the row_threads threads of a row (a power of two of at least a warp); every thread of the block takes part
__device__ __forceinline__ float row_max(float v, int row_threads, float *red) {
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    if (row_threads == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int w0 = threadIdx.x / row_threads * (row_threads / 32);
    for (int w = 0; w < row_threads / 32; ++w) v = fmaxf(v, red[w0 + w]);
    return v;
}

__device__ __forceinline__ int row_sum(int v, int row_threads, int *red) {
    v = __reduce_add_sync(0xffffffffu, v);
    if (row_threads == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int w0 = threadIdx.x / row_threads * (row_threads / 32);
    int s = 0;
    for (int w = 0; w < row_threads / 32; ++w) s += red[w0 + w];
    return s;
}

// 8 elements from their bytes.
template <int DT>
__device__ __forceinline__ void unpack8(const uint4 *w, float (&v)[8]) {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    if constexpr (DT == HQ_DT_F32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(u[k]);
        v[4] = __uint_as_float(w[1].x); v[5] = __uint_as_float(w[1].y); v[6] = __uint_as_float(w[1].z); v[7] = __uint_as_float(w[1].w);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (DT == HQ_DT_BF16) {
                v[2 * k] = __uint_as_float(u[k] << 16);
                v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[k]));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            }
        }
    }
}

__device__ __forceinline__ void load8x(const void *x, long long i, int dtype, float (&v)[8]) {
    if (dtype == HQ_DT_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + i), w[2] = {p[0], p[1]};
        unpack8<HQ_DT_F32>(w, v);
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
        if (dtype == HQ_DT_BF16) unpack8<HQ_DT_BF16>(&w, v); else unpack8<HQ_DT_F16>(&w, v);
    }
}

// Rows of x to f16 terms at their slots' places, each row scaled so that its largest
// finite element lies in [2^13, 2^14).
__device__ void pack_rows(const PrepArgs &a, int block) {
    __shared__ float red[kPrepThreads / 32];
    __shared__ int redi[kPrepThreads / 32];
    const int per = kPrepThreads / a.row_threads, tr = threadIdx.x % a.row_threads;
    for (int r0 = block * per; r0 < a.x_rows; r0 += a.pack_blocks * per) {
        const int r = r0 + threadIdx.x / a.row_threads;
        const bool live = r < a.x_rows;
        const long long base = (long long)r * a.cols;
        float s1 = 1.f, s2 = 1.f;
        int e = 0;
        if (a.x_exp) {
            float top = 0.f;
            for (long long j = 8 * tr; live && j < a.cols; j += 8 * a.row_threads) {
                float v[8];
                load8x(a.x, base + j, a.dtype, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) { const float f = fabsf(v[k]); if (f < INFINITY) top = fmaxf(top, f); }
            }
            top = row_max(top, a.row_threads, red);
            if (top > 0.f) { frexpf(top, &e); e -= 14; }
            s1 = pow2(-(e / 2));
            s2 = pow2(-(e - e / 2));
        }
        constexpr int U = 8;                                // copies that one reading of the row serves
        for (int c0 = 0; c0 < a.copies; c0 += U) {
            int at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int slot = r * a.copies + c0 + u;
                const bool mine = live && c0 + u < a.copies;
                at[u] = mine && !a.ids ? slot : -1;
                if (a.pos && mine) at[u] = a.pos[slot];
                if (a.ids && !a.pos && c0 + u < a.copies) {
                    // few slots: the place is the number of slots that sort before this one
                    const int id = live ? a.ids[slot] : -1;
                    int before = 0;
                    for (int s = tr; s < a.n_slots; s += a.row_threads) {
                        const int o = a.ids[s];
                        before += o >= 0 && (o < id || (o == id && s < slot)) ? 1 : 0;
                    }
                    before = row_sum(before, a.row_threads, redi);
                    const bool ok = id >= 0 && id < a.n_mats;
                    at[u] = ok ? before : -1;
                    if (live && tr == 0) {
                        if (ok) a.order[before] = slot;
                        else atomicOr(a.fault, kFaultExpertId);
                    }
                }
                if (mine && at[u] < 0)
                    for (long long j = tr; j < a.y_cols; j += a.row_threads)
                        store_elem(a.y, (long long)slot * a.y_cols + j, a.y_dtype, __int_as_float(0x7fc00000));
                if (at[u] >= 0 && a.x_exp && tr == 0) a.x_exp[at[u]] = e;
            }
            for (long long j = 8 * tr; live && j < a.cols; j += 8 * a.row_threads) {
                float v[8];
                uint32_t h[4], l[4];
                load8x(a.x, base + j, a.dtype, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f0 = v[2 * k] * s1 * s2, f1 = v[2 * k + 1] * s1 * s2;
                    // Of two terms, an infinity or a NaN is the second one: the first meets the weights' second terms as well,
                    // whose zeros and other signs would make NaN of an infinity.
                    const __half2 p = a.lo ? __floats2half2_rn(fminf(fmaxf(f0, -65504.f), 65504.f), fminf(fmaxf(f1, -65504.f), 65504.f))
                                           : __floats2half2_rn(f0, f1);
                    h[k] = *reinterpret_cast<const uint32_t *>(&p);
                    const __half2 q = __floats2half2_rn(f0 - __low2float(p), f1 - __high2float(p));
                    l[k] = *reinterpret_cast<const uint32_t *>(&q);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (at[u] < 0) continue;
                    *reinterpret_cast<uint4 *>(a.hi + (long long)at[u] * a.cols + j) = make_uint4(h[0], h[1], h[2], h[3]);
                    if (a.lo) *reinterpret_cast<uint4 *>(a.lo + (long long)at[u] * a.cols + j) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            }
        }
    }
}

// One tile of tokens: its distinct adapters in the order of their first token, and each token's place among them.
__device__ void list_tile(const PrepArgs &a, int tt) {
    __shared__ int ids[kMaxTokens], first[kMaxTokens];
    const int start = tt * a.tile_n, n = min(a.tile_n, a.n_tokens - start), j = threadIdx.x;
    int id = -1;
    if (j < n) {
        id = a.adapter_ids[start + j];
        ids[j] = id;
    }
    __syncthreads();
    if (j < n) {
        int f = 0;
        while (ids[f] != id) ++f;
        first[j] = f;
    }
    __syncthreads();
    if (j < n) {
        const bool ok = id >= 0 && id < a.n_adapters;
        int place = id == -1 ? -1 : -2;
        if (ok) {
            place = 0;
            for (int i = 0; i < first[j]; ++i) place += first[i] == i && ids[i] >= 0 && ids[i] < a.n_adapters ? 1 : 0;
            if (first[j] == j) a.tile_list[start + place] = id;
        } else if (place == -2) {
            atomicOr(a.fault, kFaultAdapterId);
        }
        a.place[start + j] = place;
    }
    const int count = __syncthreads_count(j < n && first[j] == j && id >= 0 && id < a.n_adapters);
    if (j == 0) a.tile_count[tt] = count;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t a0, const uint32_t a1, const uint32_t a2, const uint32_t a3,
                                         const uint32_t b0, const uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// u[t][k] = scale A[adapter][k] . x[t] for a window of tokens.  Its tokens are put into groups of at most 8 NT of one
// adapter, numbered by their first token, of which this block takes every turns-th: an adapter's A is read once for a group.
// x is one (bf16), two (f16) or three (f32) bf16 terms, exactly.  Warps take 32 ranks each, and the columns are split
// over what warps that leaves and over a cluster; their order inside a product is a lane's own (8 neighbours a
// lane), the same for both operands.
template <int DT, int NT>
__device__ void adapter_down(const PrepArgs &a, int window, int turn) {
    constexpr int TERMS = DT == HQ_DT_BF16 ? 1 : DT == HQ_DT_F16 ? 2 : 3, N = 8 * NT, WARPS = kPrepThreads / 32;
    constexpr int kXVecs = DT == HQ_DT_F32 ? 2 : 1;
    extern __shared__ float part[];                         // [slices][32 halves][N], then [down_split][32 halves][N]
    __shared__ alignas(16) int ids[kWindow];
    __shared__ int heads[kWindow / 32], tok[N], group_id, group_first;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int halves = a.rank <= 32 ? 1 : 2, slices = WARPS / halves, vals = halves * 32 * N;
    const int r0 = warp % halves * 32 + g, slice = warp / halves;
    float *joined = part + slices * vals;
    const int t0 = window * kWindow, crank = a.down_split > 1 ? (int)cluster_ctarank() : 0;
    const int units = (int)(a.cols / 32);
    const int u_lo = (int)((long long)units * crank / a.down_split), u_hi = (int)((long long)units * (crank + 1) / a.down_split);
    if (a.down_split > 1) {
        cluster_arrive_relaxed();
        cluster_wait();                                     // the first block runs: its shared memory may be written
    }
    // of a token: how many before it share its adapter; every N-th of those heads a group
    int id = -1, before = 0, nth = -1;
    if (threadIdx.x < kWindow) {
        if (t0 + threadIdx.x < a.n_tokens) id = a.adapter_ids[t0 + threadIdx.x];
        if (id >= a.n_adapters) id = -1;
        ids[threadIdx.x] = id;
    }
    __syncthreads();
    if (threadIdx.x < kWindow) {
        for (int k = 0; id >= 0 && k < (int)threadIdx.x; k += 4) {
            const int4 o = *reinterpret_cast<const int4 *>(ids + k);
            before += (o.x == id) + (o.y == id && k + 1 < threadIdx.x) + (o.z == id && k + 2 < threadIdx.x) + (o.w == id && k + 3 < threadIdx.x);
        }
        const uint32_t h = __ballot_sync(0xffffffffu, id >= 0 && before % N == 0);
        if (lane == 0) heads[warp] = __popc(h);
        if ((h >> lane) & 1) nth = __popc(h & ((1u << lane) - 1));
    }
    __syncthreads();
    int groups = 0;
    for (int w = 0; w < kWindow / 32; ++w) {
        if (nth >= 0 && w < warp) nth += heads[w];
        groups += heads[w];
    }
    for (int grp = turn; grp < groups; grp += a.down_turns) {
        __syncthreads();                                    // the last group's sums are read, and its tokens
        if (nth == grp) { group_id = id; group_first = before; }
        if (threadIdx.x < N) tok[threadIdx.x] = -1;
        __syncthreads();
        const int ad = group_id;
        if (id >= 0 && id == ad && before >= group_first && before < group_first + N) tok[before - group_first] = t0 + threadIdx.x;
        __syncthreads();
        int mine[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) mine[n] = max(tok[8 * n + g], tok[0] & -(tok[8 * n + g] < 0));
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        const uint16_t *A = a.A + ((long long)ad * a.rank + r0) * a.cols + c * 8;
        // Units of 32 columns, two on their way while one is multiplied.  Places without a token repeat the group's first:
        // what they add up is not stored.
        struct Unit { uint4 p[4], x[NT][kXVecs]; } buf[3];
        auto load = [&](Unit &b, int un) {
            const long long col = un * 32ll;
#pragma unroll
            for (int h = 0; h < 4; ++h) {                   // rows g and g + 8 of two tiles of 16 ranks
                b.p[h] = make_uint4(0, 0, 0, 0);
                if (r0 + 8 * h < a.rank) b.p[h] = *reinterpret_cast<const uint4 *>(A + 8 * h * a.cols + col);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kXVecs; ++i)
                    b.x[n][i] = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) +
                                                                ((long long)mine[n] * a.cols + col + c * 8) * (DT == HQ_DT_F32 ? 4 : 2))[i];
        };
        auto multiply = [&](const Unit &b) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float v[8];
                unpack8<DT>(b.x[n], v);
#pragma unroll
                for (int i = 0; i < TERMS; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = i + 1 < TERMS ? take_term<false>(v[2 * k], v[2 * k + 1]) : take_term<true>(v[2 * k], v[2 * k + 1]);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint4 lo = b.p[2 * m], hi = b.p[2 * m + 1];
                        mma_bf16(acc[m][n], lo.x, hi.x, lo.y, hi.y, w[0], w[1]);
                        mma_bf16(acc[m][n], lo.z, hi.z, lo.w, hi.w, w[2], w[3]);
                    }
                }
            }
        };
        const int u0 = u_lo + slice;
        if (u0 < u_hi) load(buf[0], u0);
        if (u0 + slices < u_hi) load(buf[1], u0 + slices);
#pragma unroll 1
        for (int un = u0; un < u_hi; un += 3 * slices)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (un + (k + 2) * slices < u_hi) load(buf[(k + 2) % 3], un + (k + 2) * slices);
                if (un + k * slices < u_hi) multiply(buf[k]);
            }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[slice * vals + (r0 + 16 * m + (i >> 1) * 8) * N + 8 * n + 2 * c + (i & 1)] = acc[m][n][i];
        __syncthreads();
        for (int i = threadIdx.x; i < a.rank * N; i += kPrepThreads) {
            float s = 0.f;
            for (int w = 0; w < slices; ++w) s += part[w * vals + i];
            if (a.down_split > 1) st_shared_cluster_f32(map_shared_rank(smem_u32(joined + crank * vals + i), 0), s);
            else joined[i] = s;
        }
        if (a.down_split > 1) cluster_sync(); else __syncthreads();
        if (crank == 0) {
            const float scale = a.scales[ad];
            for (int i = threadIdx.x; i < a.rank * N; i += kPrepThreads) {
                const int k = i / N, t = i % N;
                float s = 0.f;
                for (int d = 0; d < a.down_split; ++d) s += joined[d * vals + i];
                if (tok[t] >= 0) a.u[(long long)tok[t] * a.rank + k] = scale * s;
            }
        }
        if (a.down_split > 1) cluster_sync();
    }
}

// Grouped products, and tokens without adapters: the tiles (of few slots), and the tokens' terms.  A copy, bound by memory
// where it is long (4096 tokens of 2048 columns to eight places each: 35 us, 4.3 TB/s) and by latency where it is not (9 us at 5
// tokens).  A copy a slot, so that the products fetch a tile of tokens with one instruction.
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const __grid_constant__ PrepArgs a) {
    extern __shared__ float dyn[];
    griddep_wait();
    griddep_launch_dependents();                            // after the wait: the products' first weights rely on it
    const int b = blockIdx.x;
    if (b < a.plan_blocks) plan_slots<kPrepThreads, false>(a, reinterpret_cast<int *>(dyn), 1, 0);
    else pack_rows(a, b - a.plan_blocks);
}

// With adapters: the tokens' terms, each tile's adapters, and u, at once.  Bound by the latency of the loads of A and x, of
// which a warp has two units on their way, one block of 126 registers a thread on a multiprocessor: 2011 tokens at rank 64 and 4096
// columns 31 us, 64 tokens at rank 16 15 us, both in two waves of blocks; one token 12 us
// (a block a group of tokens instead of one an adapter and 16 tokens: 44 us and 23 us before).
__global__ void __launch_bounds__(kPrepThreads) prepare_adapters_kernel(const __grid_constant__ PrepArgs a) {
    griddep_wait();
    griddep_launch_dependents();                            // after the wait: the products' first weights rely on it
    int b = blockIdx.x;
    if (b < a.pack_blocks) { pack_rows(a, b); return; }
    b -= a.pack_blocks;
    if (b < a.list_blocks) { if (b * (long long)a.tile_n < a.n_tokens) list_tile(a, b); return; }
    b = (b - a.list_blocks) / a.down_split;
    const int turn = b % a.down_turns;
    b /= a.down_turns;
    if (a.dtype == HQ_DT_F32) adapter_down<HQ_DT_F32, 1>(a, b, turn);
    else if (a.down_tokens == 8) {
        if (a.dtype == HQ_DT_BF16) adapter_down<HQ_DT_BF16, 1>(a, b, turn);
        else adapter_down<HQ_DT_F16, 1>(a, b, turn);
    } else {
        if (a.dtype == HQ_DT_BF16) adapter_down<HQ_DT_BF16, 2>(a, b, turn);
        else adapter_down<HQ_DT_F16, 2>(a, b, turn);
    }
}

// y[t][i] = sum_k router_w[t][k] part[t][k][i], V columns a thread.  A read of the slots' sums, from L2 where they fit: 517
// tokens of 8 slots and 2048 rows 9 us, 3.7 TB/s.
template <int V>
__global__ void __launch_bounds__(256) combine_kernel(const float *part, const float *router_w, void *y, long long n_tokens,
                                                      int n_active, long long rows, int dtype) {
    griddep_launch_dependents();
    griddep_wait();
    const long long per = rows / V;
    for (long long o = blockIdx.x * 256ll + threadIdx.x; o < n_tokens * per; o += gridDim.x * 256ll) {
        const long long t = o / per, i = o % per * V;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
#pragma unroll 4
        for (int k = 0; k < n_active; ++k) {
            const float w = router_w[t * n_active + k];
            const float *p = part + (t * n_active + k) * rows + i;
            if constexpr (V == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p);
                s[0] = fmaf(w, v.x, s[0]); s[1] = fmaf(w, v.y, s[1]); s[2] = fmaf(w, v.z, s[2]); s[3] = fmaf(w, v.w, s[3]);
            } else {
                s[0] = fmaf(w, p[0], s[0]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) store_elem(y, t * rows + i + j, dtype, s[j]);
    }
}

// The largest finite |d| of a matrix, a block a matrix: set-up, once a weight, one read of the scales (two bytes of each block, so
// of every sector).  128 experts of 1536 x 2048 64 us; a single matrix is bound by its one block's loads, 151936 x 2048 1.6 ms.
__global__ void __launch_bounds__(1024) weight_exponents_kernel(int bytes, const uint8_t *W, int32_t *w_exp,
                                                                long long blocks) {
    griddep_wait();
    __shared__ float red[32];
    const uint8_t *w = W + blockIdx.x * blocks * bytes;
    float m = 0.f;
    for (long long b = threadIdx.x; b < blocks; b += blockDim.x) {
        const float d = fabsf(__half2float(*reinterpret_cast<const __half *>(w + b * bytes)));
        if (d < INFINITY) m = fmaxf(m, d);
    }
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = red[threadIdx.x];
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        int e = 0;
        if (m > 0.f) frexpf(m * (bytes == 34 ? 128.f : 8.f), &e);
        if (threadIdx.x == 0) w_exp[blockIdx.x] = e - 14;
    }
}

// Test-only: one of the library's bounded waits, on a barrier that nothing arrives on.
__global__ void __launch_bounds__(32) wait_selftest_kernel(int wait, uint32_t prior, uint32_t *fault, long long limit_cycles) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort = 0;
        fence_mbar_init();
        if (prior) atomicOr(fault, prior);
    }
    __syncwarp();
    if (threadIdx.x == 0) {
        if (wait == 0) mbar_wait(smem_u32(&bar), 0, &abort, fault, limit_cycles);
        else if (wait == 1) mbar_wait_cluster(smem_u32(&bar), 0, &abort, fault, limit_cycles);
        else if (wait == 2) tc_wait(smem_u32(&bar), 0, &abort, fault, (uint32_t)limit_cycles);
        else tc_wait_go(false, smem_u32(&bar), 0, &abort, fault, max(1u, (uint32_t)(limit_cycles >> 16)));
    }
    __syncwarp();
}

// ------------------------------------------------------------------ host side

template <class... P, class... A>
hq_status launch(void (*kern)(P...), int grid, int threads, size_t smem, int cluster, cudaStream_t stream, const char *what,
                 A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "%s launch: %s", what, cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

hq_status encode(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint32_t rank, const uint64_t *dims,
                 const uint64_t *strides, const uint32_t *box, bool swizzle) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!enc) return set_error(HQ_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t d[3], s[2];
    cuuint32_t b[3], one[3] = {1, 1, 1};
    for (uint32_t i = 0; i < rank; ++i) { d[i] = dims[i]; b[i] = box[i]; if (i) s[i - 1] = strides[i - 1]; }
    const CUresult r = enc(m, dt, rank, const_cast<void *>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(HQ_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return HQ_OK;
}

int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Where the workspace's parts begin.
struct Layout {
    int64_t hi = 0, lo = 0, x_exp = 0, order = 0, pos = 0, n_tiles = 0, tiles = 0, part = 0;
    int64_t u = 0, tile_count = 0, tile_list = 0, place = 0, total = 0;
};

// Tiles of tokens at most: an expert's tiles but its last hold 16 tokens or more.
int64_t most_tiles(const MatmulArgs &a) {
    const int64_t slots = a.n_tokens * a.n_active;
    return slots / 16 + std::min(slots, a.n_mats) + 1;
}

Layout layout(const MatmulArgs &a) {
    Layout l;
    const int64_t slots = a.n_tokens * a.n_active;          // rows of the token operand
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t p = at; at += up256(bytes); return p; };
    if (a.n_tokens == 0) return l;
    if (a.moe || a.dtype != HQ_DT_F16) {
        l.hi = take(slots * a.cols * 2);
        if (a.dtype == HQ_DT_F32) l.lo = take(slots * a.cols * 2);
        l.x_exp = take(slots * 4);
    }
    if (a.moe) {
        l.n_tiles = take(4);
        l.order = take(slots * 4);
        l.pos = take(slots * 4);
        l.tiles = take(most_tiles(a) * (int64_t)sizeof(TileRec));
        if (a.epilogue == HQ_MOE_EPI_COMBINE) l.part = take(slots * a.rows * 4);
    } else if (a.rank > 0) {
        l.u = take(a.n_tokens * a.rank * 4);
        l.tile_count = take((a.n_tokens / 16 + 1) * 4);
        l.tile_list = take(a.n_tokens * 4);
        l.place = take(a.n_tokens * 4);
    }
    l.total = at;
    return l;
}

struct TcPlan { int tile_n, ksplit, grid, raw_slots, x_slots, x_k, deep, tmem_cols; size_t smem; uint32_t off_raw, off_red; };

// Memory of a launch with tiles of p->tile_n tokens and the columns split over p->ksplit CTAs; false if it does not fit.
bool fit_smem(const DeviceInfo &dev, int fmt, bool split, TcPlan *p) {
    const int terms = split ? 2 : 1;
    const int chunk = (fmt == 8 ? Fmt<8>::kChunk : Fmt<4>::kChunk) * kTileRows;
    const int per = (p->tile_n / 16 + p->ksplit - 1) / p->ksplit * 2;
    const size_t red = p->ksplit > 1 ? (size_t)(p->ksplit - 1) * per * 8 * kTileRows * 4 : 0;
    const size_t fixed = red + kOffX;
    const size_t room = (size_t)dev.max_smem_optin, xb = (size_t)p->tile_n * 128 * terms;
    // Tokens in units of 64 columns, weights in chunks of 256: as many raw chunks as leave six units (eight for a fourth
    // chunk), which at 400 cycles each or more cover a copy's way from L2; at least four and one.
    auto units = [&](int raw) { return (int)((room - std::min(room, fixed + (size_t)raw * chunk)) / xb); };
    p->raw_slots = 0;
    for (int raw = kMaxRaw; raw >= 1 && !p->raw_slots; --raw)
        if (units(raw) >= (raw == kMaxRaw ? 8 : 6)) p->raw_slots = raw;
    for (int raw = kMaxRaw; raw >= 1 && !p->raw_slots; --raw)
        if (units(raw) >= 4) p->raw_slots = raw;
    if (!p->raw_slots) return false;
    // in as few slots as leave four
    const int n = units(p->raw_slots);
    p->x_k = n >= 16 ? 4 : n >= 8 ? 2 : 1;
    p->x_slots = p->x_k == 4 ? 4 : std::min(kMaxX, n / p->x_k);
    const int columns = p->x_k * p->x_slots;
    uint32_t at = (uint32_t)(kOffX + xb * columns);
    p->off_raw = at;
    at += (uint32_t)(p->raw_slots * chunk);
    p->off_red = at;
    p->smem = at + red;
    return true;
}

// Tokens of a tile and column split of the launch: the least estimated time over the choices.
// `groups` groups of about `n` tokens each (one group where nothing is grouped); the device may find other sizes,
// which the tile's capacity then cuts.
bool make_plan(const DeviceInfo &dev, int fmt, bool split, int64_t groups, int64_t n, int64_t n_rt, int n_chunks, TcPlan *best) {
    const int most = split ? kMaxTokensSplit : kMaxTokens;
    double best_t = 0;
    bool any = false;
    for (int tn = 16; tn <= most; tn += 16) {
        const int64_t tt = (n + tn - 1) / tn;
        const int used = (int)std::min<int64_t>(tn, (n + 15) / 16 * 16);
        if (used < tn) break;                               // a larger tile only holds air
        for (int ks = 1; ks <= 8 && ks <= n_chunks; ks *= 2) {
            TcPlan p = {};
            p.tile_n = tn;
            p.ksplit = ks;
            if (!fit_smem(dev, fmt, split, &p)) continue;
            const int64_t clusters = dev.num_sms / ks;
            const int64_t waves = (groups * tt * n_rt + clusters - 1) / clusters;
            // cycles of a chunk: its products, or decode and the weights' share of the memory bandwidth; of an item, the
            // gap between two tiles' products; at the end, the last tile's outputs, which a column split makes every
            // item wait for
            const double chunk = std::max<double>(split ? 28.0 * std::max(tn, 32) : 8.5 * tn, split ? 2200.0 : 1700.0);
            const double out = 3000.0 + 100.0 * tn;
            const double time = waves * (chunk * ((n_chunks + ks - 1) / ks) + 1200.0 + (ks > 1 ? 5000.0 + out / ks : 0.0)) + out;
            if (!any || time < best_t) { any = true; best_t = time; *best = p; }
        }
    }
    if (!any) return false;
    // TMEM: two buffers of accumulators (f32: of both kinds, and the running sums), and one or two buffers of decoded chunks
    const int sums = best->tile_n * (split ? 5 : 2), slots = 4 * kSlotCols * (split ? 2 : 1);
    best->deep = sums + 2 * slots <= 512;
    best->tmem_cols = 32;
    while (best->tmem_cols < sums + slots * (best->deep ? 2 : 1)) best->tmem_cols *= 2;
    best->grid = dev.num_sms / best->ksplit * best->ksplit;
    return true;
}

// Raises a kernel's shared-memory opt-in, once per device (`dynamic`: all that its static arrays leave).
template <auto KERNEL>
hq_status configure(int dynamic) {
    static std::atomic<bool> done[64];
    int d = 0;
    cudaGetDevice(&d);
    if (d >= 0 && d < 64 && done[d].load(std::memory_order_acquire)) return HQ_OK;
    const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, dynamic);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    if (d >= 0 && d < 64) done[d].store(true, std::memory_order_release);
    return HQ_OK;
}

template <int FMT, bool SPLIT, int OT>
hq_status launch_tc(const TcArgs &t, const TcPlan &p, cudaStream_t stream) {
    hq_status st = configure<matmul_tc_kernel<FMT, SPLIT, OT>>(232448);
    return st != HQ_OK ? st : launch(matmul_tc_kernel<FMT, SPLIT, OT>, p.grid, Roles<SPLIT>::kThreads, p.smem, p.ksplit, stream, "matmul", t);
}

template <int FMT>
hq_status launch_tc(const TcArgs &t, const TcPlan &p, bool split, int out, cudaStream_t stream) {
    if (split) return launch_tc<FMT, true, HQ_DT_F32>(t, p, stream);
    if (out == HQ_DT_F32) {                                 // the sums that the combine kernel takes
        if constexpr (FMT == 8) return launch_tc<FMT, false, HQ_DT_F32>(t, p, stream);
        return set_error(HQ_ERR_UNSUPPORTED, "f32 sums of 16-bit tokens are grouped products'");
    }
    return out == HQ_DT_F16 ? launch_tc<FMT, false, HQ_DT_F16>(t, p, stream) : launch_tc<FMT, false, HQ_DT_BF16>(t, p, stream);
}

}  // namespace

int64_t matmul_workspace(const MatmulArgs &a) {
    if (most_tiles(a) * ((a.rows + kTileRows - 1) / kTileRows) > 0x7fff0000LL)     // (a few steps of the grid fit an int behind them)
        return set_error(HQ_ERR_SHAPE, "more than 2^31 tiles of 16 tokens and 128 rows");
    return layout(a).total;
}

hq_status launch_matmul(const MatmulArgs &a, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    const Layout l = layout(a);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const bool split = a.dtype == HQ_DT_F32;
    const int64_t slots = a.n_tokens * a.n_active, n_rt = (a.rows + kTileRows - 1) / kTileRows;
    const int chunk = a.fmt == 8 ? Fmt<8>::kChunk : Fmt<4>::kChunk;
    const int n_chunks = (int)(a.cols / 256);

    TcPlan p;
    const int64_t groups = a.moe ? std::min(a.n_mats, slots) : 1;
    const int64_t typical = a.moe ? std::max<int64_t>(16, (slots + groups - 1) / groups * 3 / 2) : a.n_tokens;
    if (!make_plan(*dev, a.fmt, split, groups, typical, n_rt, n_chunks, &p))
        return set_error(HQ_ERR_UNSUPPORTED, "the device's shared memory is too small");

    PrepArgs q = {};
    q.x = a.x;
    q.cols = a.cols;
    q.dtype = a.dtype;
    q.fault = dev->fault;
    q.n_tokens = (int)a.n_tokens;
    q.tile_n = p.tile_n;
    q.down_split = 1;
    const bool pack = a.moe || a.dtype != HQ_DT_F16;
    if (pack) {
        q.x_rows = (int)(a.moe && a.x_per_slot ? slots : a.n_tokens);
        q.copies = (int)(slots / q.x_rows);
        q.hi = reinterpret_cast<__half *>(ws + l.hi);
        q.lo = split ? reinterpret_cast<__half *>(ws + l.lo) : nullptr;
        q.x_exp = a.dtype == HQ_DT_F16 ? nullptr : reinterpret_cast<int32_t *>(ws + l.x_exp);
        q.row_threads = 32;
        while (q.row_threads < kPrepThreads && q.row_threads * 8 < a.cols) q.row_threads *= 2;
        const int per = kPrepThreads / q.row_threads;
        q.pack_blocks = (int)std::min<int64_t>((q.x_rows + per - 1) / per, (int64_t)dev->num_sms * 16);
    }
    size_t prep_smem = 0;
    int down_blocks = 0;
    if (a.moe) {
        q.ids = a.idx;
        q.w_exp = a.w_exp;
        q.n_slots = (int)slots;
        q.n_mats = (int)a.n_mats;
        q.order = reinterpret_cast<int32_t *>(ws + l.order);
        q.n_tiles = reinterpret_cast<int32_t *>(ws + l.n_tiles);
        q.tiles = reinterpret_cast<TileRec *>(ws + l.tiles);
        const bool comb = a.epilogue == HQ_MOE_EPI_COMBINE;
        q.y = comb ? ws + l.part : a.y;
        q.y_dtype = comb ? HQ_DT_F32 : a.dtype;
        q.y_cols = a.epilogue == HQ_MOE_EPI_SWIGLU ? a.rows / 2 : a.rows;
        if (slots <= kSelfPlan) {
            q.plan_blocks = 1;
            prep_smem = (size_t)a.n_mats * 4;
        } else {
            q.pos = reinterpret_cast<int32_t *>(ws + l.pos);
            // a cluster of blocks where one would take more than a few loads a thread
            const int blocks = slots > 8192 ? 8 : 1;
            st = configure<plan_kernel>(2 * 8192 * 4);
            if (st == HQ_OK) st = launch(plan_kernel, blocks, 1024, (size_t)a.n_mats * 8, blocks, stream, "plan", q);
            if (st != HQ_OK) return st;
        }
    } else if (a.n_adapters > 0) {
        q.adapter_ids = a.idx;
        q.A = a.A;
        q.scales = a.scales;
        q.n_adapters = a.n_adapters;
        q.rank = a.rank;
        q.u = reinterpret_cast<float *>(ws + l.u);
        q.tile_count = reinterpret_cast<int32_t *>(ws + l.tile_count);
        q.tile_list = reinterpret_cast<int32_t *>(ws + l.tile_list);
        q.place = reinterpret_cast<int32_t *>(ws + l.place);
        // groups of 8 tokens (f32: three terms; or all there are) or 16; about two blocks for each multiprocessor, over the windows and what
        // groups they may have (one runs there at a time, for its registers), and a cluster of blocks over the columns where those are few
        q.down_tokens = split || a.n_tokens <= 8 ? 8 : 16;
        const int64_t windows = (a.n_tokens + kWindow - 1) / kWindow, in_window = std::min<int64_t>(kWindow, a.n_tokens);
        const int64_t most = std::min<int64_t>(in_window, a.n_adapters + (in_window + q.down_tokens - 1) / q.down_tokens);
        q.down_turns = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2 * dev->num_sms / windows));
        const int64_t work = windows * q.down_turns;
        while (q.down_split < 8 && work * q.down_split * 2 <= dev->num_sms * 3 / 2 && a.cols / 32 / (q.down_split * 2) >= 16) q.down_split *= 2;
        const int ks = q.down_split;
        q.pack_blocks = (q.pack_blocks + ks - 1) / ks * ks;
        q.list_blocks = (int)(((a.n_tokens + p.tile_n - 1) / p.tile_n + ks - 1) / ks * ks);
        down_blocks = (int)work * ks;
        const int halves = a.rank <= 32 ? 1 : 2;
        prep_smem = (size_t)(kPrepThreads / 32 / halves + ks) * (halves * 32) * q.down_tokens * 4;
    }
    const int prep_grid = q.plan_blocks + q.pack_blocks + q.list_blocks + down_blocks;
    if (prep_grid > 0) {
        if (down_blocks > 0) {
            st = configure<prepare_adapters_kernel>(64 * 1024);
            if (st == HQ_OK) st = launch(prepare_adapters_kernel, prep_grid, kPrepThreads, prep_smem, q.down_split, stream, "prepare", q);
        } else {
            st = launch(prepare_kernel, prep_grid, kPrepThreads, prep_smem, 1, stream, "prepare", q);
        }
        if (st != HQ_OK) return st;
    }

    TcArgs t = {};
    const uint64_t w_dims[2] = {(uint64_t)n_chunks * chunk / 2, (uint64_t)(a.n_mats * a.rows)}, w_stride = (uint64_t)n_chunks * chunk;
    const uint32_t w_box[2] = {(uint32_t)chunk / 2, kTileRows};
    st = encode(&t.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.W, 2, w_dims, &w_stride, w_box, false);
    const void *xh = pack ? (const void *)(ws + l.hi) : a.x;
    // the tokens as [64 columns][tokens][groups of 64 columns]: a box is a stage, laid out as its operands are
    auto encode_x = [&](CUtensorMap *m, const void *base, uint32_t rows) {
        const uint64_t dims[3] = {64, (uint64_t)slots, (uint64_t)a.cols / 64}, strides[2] = {(uint64_t)a.cols * 2, 128};
        const uint32_t box[3] = {64, rows, (uint32_t)p.x_k};
        if (st == HQ_OK) st = encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 3, dims, strides, box, true);
    };
    for (int b = a.moe ? 0 : kBoxes - 1; b < kBoxes; ++b) {
        const uint32_t rows = b == kBoxes - 1 ? (uint32_t)p.tile_n : 16u << b;
        if (rows > (uint32_t)p.tile_n) continue;
        encode_x(&t.map_x[b], xh, rows);
        if (split) encode_x(&t.map_lo[b], ws + l.lo, rows);
    }
    if (st != HQ_OK) return st;
    t.z.w_exp = a.w_exp;
    t.z.x_exp = q.x_exp;
    t.z.order = q.order;
    t.z.tiles = q.tiles;
    t.z.n_tiles = q.n_tiles;
    t.z.tile_count = q.tile_count;
    t.z.tile_list = q.tile_list;
    t.z.place = q.place;
    t.z.B = a.B;
    t.z.u = q.u;
    t.z.rank = a.rank;
    t.z.y = a.moe ? q.y : a.y;
    t.z.fault = dev->fault;
    t.z.rows = a.rows;
    t.z.n_tokens = (int)a.n_tokens;
    t.z.n_tt = (int)((a.n_tokens + p.tile_n - 1) / p.tile_n);
    t.z.n_rt = (int)n_rt;
    t.z.n_items = (int)((a.moe ? most_tiles(a) : t.z.n_tt) * t.z.n_rt);
    t.z.n_chunks = n_chunks;
    t.z.tile_n = p.tile_n;
    t.z.raw_slots = p.raw_slots;
    t.z.x_slots = p.x_slots;
    t.z.x_k = p.x_k;
    t.z.deep = p.deep;
    t.z.ksplit = p.ksplit;
    t.z.step = p.grid / p.ksplit;
    t.z.tmem_cols = p.tmem_cols;
    t.z.epilogue = a.epilogue == HQ_MOE_EPI_SWIGLU ? HQ_MOE_EPI_SWIGLU : 0;
    t.z.stream_w = !a.moe && t.z.n_tt == 1;
    t.z.early = !a.moe && prep_grid > 0;
    t.z.off_raw = p.off_raw;
    t.z.off_red = p.off_red;
    const int out = a.epilogue == HQ_MOE_EPI_COMBINE ? HQ_DT_F32 : a.dtype;
    st = a.fmt == 8 ? launch_tc<8>(t, p, split, out, stream) : launch_tc<4>(t, p, split, out, stream);
    if (st != HQ_OK) return st;
    if (a.epilogue == HQ_MOE_EPI_COMBINE) {
        const bool four = a.rows % 4 == 0;
        const int grid = (int)std::min<int64_t>((a.n_tokens * a.rows / (four ? 4 : 1) + 255) / 256, dev->num_sms * 16);
        st = launch(four ? combine_kernel<4> : combine_kernel<1>, grid, 256, 0, 1, stream, "combine",
                    (const float *)(ws + l.part), a.router_w, a.y, (long long)a.n_tokens, a.n_active, (long long)a.rows, a.dtype);
    }
    return st;
}

hq_status launch_wait_selftest(int wait, uint32_t prior, uint32_t *fault, int64_t cycles, cudaStream_t stream) {
    note_launch();
    wait_selftest_kernel<<<1, 32, 0, stream>>>(wait, prior, fault, (long long)cycles);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "self-test launch: %s", cudaGetErrorString(e));
    return HQ_OK;
}

hq_status launch_weight_exponents(int fmt, const void *W, int32_t *w_exp, int64_t n_mats, int64_t rows, int64_t cols,
                                  cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    return launch(weight_exponents_kernel, (int)n_mats, 1024, 0, 1, stream, "exponents", fmt == HQ_FMT_Q8_0 ? 34 : 18,
                  (const uint8_t *)W, w_exp, (long long)(rows * (cols / 32)));
}

}  // namespace hq
