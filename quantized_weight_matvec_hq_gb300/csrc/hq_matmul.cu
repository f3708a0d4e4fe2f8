// hq_matmul.cu -- products of many tokens with quantized weights on the tensor
// cores: grouped by expert, or shared with an adapter per request.
//
//   y[s][i] = sum_j w[m(s)][i][j] x[s][j],  w = d q (Q8_0) or d (n - 8) (Q4_0)
//
// A prepare kernel lays the call out, then one persistent kernel multiplies:
//  * The weights are the M operand (128 rows of W a tile) and the tokens the N
//    operand (16 to 256 a tile), so ragged groups of tokens cost what they are.
//  * Raw blocks come by TMA (256 columns of 128 rows a stage).  Two groups of four warps
//    decode them, a quarter (64 columns) at a time, to 16-bit floats in the swizzled layout the tensor core
//    reads; quarters take turns over four operand slots.
//  * Tokens come by TMA, an expert's tokens next to each other (the prepare kernel sorts them).
//  * Adapters are further columns of the same product: a tile's distinct adapters' B, side by side, times each token's
//    u = A x at its own adapter's place and zero elsewhere.
//  * Accumulators live in TMEM, two of them, so a tile's outputs are formed while the next one is
//    multiplied.
//  * Few tiles: a cluster splits the columns and joins its partial sums in a
//    fixed order through distributed shared memory.
//
// Numbers.  Decoded weights are d 2^-e q rounded to f16 (11 bits; e per matrix,
// so that the range of f16 fits the matrix), where bf16 would keep 8.  Tokens of
// bf16 become f16 exactly, scaled by a power of two per token (what lies 2^-29 below a
// token's largest element is rounded to 2^-39 of it).  f32 tokens and weights are two
// f16 terms each (22 bits) and three products; sums of 256 columns leave the
// tensor core, whose adds may truncate, and are added in fp32 to the running
// sum, with the two small products in an accumulator of their own.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "hq_internal.h"
#include "hq_tc.cuh"

namespace hq {
namespace {

// ------------------------------------------------------------------ shared with the host

constexpr int kTileRows = 128;
constexpr int kMaxTokens = 240;             // tokens of a tile: what four operand slots leave room for
constexpr int kMaxTokensSplit = 48;         // f32: twice the operands
constexpr int kSlots = 4;
constexpr int kABytes = kTileRows * 128;
constexpr int kEpiWarps = 8, kDecodeWarps = 8;
constexpr int kWarpW = kEpiWarps + kDecodeWarps, kWarpX = kWarpW + 1, kWarpMma = kWarpX + 1;
constexpr int kThreads = 32 * (kWarpMma + 1);
constexpr int kPrepThreads = 512;
constexpr int kMaxRaw = 4;

template <int FMT> struct Fmt;
template <> struct Fmt<8> { static constexpr int kChunk = 272, kVecs = 5; };   // bytes of 8 blocks; 16-byte units a quarter touches
template <> struct Fmt<4> { static constexpr int kChunk = 144, kVecs = 3; };

// Virtual ranks of an adapter stage: u is two bf16 terms (16 bits) of 32 ranks, or three (f32) of 16.
template <bool SPLIT> struct Ext { static constexpr int kRanks = SPLIT ? 16 : 32, kTerms = SPLIT ? 3 : 2; };

// One tile of tokens of one expert: sorted slots [start, start + n).
struct TileRec { int mat, start, n, w_exp; };

struct TcArgs {
    CUtensorMap map_w, map_x64, map_x16, map_lo64, map_lo16;
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
    int tile_n, raw_slots, ksplit, tmem_cols;
    int dtype, epilogue, rank, stream_w;
    uint32_t zero;                  // 0, unknown to the compiler
    uint32_t off_x, off_raw, off_red, off_meta;
};

struct Meta {
    uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw], full[kSlots], empty[kSlots];
    uint64_t acc_full[2], acc_empty[2], red_full, red_empty, done;
    uint32_t tmem;
    int abort;
    int slot[kMaxTokens];
    float2 scale[kMaxTokens];
};

struct Item { int mat, rt, start, n, w_exp, count; };

// Work item `w`: a tile of rows and a tile of tokens.  Grouped: an expert's row tiles follow one another, so
// that its weights are read again from L2 if it has several tiles of tokens; one matrix: a row tile's token
// tiles follow one another.
__device__ __forceinline__ Item get_item(const TcArgs &a, int w) {
    Item t;
    if (a.tiles) {
        const TileRec r = a.tiles[w / a.n_rt];
        t.rt = w % a.n_rt;
        t.mat = r.mat;
        t.start = r.start;
        t.n = r.n;
        t.w_exp = r.w_exp;
        t.count = 0;
    } else {
        const int tt = w % a.n_tt;
        t.mat = 0;
        t.rt = w / a.n_tt;
        t.start = tt * a.tile_n;
        t.n = min(a.tile_n, a.n_tokens - t.start);
        t.w_exp = *a.w_exp;
        t.count = a.tile_count ? a.tile_count[tt] : 0;
    }
    return t;
}

// Adapter stages of a tile, an even number, and this CTA's share of them.
template <bool SPLIT>
__device__ __forceinline__ int2 ext_range(const TcArgs &a, const Item &t, int rank) {
    const int pairs = (t.count * a.rank + 2 * Ext<SPLIT>::kRanks - 1) / (2 * Ext<SPLIT>::kRanks);
    return make_int2(2 * (pairs * rank / a.ksplit), 2 * (pairs * (rank + 1) / a.ksplit));
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// ------------------------------------------------------------------ decode

// A shared-memory load that stays before the barrier operations that follow it.
__device__ __forceinline__ void ld_shared_volatile(uint32_t addr, uint32_t *v) {
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

// Two blocks (64 columns) of one row: `w` holds the quarter's 16-byte units,
// block 0 starts at word I0.  The bytes q + 128 (Q8_0) or n (Q4_0) go into the
// mantissa of 1024, whose integers f16 holds exactly; 1024 + bias is subtracted
// exactly, and the product with the scaled d is rounded once.
template <int FMT, bool SPLIT, int I0>
__device__ __forceinline__ void decode_quarter(const uint32_t *w, float wscale, uint8_t *dst, int row) {
    const __half2 bias = FMT == 8 ? __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480))    // 1152
                                  : __half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));   // 1032
    constexpr int kWords = FMT == 8 ? 8 : 4;
    uint8_t *line = dst + row * 128;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t dw = b == 0 ? w[I0] & 0xffffu : w[I0 + kWords] >> 16;
        const __half ds = __float2half_rn(__half2float(__ushort_as_half((unsigned short)dw)) * wscale);
        const __half2 d = __half2half2(ds);
        uint32_t q[kWords];
#pragma unroll
        for (int j = 0; j < kWords; ++j)
            q[j] = b == 0 ? __funnelshift_r(w[I0 + j], w[I0 + j + 1], 16) : w[I0 + kWords + 1 + j];
#pragma unroll
        for (int c = 0; c < 4; ++c) {                    // 16-byte units of 8 columns
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v;
                if constexpr (FMT == 8) v = q[2 * c + h] ^ 0x80808080u;
                else v = (c < 2 ? q[2 * c + h] : q[2 * (c - 2) + h] >> 4) & 0x0f0f0f0fu;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint32_t m = prmt(v, 0x64646464u, p ? 0x4342u : 0x4140u);
                    const __half2 n = __hsub2(*reinterpret_cast<const __half2 *>(&m), bias);
                    const __half2 r = __hmul2(n, d);
                    hi[2 * h + p] = *reinterpret_cast<const uint32_t *>(&r);
                    if constexpr (SPLIT) {
                        const __half2 l = __hfma2(n, d, __hneg2(r));
                        lo[2 * h + p] = *reinterpret_cast<const uint32_t *>(&l);
                    }
                }
            }
            const int unit = ((4 * b + c) ^ (row & 7)) << 4;
            *reinterpret_cast<uint4 *>(line + unit) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (SPLIT) *reinterpret_cast<uint4 *>(line + kABytes + unit) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// ------------------------------------------------------------------ outputs

__device__ __forceinline__ void store_elem(void *y, long long i, int dtype, float v) {
    if (dtype == HQ_DT_F32) static_cast<float *>(y)[i] = v;
    else if (dtype == HQ_DT_F16) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

// z / (1 + e^-z).  The approximate exponential and quotient are within 2^-21 (1 + |z| / 4) of it.
__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// The 8 columns from c0 of output row `row` (its sums in v): scales, SwiGLU with the neighbouring lane's row, store.
__device__ __forceinline__ void finish8(const TcArgs &a, const Meta *m, int c0, int n, long long row, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 s = m->scale[c0 + j];
        v[j] = v[j] * s.x * s.y;
    }
    if (a.epilogue == HQ_MOE_EPI_SWIGLU) {
        // even lanes hold gate rows, odd lanes up rows: each finishes every other token
        const bool odd = threadIdx.x & 1;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const float h = odd ? silu(got) * v[j + 1] : silu(v[j]) * got;
            const int c = c0 + j + (odd ? 1 : 0);
            if (c < n && row < a.rows) store_elem(a.y, (long long)m->slot[c] * (a.rows / 2) + row / 2, a.dtype, h);
        }
        return;
    }
    if (row < a.rows) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c0 + j < n) store_elem(a.y, (long long)m->slot[c0 + j] * a.rows + row, a.dtype, v[j]);
    }
}

// ------------------------------------------------------------------ adapter stages

// Virtual ranks [v0, v0 + kRanks) of one row of the tile's adapters' B, packed in pairs.
template <bool SPLIT>
__device__ __forceinline__ void load_b(const TcArgs &a, const int32_t *list, int total, int v0, long long row, uint32_t (&b)[16]) {
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

// Row `c` of the token operand: u of the token's own adapter at its virtual ranks, as bf16 terms side by side, zero elsewhere.
template <bool SPLIT>
__device__ __forceinline__ void store_u(const TcArgs &a, const Item &t, int v0, int c, uint8_t *dst) {
    constexpr int R = Ext<SPLIT>::kRanks, T = Ext<SPLIT>::kTerms;
    const int place = c < t.n ? a.place[t.start + c] : -1;
    const int lo = place * a.rank - v0;                     // virtual rank v0 + k is rank k - lo of the adapter
    const bool any = place >= 0 && lo < R && lo + a.rank > 0;
    float s1 = 0.f, s2 = 0.f;
    if (any) {
        const int e = -(t.w_exp + (a.x_exp ? a.x_exp[t.start + c] : 0));
        s1 = pow2(e / 2);
        s2 = pow2(e - e / 2);
    }
    uint8_t *line = dst + c * 128;
    const float *u = a.u + (long long)(t.start + c) * a.rank;
#pragma unroll
    for (int k0 = 0; k0 < R; k0 += 8) {
        uint32_t w[T][4] = {};
        if (any) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = k0 + k - lo;
                float f = r >= 0 && r < a.rank ? u[r] * s1 * s2 : 0.f;
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    const __nv_bfloat16 h = __float2bfloat16_rn(f);
                    f -= __bfloat162float(h);
                    w[i][k / 2] |= (uint32_t)__bfloat16_as_ushort(h) << (16 * (k & 1));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < T; ++i)
            *reinterpret_cast<uint4 *>(line + (((i * R + k0) / 8 ^ (c & 7)) << 4)) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    }
}

// ------------------------------------------------------------------ the kernel

template <int FMT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) matmul_tc_kernel(const __grid_constant__ TcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Meta *m = reinterpret_cast<Meta *>(smem + a.off_meta);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int kTerms = SPLIT ? 2 : 1;
    constexpr int kChunkBytes = kTileRows * Fmt<FMT>::kChunk;
    const int rank = a.ksplit > 1 ? (int)cluster_ctarank() : 0;
    const uint32_t a_base = smem_u32(smem), x_base = a_base + a.off_x, raw_base = a_base + a.off_raw;
    const int x_bytes = a.tile_n * 128;
    volatile int *abort = &m->abort;
    uint32_t *fault = a.fault;

    if (threadIdx.x == 0) {
        m->abort = 0;
        for (int i = 0; i < a.raw_slots; ++i) { mbar_init(smem_u32(&m->raw_full[i]), 1); mbar_init(smem_u32(&m->raw_empty[i]), kDecodeWarps); }
        for (int i = 0; i < kSlots; ++i) { mbar_init(smem_u32(&m->full[i]), 5); mbar_init(smem_u32(&m->empty[i]), 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&m->acc_full[i]), 1); mbar_init(smem_u32(&m->acc_empty[i]), kEpiWarps); }
        mbar_init(smem_u32(&m->done), 1);
        mbar_init(smem_u32(&m->red_full), (uint32_t)max(1, (a.ksplit - 1) * kEpiWarps));
        mbar_init(smem_u32(&m->red_empty), (uint32_t)max(1, (a.ksplit - 1) * kEpiWarps));
        fence_mbar_init();
    }
    if (warp == kWarpMma) tmem_alloc(smem_u32(&m->tmem), (uint32_t)a.tmem_cols);
    tc_fence_before();
    if (a.ksplit > 1) cluster_sync(); else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&m->tmem;
    griddep_launch_dependents();

    const int first = blockIdx.x / a.ksplit, step = gridDim.x / a.ksplit;
    const int c_lo = (int)((long long)a.n_chunks * rank / a.ksplit);
    const int c_hi = (int)((long long)a.n_chunks * (rank + 1) / a.ksplit);
    // one matrix's weights may be fetched before the prepare kernel is done; everything else waits for it
    if (a.tiles || warp != kWarpW) griddep_wait();
    Item t = {};
    if (a.tiles || warp != kWarpW) t = get_item(a, min(first, a.n_items - 1));
    const int n_items = a.tiles ? *a.n_tiles * a.n_rt : a.n_items;

    if (warp == kWarpW) {
        const uint64_t pol = a.stream_w ? l2_evict_first_policy() : l2_evict_normal_policy();
        uint32_t s = 0, ph = 1, it = 0;
        bool ok = true;
        for (int w = first; w < n_items && ok; w += step) {
            const int row0 = a.tiles ? (int)((long long)t.mat * a.rows + (long long)t.rt * kTileRows) : w / a.n_tt * kTileRows;
            if (a.tiles && w + step < n_items) t = get_item(a, w + step);
            for (int c = c_lo; c < c_hi; ++c, ++it) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->raw_empty[s]), ph, abort, fault));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t bar = smem_u32(&m->raw_full[s]);
                    mbar_arrive_expect_tx(bar, kChunkBytes);
                    tma_load_2d(raw_base + s * kChunkBytes, &a.map_w, c * (Fmt<FMT>::kChunk / 2), row0, bar, pol);
                }
                if (++s == (uint32_t)a.raw_slots) { s = 0; ph ^= 1; }
            }
        }
        // copies in flight end before the block's memory is given back
        for (uint32_t k = it > (uint32_t)a.raw_slots ? it - a.raw_slots : 0; !ok && k < it; ++k)
            for (int tries = 0; tries < 1 << 12 && !mbar_try_wait(smem_u32(&m->raw_full[k % a.raw_slots]), (k / a.raw_slots) & 1); ++tries) {}
    } else if (warp == kWarpX) {
        const uint64_t pol = l2_evict_normal_policy();
        uint32_t it = 0;
        bool ok = true;
        for (int w = first; w < n_items && ok; w += step) {
            const Item cur = t;
            if (w + step < n_items) t = get_item(a, w + step);
            const int n16 = round16(cur.n);
            const int2 ext = ext_range<SPLIT>(a, cur, rank);
            const int main = 4 * (c_hi - c_lo), all = main + ext.y - ext.x;
            for (int k = 0; k < all; ++k, ++it) {
                const uint32_t s = it & 3;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->empty[s]), ((it >> 2) & 1) ^ 1, abort, fault));
                if (!ok) break;
                const uint32_t bar = smem_u32(&m->full[s]);
                if (elect_one()) {
                    if (k < main) {
                        mbar_arrive_expect_tx(bar, (uint32_t)(kTerms * n16 * 128));
                        const uint32_t dst = x_base + s * (kTerms * x_bytes);
                        const int col = (4 * c_lo + k) * 64;
                        int r = 0;
                        for (; r + 64 <= n16; r += 64) {
                            tma_load_2d(dst + r * 128, &a.map_x64, col, cur.start + r, bar, pol);
                            if constexpr (SPLIT) tma_load_2d(dst + x_bytes + r * 128, &a.map_lo64, col, cur.start + r, bar, pol);
                        }
                        for (; r < n16; r += 16) {
                            tma_load_2d(dst + r * 128, &a.map_x16, col, cur.start + r, bar, pol);
                            if constexpr (SPLIT) tma_load_2d(dst + x_bytes + r * 128, &a.map_lo16, col, cur.start + r, bar, pol);
                        }
                    } else {
                        mbar_arrive(bar);               // the decode warps fill this stage
                    }
                }
            }
        }
        // a copy in flight ends before the block's memory is given back (a slot whose stage never
        // fills up runs into the limit)
        for (uint32_t k = it > 4 ? it - 4 : 0; !ok && k < it; ++k)
            for (int tries = 0; tries < 1 << 12 && !mbar_try_wait(smem_u32(&m->full[k & 3]), (k >> 2) & 1); ++tries) {}
    } else if (warp == kWarpMma) {
        uint32_t it = 0, acc = 0;
        bool ok = true;
        const uint32_t half = SPLIT ? 2u * a.tile_n : (uint32_t)a.tmem_cols / 2;
        const uint64_t desc_a = tc_desc_sw128(a_base), desc_x = tc_desc_sw128(x_base);
        const uint32_t a_step = (kTerms * kABytes) >> 4, x_step = (uint32_t)(kTerms * x_bytes) >> 4;
        for (int w = first; w < n_items && ok; w += step) {
            const Item cur = t;
            if (w + step < n_items) t = get_item(a, w + step);
            const int n16 = round16(cur.n);
            const uint32_t idesc = tc_idesc(n16, false), idesc_b = tc_idesc(n16, true);
            const int2 ext = ext_range<SPLIT>(a, cur, rank);
            const int main = 4 * (c_hi - c_lo), all = main + ext.y - ext.x;
            for (int k = 0; k < all; ++k, ++it) {
                const bool fresh = k == 0 || (SPLIT && ((k & 3) == 0 && k <= main));
                if (fresh) {
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->acc_empty[acc & 1]), ((acc >> 1) & 1) ^ 1, abort, fault));
                    if (!ok) break;
                }
                const uint32_t s = it & 3;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->full[s]), (it >> 2) & 1, abort, fault));
                if (!ok) break;
                tc_fence_after();
                const bool last = k == all - 1 || (SPLIT && k < main && (k & 3) == 3);
                if (elect_one()) {
                    const uint32_t d = tmem + (acc & 1) * half;
                    const uint64_t da = desc_a + s * a_step, db = desc_x + s * x_step;
                    if (k < main) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            tc_mma(d, da + 2 * j, db + 2 * j, idesc, !(fresh && j == 0));
                            if constexpr (SPLIT) {
                                tc_mma(d + a.tile_n, da + 2 * j, db + (x_bytes >> 4) + 2 * j, idesc, !(fresh && j == 0));
                                tc_mma(d + a.tile_n, da + (kABytes >> 4) + 2 * j, db + 2 * j, idesc, true);
                            }
                        }
                    } else {
                        // the terms of u times the same columns of B
                        constexpr int kPer = Ext<SPLIT>::kRanks / 16;
#pragma unroll
                        for (int j = 0; j < kPer * Ext<SPLIT>::kTerms; ++j)
                            tc_mma(d, da + 2 * (j % kPer), db + 2 * j, idesc_b, !(fresh && j == 0));
                    }
                    tc_commit(smem_u32(&m->empty[s]));
                    if (last) tc_commit(smem_u32(&m->acc_full[acc & 1]));
                }
                __syncwarp();
                if (last) ++acc;
            }
        }
        // every product ends before TMEM is given back
        if (elect_one()) tc_commit(smem_u32(&m->done));
        for (int tries = 0; tries < 1 << 20 && !mbar_try_wait(smem_u32(&m->done), 0); ++tries) {}
        __syncwarp();
    } else if (warp >= kEpiWarps) {
        const int g = (warp - kEpiWarps) >> 2, row = (warp & 3) * 32 + lane;
        constexpr int kUnit = FMT == 8 ? 64 : 32;           // quarter q begins within the 16-byte unit at q * kUnit bytes
        const uint32_t src = raw_base + row * Fmt<FMT>::kChunk + g * kUnit;
        uint32_t it = 0, s = 0, ph = 0;
        bool ok = true;
        for (int w = first; w < n_items && ok; w += step) {
            const Item cur = t;
            if (w + step < n_items) t = get_item(a, w + step);
            const float wscale = pow2(-cur.w_exp);
            for (int c = c_lo; c < c_hi; ++c, it += 4) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->raw_full[s]), ph, abort, fault));
                if (!ok) break;
                uint32_t v[2][4 * Fmt<FMT>::kVecs];         // quarters g and g + 2
                uint32_t seen = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < Fmt<FMT>::kVecs; ++i) {
                        ld_shared_volatile(src + s * kChunkBytes + 2 * h * kUnit + 16 * i, v[h] + 4 * i);
                        seen |= v[h][4 * i];
                    }
                // The buffer goes back to the copy engine once its values are here.  The arrival
                // takes them as an operand (masked to nothing): an arrival alone does not wait for loads
                // in flight, and overtakes them when the load unit is busy.
                seen = __reduce_or_sync(0xffffffffu, seen & a.zero);
                if (lane == 0) mbar_arrive_count(smem_u32(&m->raw_empty[s]), 1 + seen);
                if (++s == (uint32_t)a.raw_slots) { s = 0; ph ^= 1; }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t k = it + g + 2 * h, slot = k & 3;
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->empty[slot]), ((k >> 2) & 1) ^ 1, abort, fault));
                    if (!ok) break;
                    uint8_t *dst = smem + slot * (kTerms * kABytes);
                    if (g == 0) decode_quarter<FMT, SPLIT, 0>(v[h] + 2 * h, wscale, dst, row);
                    else decode_quarter<FMT, SPLIT, 1>(v[h] + 2 * h, wscale, dst, row);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m->full[slot]));
                }
                if (!ok) break;
            }
            if (!ok || cur.count == 0) continue;
            // adapter stages: group g takes every other one
            const int2 ext = ext_range<SPLIT>(a, cur, rank);
            const int32_t *list = a.tile_list + cur.start;
            const int total = cur.count * a.rank;
            const long long r = min((long long)cur.rt * kTileRows + row, a.rows - 1);
            uint32_t b[2][16];
            if (ext.x < ext.y) load_b<SPLIT>(a, list, total, (ext.x + g) * Ext<SPLIT>::kRanks, r, b[0]);
            for (int e = ext.x + g; e < ext.y; e += 4) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int ee = e + 2 * h;
                    if (ee >= ext.y) break;
                    if (ee + 2 < ext.y) load_b<SPLIT>(a, list, total, (ee + 2) * Ext<SPLIT>::kRanks, r, b[h ^ 1]);
                    const uint32_t k = it + (ee - ext.x), slot = k & 3;
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->empty[slot]), ((k >> 2) & 1) ^ 1, abort, fault));
                    if (!ok) break;
                    uint8_t *line = smem + slot * (kTerms * kABytes) + row * 128;
#pragma unroll
                    for (int i = 0; i < Ext<SPLIT>::kRanks / 8; ++i)
                        *reinterpret_cast<uint4 *>(line + ((i ^ (row & 7)) << 4)) =
                            make_uint4(b[h][4 * i], b[h][4 * i + 1], b[h][4 * i + 2], b[h][4 * i + 3]);
                    for (int x = row; x < round16(cur.n); x += kTileRows)
                        store_u<SPLIT>(a, cur, ee * Ext<SPLIT>::kRanks, x, smem + a.off_x + slot * (kTerms * x_bytes));
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m->full[slot]));
                }
                if (!ok) break;
            }
            it += ext.y - ext.x;
        }
    } else {
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int side = warp >> 2;                         // of the two warps of these rows
        const uint32_t half = SPLIT ? 2u * a.tile_n : (uint32_t)a.tmem_cols / 2;
        const uint32_t run = 4u * a.tile_n;                 // SPLIT: the running sums
        float *red = reinterpret_cast<float *>(smem + a.off_red);
        const uint32_t red_addr = smem_u32(red);
        const int my_row = (warp & 3) * 32 + lane;
        uint32_t acc = 0, item = 0;
        bool ok = true;
        for (int w = first; w < n_items; w += step, ++item) {
            // the warps leave together, and the last tile's columns are read
            if (!named_barrier_and(1, 32 * kEpiWarps, ok)) break;
            const Item cur = t;
            if (w + step < n_items) t = get_item(a, w + step);
            const int n8 = round16(cur.n) / 8;
            const long long row = (long long)cur.rt * kTileRows + my_row;
            if ((int)threadIdx.x < round16(cur.n)) {
                const int j = threadIdx.x, at = cur.start + min(j, cur.n - 1);
                const int e = cur.w_exp + (a.x_exp ? a.x_exp[at] : 0);
                const bool bad = a.place && a.place[at] == -2;      // an adapter id out of range
                m->slot[j] = a.order ? a.order[at] : at;
                m->scale[j] = make_float2(bad ? __int_as_float(0x7fc00000) : pow2(e / 2), pow2(e - e / 2));
            }
            named_barrier(1, 32 * kEpiWarps);
            // One group of 8 columns of the current accumulator; f32 adds the small products' and the
            // running sums.
            auto load8 = [&](uint32_t base, int g, bool cross, bool join, float (&v)[8]) {
                tmem_ld8(base + 8 * g, v);
                if constexpr (SPLIT) {
                    float x[8], r[8];
                    if (cross) tmem_ld8(base + a.tile_n + 8 * g, x);
                    if (join) tmem_ld8(lane_base + run + 8 * g, r);
                    tmem_wait_ld(v);
                    if (cross) {
                        tmem_wait_ld(x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += x[j];
                    }
                    if (join) {
                        tmem_wait_ld(r);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += r[j];
                    }
                } else {
                    tmem_wait_ld(v);
                }
            };
            const int2 ext = ext_range<SPLIT>(a, cur, rank);
            const int rounds = SPLIT ? c_hi - c_lo + (ext.x < ext.y ? 1 : 0) : 1;
            const int ks = a.ksplit;
            // the columns this warp sums: every other group, or (with a split) those it sends or finishes
            for (int i = 0; i < rounds - 1 && ok; ++i, ++acc) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault));
                if (!ok) break;
                tc_fence_after();
                for (int g = side; g < n8; g += 2) {
                    float v[8];
                    load8(lane_base + (acc & 1) * half, g, true, i > 0, v);
                    tmem_st8(lane_base + run + 8 * g, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&m->acc_empty[acc & 1]));
            }
            if (!ok) continue;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault));
            if (!ok) continue;
            tc_fence_after();
            const uint32_t base = lane_base + (acc & 1) * half;
            const bool join = SPLIT && rounds > 1, cross = SPLIT && ext.x == ext.y;
            if (ks == 1) {
                for (int g = side; g < n8; g += 2) {
                    float v[8];
                    load8(base, g, cross, join, v);
                    finish8(a, m, 8 * g, cur.n, row, v);
                }
            } else {
                // group g of 8 columns is finished by rank (g / 2) % ks, which receives the other ranks' sums
                const int per = (a.tile_n / 16 + ks - 1) / ks * 2;
                if (item > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&m->red_empty), (item - 1) & 1, abort, fault));
                    if (!ok) continue;
                }
                for (int g = side; g < n8; g += 2) {
                    const int to = (g >> 1) % ks;
                    if (to == rank) continue;
                    float v[8];
                    load8(base, g, cross, join, v);
                    const int from = rank - (rank > to ? 1 : 0), at = (g >> 1) / ks * 2 + side;
                    const uint32_t dst = map_shared_rank(red_addr + (uint32_t)(((from * per + at) * 8 * kTileRows + my_row) * 4), (uint32_t)to);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_cluster_f32(dst + j * (kTileRows * 4), v[j]);
                }
                __syncwarp();
                if (lane < ks && lane != rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_full), (uint32_t)lane));
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&m->red_full), item & 1, abort, fault));
                if (!ok) continue;
                for (int g = 2 * rank + side; g < n8; g += 2 * ks) {
                    float v[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    load8(base, g, cross, join, v);
                    const int at = (g >> 1) / ks * 2 + side;
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
                    finish8(a, m, 8 * g, cur.n, row, o);
                }
                __syncwarp();
                if (lane < ks && lane != rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_empty), (uint32_t)lane));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&m->acc_empty[acc & 1]));
            ++acc;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.ksplit > 1) cluster_sync();
    if (warp == kWarpMma) tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
}

// ------------------------------------------------------------------ prepare

constexpr int kSelfPlan = 1024;         // slots up to which every block finds its own places (one launch less)
constexpr int kDownTokens = 16;         // tokens of an adapter block at most

struct PrepArgs {
    const void *x;
    int dtype;
    long long cols;
    int x_rows, copies;             // each row of x goes to `copies` slots
    int x_per_slot;
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
    int n_tokens, rank, list_blocks, down_tokens, down_split;
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

// One block: counts the experts' slots, cuts each expert's slots into tiles of tokens, and (place) gives every slot its
// place.  The order within an expert is whatever the counters give; an output does not depend on it.
template <int THREADS>
__device__ void plan_slots(const PrepArgs &a, int *count, bool place) {
    __shared__ int red[32];
    for (int e = threadIdx.x; e < a.n_mats; e += THREADS) count[e] = 0;
    __syncthreads();
    for (int s0 = 0; s0 < a.n_slots; s0 += 4 * THREADS) {
        int e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { const int s = s0 + i * THREADS + threadIdx.x; e[i] = s < a.n_slots ? a.ids[s] : -1; }
#pragma unroll
        for (int i = 0; i < 4; ++i) if (e[i] >= 0 && e[i] < a.n_mats) atomicAdd(&count[e[i]], 1);
    }
    __syncthreads();
    int base_n = 0, base_t = 0;
    for (int e0 = 0; e0 < a.n_mats; e0 += THREADS) {
        const int e = e0 + threadIdx.x;
        const int n = e < a.n_mats ? count[e] : 0;
        int size = 0, nt = 0;
        if (n) {
            nt = (n + a.tile_n - 1) / a.tile_n;
            size = round16((n + nt - 1) / nt);
            nt = (n + size - 1) / size;
        }
        int all_n, all_t;
        const int at = base_n + block_scan<THREADS>(n, red, &all_n);
        const int tile = base_t + block_scan<THREADS>(nt, red, &all_t);
        const int we = n ? a.w_exp[e] : 0;
        for (int i = 0; i < nt; ++i) a.tiles[tile + i] = TileRec{e, at + i * size, min(size, n - i * size), we};
        if (e < a.n_mats) count[e] = at;
        base_n += all_n;
        base_t += all_t;
    }
    if (threadIdx.x == 0) *a.n_tiles = base_t;
    if (!place) return;
    __syncthreads();
    for (int s0 = 0; s0 < a.n_slots; s0 += 4 * THREADS) {
        int e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { const int s = s0 + i * THREADS + threadIdx.x; e[i] = s < a.n_slots ? a.ids[s] : -1; }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + i * THREADS + threadIdx.x;
            if (s >= a.n_slots) continue;
            const bool ok = e[i] >= 0 && e[i] < a.n_mats;
            const int at = ok ? atomicAdd(&count[e[i]], 1) : -1;
            a.pos[s] = at;
            if (ok) a.order[at] = s;
            else atomicOr(a.fault, kFaultExpertId);
        }
    }
}

__global__ void __launch_bounds__(1024) plan_kernel(PrepArgs a) {
    extern __shared__ int count[];
    griddep_launch_dependents();
    griddep_wait();
    plan_slots<1024>(a, count, true);
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

__device__ __forceinline__ void load8x(const void *x, long long i, int dtype, float (&v)[8]) {
    if (dtype == HQ_DT_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (dtype == HQ_DT_BF16) {
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
        for (int c = 0; c < a.copies; ++c) {
            const int slot = r * a.copies + c;
            int at = slot;
            if (a.ids) {
                if (a.pos) {
                    at = live ? a.pos[slot] : -1;
                } else {
                    // few slots: the place is the number of slots that sort before this one
                    const int id = live ? a.ids[slot] : -1;
                    int before = 0;
                    for (int s = tr; s < a.n_slots; s += a.row_threads) {
                        const int o = a.ids[s];
                        before += o >= 0 && (o < id || (o == id && s < slot)) ? 1 : 0;
                    }
                    at = row_sum(before, a.row_threads, redi);
                    if (id < 0 || id >= a.n_mats) {
                        at = -1;
                        if (live && tr == 0) atomicOr(a.fault, kFaultExpertId);
                    } else if (tr == 0) {
                        a.order[at] = slot;
                    }
                }
            }
            if (!live) continue;
            if (at < 0) {
                for (long long j = tr; j < a.y_cols; j += a.row_threads)
                    store_elem(a.y, (long long)slot * a.y_cols + j, a.y_dtype, __int_as_float(0x7fc00000));
                continue;
            }
            if (a.x_exp && tr == 0) a.x_exp[at] = e;
            for (long long j = 8 * tr; j < a.cols; j += 8 * a.row_threads) {
                float v[8];
                uint32_t h[4], l[4];
                load8x(a.x, base + j, a.dtype, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f0 = v[2 * k] * s1 * s2, f1 = v[2 * k + 1] * s1 * s2;
                    const __half2 p = __floats2half2_rn(f0, f1);
                    h[k] = *reinterpret_cast<const uint32_t *>(&p);
                    // the rest of an infinity or a NaN is nothing
                    const float g0 = f0 - __low2float(p), g1 = f1 - __high2float(p);
                    const __half2 q = __floats2half2_rn(fabsf(f0) < INFINITY ? g0 : 0.f, fabsf(f1) < INFINITY ? g1 : 0.f);
                    l[k] = *reinterpret_cast<const uint32_t *>(&q);
                }
                *reinterpret_cast<uint4 *>(a.hi + (long long)at * a.cols + j) = make_uint4(h[0], h[1], h[2], h[3]);
                if (a.lo) *reinterpret_cast<uint4 *>(a.lo + (long long)at * a.cols + j) = make_uint4(l[0], l[1], l[2], l[3]);
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

// u[t][k] = scale A[adapter][k] . x[t] for a group of 8 NT tokens: each distinct adapter of the group times all its
// tokens, of which its own are kept.  x is one (bf16), two (f16) or three (f32) bf16 terms, exactly.  The columns
// are split over the warps and a cluster; their order inside a product is a lane's own (8 neighbours a
// lane), the same for both operands.
template <int DT, int NT>
__device__ void adapter_down(const PrepArgs &a, int group) {
    constexpr int TERMS = DT == HQ_DT_BF16 ? 1 : DT == HQ_DT_F16 ? 2 : 3, N = 8 * NT, WARPS = kPrepThreads / 32;
    extern __shared__ float part[];                         // [WARPS][16 mt][N], then [down_split][16 mt][N]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int mt = (a.rank + 15) / 16, vals = mt * 16 * N;
    float *joined = part + WARPS * vals;
    const int t0 = group * N, crank = a.down_split > 1 ? (int)cluster_ctarank() : 0;
    const int units = (int)(a.cols / 32);
    const int u_lo = (int)((long long)units * crank / a.down_split), u_hi = (int)((long long)units * (crank + 1) / a.down_split);
    const int id = lane < N && t0 + lane < a.n_tokens ? a.adapter_ids[t0 + lane] : -1;
    uint32_t left = __ballot_sync(0xffffffffu, id >= 0 && id < a.n_adapters);
    while (left) {
        const int ad = __shfl_sync(0xffffffffu, id, __ffs(left) - 1);
        const uint32_t mine = __ballot_sync(0xffffffffu, id == ad);
        left &= ~mine;
        float acc[4][NT][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        const uint16_t *A = a.A + (long long)ad * a.rank * a.cols;
        for (int un = u_lo + warp; un < u_hi; un += WARPS) {
            const long long col = un * 32ll + c * 8;
            uint32_t b[NT][TERMS][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int t = t0 + 8 * n + g;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if ((mine >> (8 * n + g)) & 1) load8x(a.x, (long long)t * a.cols + col, DT, v);
#pragma unroll
                for (int i = 0; i < TERMS; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                        b[n][i][k] = *reinterpret_cast<const uint32_t *>(&h);
                        v[2 * k] -= __low2float(h);
                        v[2 * k + 1] -= __high2float(h);
                    }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m < mt) {
                    const int r = 16 * m + g;
                    uint4 p = make_uint4(0, 0, 0, 0), q = make_uint4(0, 0, 0, 0);
                    if (r < a.rank) p = *reinterpret_cast<const uint4 *>(A + r * a.cols + col);
                    if (r + 8 < a.rank) q = *reinterpret_cast<const uint4 *>(A + (r + 8) * a.cols + col);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < TERMS; ++i) {
                            mma_bf16(acc[m][n], p.x, q.x, p.y, q.y, b[n][i][0], b[n][i][1]);
                            mma_bf16(acc[m][n], p.z, q.z, p.w, q.w, b[n][i][2], b[n][i][3]);
                        }
                }
            }
        }
        __syncthreads();                                    // the last adapter's sums are read
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (m < mt) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part[warp * vals + (16 * m + g + (i >> 1) * 8) * N + 8 * n + 2 * c + (i & 1)] = acc[m][n][i];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < vals; i += kPrepThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += part[w * vals + i];
            if (a.down_split > 1) st_shared_cluster_f32(map_shared_rank(smem_u32(joined + crank * vals + i), 0), s);
            else joined[i] = s;
        }
        if (a.down_split > 1) cluster_sync(); else __syncthreads();
        if (crank == 0) {
            const float scale = a.scales[ad];
            for (int i = threadIdx.x; i < vals; i += kPrepThreads) {
                const int k = i / N, t = i % N;
                float s = 0.f;
                for (int r = 0; r < a.down_split; ++r) s += joined[r * vals + i];
                if (((mine >> t) & 1) && k < a.rank) a.u[(long long)(t0 + t) * a.rank + k] = scale * s;
            }
        }
        if (a.down_split > 1) cluster_sync();
    }
}

__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(const __grid_constant__ PrepArgs a) {
    extern __shared__ float dyn[];
    griddep_launch_dependents();
    griddep_wait();
    int b = blockIdx.x;
    if (b < a.plan_blocks) { plan_slots<kPrepThreads>(a, reinterpret_cast<int *>(dyn), false); return; }
    b -= a.plan_blocks;
    if (b < a.pack_blocks) { pack_rows(a, b); return; }
    b -= a.pack_blocks;
    if (b < a.list_blocks) { if (b * (long long)a.tile_n < a.n_tokens) list_tile(a, b); return; }
    b = (b - a.list_blocks) / a.down_split;
    if (b * (long long)a.down_tokens >= a.n_tokens) return;
    if (a.down_tokens == 8) {
        if (a.dtype == HQ_DT_BF16) adapter_down<HQ_DT_BF16, 1>(a, b);
        else if (a.dtype == HQ_DT_F16) adapter_down<HQ_DT_F16, 1>(a, b);
        else adapter_down<HQ_DT_F32, 1>(a, b);
    } else {
        if (a.dtype == HQ_DT_BF16) adapter_down<HQ_DT_BF16, 2>(a, b);
        else if (a.dtype == HQ_DT_F16) adapter_down<HQ_DT_F16, 2>(a, b);
        else adapter_down<HQ_DT_F32, 2>(a, b);
    }
}

// y[t][i] = sum_k router_w[t][k] part[t][k][i], V columns a thread
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

hq_status encode(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t outer,
                 uint64_t stride, uint32_t box_inner, uint32_t box_outer, bool swizzle) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!enc) return set_error(HQ_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {stride};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
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

struct TcPlan { int tile_n, ksplit, grid, raw_slots, tmem_cols; size_t smem; uint32_t off_x, off_raw, off_red, off_meta; };

// Memory of a launch with tiles of p->tile_n tokens and the columns split over p->ksplit CTAs; false if it does not fit.
bool fit_smem(const DeviceInfo &dev, int fmt, bool split, TcPlan *p) {
    const int terms = split ? 2 : 1;
    const int chunk = (fmt == 8 ? Fmt<8>::kChunk : Fmt<4>::kChunk) * kTileRows;
    const int per = (p->tile_n / 16 + p->ksplit - 1) / p->ksplit * 2;
    const size_t red = p->ksplit > 1 ? (size_t)(p->ksplit - 1) * per * 8 * kTileRows * 4 : 0;
    const size_t fixed = (size_t)kSlots * (kABytes + p->tile_n * 128) * terms + red + sizeof(Meta) + 128;
    const size_t room = (size_t)dev.max_smem_optin;
    if (fixed + chunk > room) return false;
    p->raw_slots = (int)std::min<size_t>(kMaxRaw, (room - fixed) / chunk);
    uint32_t at = (uint32_t)(kSlots * kABytes * terms);
    p->off_x = at;
    at += (uint32_t)(kSlots * p->tile_n * 128 * terms);
    p->off_raw = at;
    at += (uint32_t)(p->raw_slots * chunk);
    p->off_red = at;
    at += (uint32_t)red;
    p->off_meta = (at + 127) & ~127u;
    p->smem = p->off_meta + sizeof(Meta);
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
            // cycles of 64 columns: the products, or decode and the weights' share of the memory bandwidth
            const double stage = std::max<double>(split ? 9.0 * std::max(tn, 32) : 2.2 * tn, 380.0);
            const double end = 1500.0 + 16.0 * tn + (ks > 1 ? 1500.0 + 12.0 * tn : 0.0);
            const double time = waves * (stage * 4 * ((n_chunks + ks - 1) / ks)) + end * (1 + 0.15 * (waves - 1));
            if (!any || time < best_t) { any = true; best_t = time; *best = p; }
        }
    }
    if (!any) return false;
    best->tmem_cols = 32;
    while (best->tmem_cols < best->tile_n * (split ? 5 : 2)) best->tmem_cols *= 2;
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

template <int FMT, bool SPLIT>
hq_status launch_tc(const TcArgs &t, const TcPlan &p, cudaStream_t stream) {
    auto kern = matmul_tc_kernel<FMT, SPLIT>;
    hq_status st = configure<matmul_tc_kernel<FMT, SPLIT>>(232448);
    return st != HQ_OK ? st : launch(kern, p.grid, kThreads, p.smem, p.ksplit, stream, "matmul", t);
}

}  // namespace

int64_t matmul_workspace(const MatmulArgs &a) { return layout(a).total; }

hq_status launch_matmul(const MatmulArgs &a, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    const Layout l = layout(a);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const bool split = a.dtype == HQ_DT_F32;
    const int64_t slots = a.n_tokens * a.n_active, n_rt = (a.rows + kTileRows - 1) / kTileRows;
    if (most_tiles(a) * n_rt > 0x7fffffffLL)
        return set_error(HQ_ERR_SHAPE, "more than 2^31 tiles");
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
            st = launch(plan_kernel, 1, 1024, (size_t)a.n_mats * 4, 1, stream, "plan", q);
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
        // 8 tokens a block while the blocks are few, and a cluster of blocks over the columns to fill the device
        q.down_tokens = a.n_tokens <= 512 ? 8 : kDownTokens;
        const int64_t tg = (a.n_tokens + q.down_tokens - 1) / q.down_tokens;
        while (q.down_split < 8 && tg * q.down_split * 2 <= 2 * dev->num_sms && a.cols / 32 / (q.down_split * 2) >= 16) q.down_split *= 2;
        const int ks = q.down_split;
        q.pack_blocks = (q.pack_blocks + ks - 1) / ks * ks;
        q.list_blocks = (int)(((a.n_tokens + p.tile_n - 1) / p.tile_n + ks - 1) / ks * ks);
        down_blocks = (int)tg * ks;
        prep_smem = (size_t)(kPrepThreads / 32 + ks) * ((a.rank + 15) / 16 * 16) * q.down_tokens * 4;
    }
    const int prep_grid = q.plan_blocks + q.pack_blocks + q.list_blocks + down_blocks;
    if (prep_grid > 0) {
        st = configure<prepare_kernel>(160 * 1024);
        if (st != HQ_OK) return st;
        st = launch(prepare_kernel, prep_grid, kPrepThreads, prep_smem, q.down_split, stream, "prepare", q);
        if (st != HQ_OK) return st;
    }

    TcArgs t = {};
    st = encode(&t.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.W, (uint64_t)n_chunks * chunk / 2, (uint64_t)(a.n_mats * a.rows),
                (uint64_t)n_chunks * chunk, (uint32_t)chunk / 2, kTileRows, false);
    const void *xh = pack ? (const void *)(ws + l.hi) : a.x;
    auto encode_x = [&](CUtensorMap *m, const void *base, uint32_t box) {
        if (st == HQ_OK)
            st = encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, (uint64_t)a.cols, (uint64_t)slots, (uint64_t)a.cols * 2, 64, box, true);
    };
    encode_x(&t.map_x64, xh, 64);
    encode_x(&t.map_x16, xh, 16);
    if (split) {
        encode_x(&t.map_lo64, ws + l.lo, 64);
        encode_x(&t.map_lo16, ws + l.lo, 16);
    }
    if (st != HQ_OK) return st;
    t.w_exp = a.w_exp;
    t.x_exp = q.x_exp;
    t.order = q.order;
    t.tiles = q.tiles;
    t.n_tiles = q.n_tiles;
    t.tile_count = q.tile_count;
    t.tile_list = q.tile_list;
    t.place = q.place;
    t.B = a.B;
    t.u = q.u;
    t.rank = a.rank;
    t.y = a.moe ? q.y : a.y;
    t.fault = dev->fault;
    t.rows = a.rows;
    t.n_tokens = (int)a.n_tokens;
    t.n_tt = (int)((a.n_tokens + p.tile_n - 1) / p.tile_n);
    t.n_rt = (int)n_rt;
    t.n_items = (int)((a.moe ? most_tiles(a) : t.n_tt) * n_rt);
    t.n_chunks = n_chunks;
    t.tile_n = p.tile_n;
    t.raw_slots = p.raw_slots;
    t.ksplit = p.ksplit;
    t.tmem_cols = p.tmem_cols;
    t.dtype = a.epilogue == HQ_MOE_EPI_COMBINE ? HQ_DT_F32 : a.dtype;
    t.epilogue = a.epilogue == HQ_MOE_EPI_SWIGLU ? HQ_MOE_EPI_SWIGLU : 0;
    t.stream_w = !a.moe && t.n_tt == 1;
    t.off_x = p.off_x;
    t.off_raw = p.off_raw;
    t.off_red = p.off_red;
    t.off_meta = p.off_meta;
    st = a.fmt == 8 ? (split ? launch_tc<8, true>(t, p, stream) : launch_tc<8, false>(t, p, stream))
                    : (split ? launch_tc<4, true>(t, p, stream) : launch_tc<4, false>(t, p, stream));
    if (st != HQ_OK) return st;
    if (a.epilogue == HQ_MOE_EPI_COMBINE) {
        const bool four = a.rows % 4 == 0;
        const int grid = (int)std::min<int64_t>((a.n_tokens * a.rows / (four ? 4 : 1) + 255) / 256, dev->num_sms * 16);
        st = launch(four ? combine_kernel<4> : combine_kernel<1>, grid, 256, 0, 1, stream, "combine",
                    (const float *)(ws + l.part), a.router_w, a.y, (long long)a.n_tokens, a.n_active, (long long)a.rows, a.dtype);
    }
    return st;
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
