// hq_matmul.cu -- products of many tokens with quantized weights on the tensor
// cores: grouped by expert, or shared with an adapter per request.
//
//   y[s][i] = sum_j w[m(s)][i][j] x[s][j],  w = d q (Q8_0) or d (n - 8) (Q4_0)
//
// A prepare kernel lays the call out, then one persistent kernel multiplies:
//  * The weights are the M operand (128 rows of W a tile) and the tokens the N
//    operand (16 to 256 a tile), so ragged groups of tokens cost what they are.
//  * Raw blocks come by TMA (256 columns of 128 rows a stage); sixteen warps
//    decode them to 16-bit floats in the swizzled layout the tensor core reads;
//    group q of four warps owns quarter q of every stage (64 columns) and
//    operand slot q, so the four groups work on a stage at once.
//  * Tokens come by TMA: a tiled load, or four gathered rows an instruction
//    where an expert's tokens are scattered.
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

#include "hq_internal.h"
#include "hq_tc.cuh"

namespace hq {
namespace {

// ------------------------------------------------------------------ shared with the host

constexpr int kTileRows = 128;
constexpr int kMaxTokens = 256;             // tokens of a tile
constexpr int kMaxTokensSplit = 64;         // f32: twice the operands, five accumulators
constexpr int kASlots = 4;                  // one per decode group
constexpr int kABytes = kTileRows * 128;
constexpr int kEpiWarps = 4, kDecodeWarps = 16;
constexpr int kWarpW = kEpiWarps + kDecodeWarps, kWarpX = kWarpW + 1, kWarpMma = kWarpX + 1;
constexpr int kThreads = 32 * (kWarpMma + 1);
constexpr int kPrepThreads = 512;
constexpr int kMaxRaw = 4, kMaxX = 8;

template <int FMT> struct Fmt;
template <> struct Fmt<8> { static constexpr int kChunk = 272, kVecs = 5; };   // bytes of 8 blocks; 16-byte units a quarter touches
template <> struct Fmt<4> { static constexpr int kChunk = 144, kVecs = 3; };

// One tile of tokens of one expert: sorted slots [start, start + n); tiles
// [first, first + count) are the expert's.
struct TileRec { int mat, start, n, first, count, pad0, pad1, pad2; };

struct TcArgs {
    CUtensorMap map_w, map_x, map_xlo;
    const int32_t *w_exp;
    const int32_t *x_exp;           // [token rows], or NULL: 0
    const int32_t *order;           // sorted slot ids, or NULL: slot = token
    const TileRec *tiles;
    const int32_t *n_tiles;         // device count (grouped)
    const int32_t *adapter_ids;     // or NULL
    const uint16_t *B;
    const float *u;                 // [n_tokens][rank_pad], scaled
    long long n_adapters;
    void *y;
    uint32_t *fault;
    long long rows;
    int n_tokens, n_tt, n_items, n_rt, n_chunks, x_div;      // x row = slot / x_div
    int tile_n, x_slots, raw_slots, ksplit, tmem_cols;
    int dtype, epilogue, rank, rank_pad, stream_w;
    uint32_t zero;                  // 0, unknown to the compiler
    uint32_t off_x, off_raw, off_red, off_meta;
};

struct Meta {
    uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw], x_full[kMaxX], x_empty[kMaxX], a_full[kASlots], a_empty[kASlots];
    uint64_t acc_full[2], acc_empty[2], red_full, red_empty, done;
    uint32_t tmem;
    int abort;
    int slot[kMaxTokens], adapter[kMaxTokens];
    float2 scale[kMaxTokens];
};

struct Item { int mat, rt, start, n; };

__device__ __forceinline__ Item get_item(const TcArgs &a, int w) {
    Item t;
    if (a.tiles) {
        const TileRec r = a.tiles[w / a.n_rt];
        const int local = w - r.first * a.n_rt;
        t.rt = local / r.count;
        const TileRec s = a.tiles[r.first + local % r.count];
        t.mat = s.mat;
        t.start = s.start;
        t.n = s.n;
    } else {
        t.mat = 0;
        t.rt = w / a.n_tt;
        t.start = w % a.n_tt * a.tile_n;
        t.n = min(a.tile_n, a.n_tokens - t.start);
    }
    return t;
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

// v[j] += sum_k B[adapter][row][k] u[token][k] for the 8 columns from c0; equal adapters next to
// each other share the row of B.
__device__ __forceinline__ void add_adapters(const TcArgs &a, const Meta *m, int c0, int n, long long row, float (&v)[8]) {
    int j = 0;
    while (j < 8 && c0 + j < n) {
        const int ad = m->adapter[c0 + j];
        int end = j + 1;
        while (end < 8 && c0 + end < n && m->adapter[c0 + end] == ad) ++end;
        if (ad < -1 || ad >= a.n_adapters) {
            if (threadIdx.x == 0) atomicOr(a.fault, kFaultAdapterId);
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i >= j && i < end) v[i] = __int_as_float(0x7fc00000);
        } else if (ad >= 0) {
            const uint16_t *b = a.B + ((long long)ad * a.rows + min(row, a.rows - 1)) * a.rank;
            for (int k0 = 0; k0 < a.rank_pad; k0 += 8) {
                float bv[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) bv[k] = k0 + k < a.rank ? __uint_as_float((uint32_t)b[k0 + k] << 16) : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i >= j && i < end) {
                        const float4 *u = reinterpret_cast<const float4 *>(a.u + (long long)m->slot[c0 + i] * a.rank_pad + k0);
                        const float4 p = u[0], q = u[1];
                        float t = v[i];
                        t = fmaf(bv[0], p.x, t); t = fmaf(bv[1], p.y, t); t = fmaf(bv[2], p.z, t); t = fmaf(bv[3], p.w, t);
                        t = fmaf(bv[4], q.x, t); t = fmaf(bv[5], q.y, t); t = fmaf(bv[6], q.z, t); t = fmaf(bv[7], q.w, t);
                        v[i] = t;
                    }
                }
            }
        }
        j = end;
    }
}

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }

// The 8 columns from c0 of output row `row` (its sums in v): scales, adapter
// term, SwiGLU with the neighbouring lane's row, store.
__device__ __forceinline__ void finish8(const TcArgs &a, const Meta *m, int c0, int n, long long row, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 s = m->scale[min(c0 + j, n - 1)];
        v[j] = v[j] * s.x * s.y;
    }
    if (a.adapter_ids) add_adapters(a, m, c0, n, row, v);
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

// ------------------------------------------------------------------ the kernel

template <int FMT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) matmul_tc_kernel(const __grid_constant__ TcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Meta *m = reinterpret_cast<Meta *>(smem + a.off_meta);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kTerms = SPLIT ? 2 : 1;
    const uint32_t rank = a.ksplit > 1 ? cluster_ctarank() : 0;
    const uint32_t a_base = smem_u32(smem), x_base = a_base + a.off_x, raw_base = a_base + a.off_raw;
    const int x_bytes = a.tile_n * 128;
    volatile int *abort = &m->abort;
    uint32_t *fault = a.fault;

    if (threadIdx.x == 0) {
        m->abort = 0;
        for (int i = 0; i < a.raw_slots; ++i) { mbar_init(smem_u32(&m->raw_full[i]), 1); mbar_init(smem_u32(&m->raw_empty[i]), kDecodeWarps); }
        for (int i = 0; i < a.x_slots; ++i) { mbar_init(smem_u32(&m->x_full[i]), 1); mbar_init(smem_u32(&m->x_empty[i]), 1); }
        for (int i = 0; i < kASlots; ++i) { mbar_init(smem_u32(&m->a_full[i]), 4); mbar_init(smem_u32(&m->a_empty[i]), 1); }
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
    // dense weights may be fetched before the prepare kernel is done; everything else waits for it
    if (a.tiles || warp != kWarpW) griddep_wait();
    const int n_items = a.tiles ? *a.n_tiles * a.n_rt : a.n_items;

    if (warp == kWarpW) {
        if (lane == 0) {
            const uint64_t pol = a.stream_w ? l2_evict_first_policy() : l2_evict_normal_policy();
            uint32_t it = 0;
            bool ok = true;
            for (int w = first; w < n_items && ok; w += step) {
                const Item t = get_item(a, w);
                const int row0 = (int)((long long)t.mat * a.rows + (long long)t.rt * kTileRows);
                for (int c = c_lo; c < c_hi && ok; ++c, ++it) {
                    const uint32_t s = it % a.raw_slots, ph = (it / a.raw_slots) & 1;
                    ok = mbar_wait(smem_u32(&m->raw_empty[s]), ph ^ 1, abort, fault);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&m->raw_full[s]);
                    mbar_arrive_expect_tx(bar, kTileRows * Fmt<FMT>::kChunk);
                    tma_load_2d(raw_base + s * (kTileRows * Fmt<FMT>::kChunk), &a.map_w, c * (Fmt<FMT>::kChunk / 2), row0, bar, pol);
                }
            }
            // copies in flight end before the block's memory is given back
            for (uint32_t k = it > (uint32_t)a.raw_slots ? it - a.raw_slots : 0; !ok && k < it; ++k)
                for (int tries = 0; tries < 1 << 16 && !mbar_try_wait(smem_u32(&m->raw_full[k % a.raw_slots]), (k / a.raw_slots) & 1); ++tries) {}
        }
    } else if (warp == kWarpX) {
        uint32_t it = 0;
        bool ok = true;
        for (int w = first; w < n_items && ok; w += step) {
            const Item t = get_item(a, w);
            const int groups = (t.n + 3) / 4;
            int4 r[2];
            if (a.order) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = a.order[t.start + min((lane + 32 * h) * 4 + i, t.n - 1)] / a.x_div;
                    r[h] = make_int4(v[0], v[1], v[2], v[3]);
                }
            }
            for (int k = 4 * c_lo; k < 4 * c_hi && ok; ++k, ++it) {
                const uint32_t s = it % a.x_slots, ph = (it / a.x_slots) & 1;
                ok = mbar_wait(smem_u32(&m->x_empty[s]), ph ^ 1, abort, fault);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t bar = smem_u32(&m->x_full[s]);
                const uint32_t dst = x_base + s * (kTerms * x_bytes);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(kTerms * (a.order ? groups * 512 : x_bytes)));
                __syncwarp();
                if (a.order) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = lane + 32 * h;
                        if (g < groups) {
                            tma_gather4(dst + g * 512, &a.map_x, k * 64, r[h], bar);
                            if constexpr (SPLIT) tma_gather4(dst + x_bytes + g * 512, &a.map_xlo, k * 64, r[h], bar);
                        }
                    }
                } else if (lane == 0) {
                    const uint64_t pol = l2_evict_normal_policy();
                    tma_load_2d(dst, &a.map_x, k * 64, t.start, bar, pol);
                    if constexpr (SPLIT) tma_load_2d(dst + x_bytes, &a.map_xlo, k * 64, t.start, bar, pol);
                }
            }
        }
        for (uint32_t k = it > (uint32_t)a.x_slots ? it - a.x_slots : 0; !ok && k < it; ++k)
            for (int tries = 0; tries < 1 << 16 && !mbar_try_wait(smem_u32(&m->x_full[k % a.x_slots]), (k / a.x_slots) & 1); ++tries) {}
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            uint32_t it = 0, acc = 0;
            bool ok = true;
            const uint32_t half = SPLIT ? 2u * a.tile_n : (uint32_t)a.tmem_cols / 2;
            for (int w = first; w < n_items && ok; w += step) {
                const Item t = get_item(a, w);
                const int n16 = round16(t.n);
                const uint32_t idesc = tc_idesc_f16(n16);
                for (int k = 4 * c_lo; k < 4 * c_hi && ok; ++k, ++it) {
                    const bool fresh = SPLIT ? (k & 3) == 0 : k == 4 * c_lo;
                    if (fresh) {
                        ok = mbar_wait(smem_u32(&m->acc_empty[acc & 1]), ((acc >> 1) & 1) ^ 1, abort, fault);
                        if (!ok) break;
                    }
                    const uint32_t sa = it % kASlots, sx = it % a.x_slots;
                    ok = mbar_wait(smem_u32(&m->x_full[sx]), (it / a.x_slots) & 1, abort, fault) &&
                         mbar_wait(smem_u32(&m->a_full[sa]), (it / kASlots) & 1, abort, fault);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (acc & 1) * half;
                    const uint64_t da = tc_desc_sw128(a_base + sa * (kTerms * kABytes));
                    const uint64_t db = tc_desc_sw128(x_base + sx * (kTerms * x_bytes));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        tc_mma_f16(d, da + 2 * j, db + 2 * j, idesc, !(fresh && j == 0));
                        if constexpr (SPLIT) {
                            tc_mma_f16(d + a.tile_n, da + 2 * j, db + (x_bytes >> 4) + 2 * j, idesc, !(fresh && j == 0));
                            tc_mma_f16(d + a.tile_n, da + (kABytes >> 4) + 2 * j, db + 2 * j, idesc, true);
                        }
                    }
                    tc_commit(smem_u32(&m->a_empty[sa]));
                    tc_commit(smem_u32(&m->x_empty[sx]));
                    if (SPLIT ? (k & 3) == 3 : k == 4 * c_hi - 1) {
                        tc_commit(smem_u32(&m->acc_full[acc & 1]));
                        ++acc;
                    }
                }
            }
            // every product ends before TMEM is given back
            tc_commit(smem_u32(&m->done));
            for (int tries = 0; tries < 1 << 20 && !mbar_try_wait(smem_u32(&m->done), 0); ++tries) {}
        }
        __syncwarp();
    } else if (warp >= kEpiWarps) {
        const int q = (warp - kEpiWarps) >> 2, row = ((warp - kEpiWarps) & 3) * 32 + lane;
        constexpr int kUnit = FMT == 8 ? 64 : 32;           // 16-byte units where quarter q begins, in bytes per q
        const uint8_t *src = smem + a.off_raw + row * Fmt<FMT>::kChunk + q * kUnit;
        uint8_t *dst = smem + q * (kTerms * kABytes);
        uint32_t it = 0;
        bool ok = true;
        for (int w = first; w < n_items && ok; w += step) {
            const Item t = get_item(a, w);
            const float wscale = pow2(-a.w_exp[t.mat]);
            for (int c = c_lo; c < c_hi && ok; ++c, ++it) {
                const uint32_t s = it % a.raw_slots;
                ok = mbar_wait(smem_u32(&m->raw_full[s]), (it / a.raw_slots) & 1, abort, fault);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint32_t v[4 * Fmt<FMT>::kVecs];
                const uint4 *p = reinterpret_cast<const uint4 *>(src + s * (kTileRows * Fmt<FMT>::kChunk));
#pragma unroll
                for (int i = 0; i < Fmt<FMT>::kVecs; ++i) ld_shared_volatile(smem_u32(p + i), v + 4 * i);
                // The buffer goes back to the copy engine once its values are here.  The arrival
                // takes them as an operand (masked to nothing): an arrival alone does not wait for loads
                // in flight, and overtakes them when the load unit is busy.
                uint32_t seen = 0;
#pragma unroll
                for (int i = 0; i < Fmt<FMT>::kVecs; ++i) seen |= v[4 * i];
                seen = __reduce_or_sync(0xffffffffu, seen & a.zero);
                if (lane == 0) mbar_arrive_count(smem_u32(&m->raw_empty[s]), 1 + seen);
                ok = mbar_wait(smem_u32(&m->a_empty[q]), (it & 1) ^ 1, abort, fault);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (q == 0) decode_quarter<FMT, SPLIT, 0>(v, wscale, dst, row);
                else if (q == 1) decode_quarter<FMT, SPLIT, 1>(v, wscale, dst, row);
                else if (q == 2) decode_quarter<FMT, SPLIT, 2>(v, wscale, dst, row);
                else decode_quarter<FMT, SPLIT, 3>(v, wscale, dst, row);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&m->a_full[q]));
            }
        }
    } else {
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t half = SPLIT ? 2u * a.tile_n : (uint32_t)a.tmem_cols / 2;
        const uint32_t run = 4u * a.tile_n;                 // SPLIT: the running sums
        float *red = reinterpret_cast<float *>(smem + a.off_red);
        const uint32_t red_addr = smem_u32(red);
        uint32_t acc = 0, item = 0;
        bool ok = true;
        for (int w = first; w < n_items; w += step, ++item) {
            // the four warps leave together, and the last tile's columns are read
            if (!named_barrier_and(1, 32 * kEpiWarps, ok)) break;
            const Item t = get_item(a, w);
            const int n8 = round16(t.n) / 8;
            const long long row = (long long)t.rt * kTileRows + warp * 32 + lane;
            const int e_w = a.w_exp[t.mat];
            for (int j = threadIdx.x; j < t.n; j += 32 * kEpiWarps) {
                const int slot = a.order ? a.order[t.start + j] : t.start + j;
                const int e = e_w + (a.x_exp ? a.x_exp[slot / a.x_div] : 0);
                m->slot[j] = slot;
                m->scale[j] = make_float2(pow2(e / 2), pow2(e - e / 2));
                if (a.adapter_ids) m->adapter[j] = a.adapter_ids[slot];
            }
            named_barrier(1, 32 * kEpiWarps);
            auto load8 = [&](uint32_t base, int g, bool last, bool join, float (&v)[8]) {
                tmem_ld8(base + 8 * g, v);
                if constexpr (SPLIT) {
                    float x[8], r[8];
                    tmem_ld8(base + a.tile_n + 8 * g, x);
                    if (join) tmem_ld8(lane_base + run + 8 * g, r);
                    tmem_wait_ld(v);
                    tmem_wait_ld(x);
                    if (join) tmem_wait_ld(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] + x[j];
                    if (join) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += r[j];
                    }
                    if (!last) { tmem_st8(lane_base + run + 8 * g, v); }
                } else {
                    tmem_wait_ld(v);
                }
            };
            if constexpr (SPLIT) {
                for (int c = c_lo; c < c_hi - 1 && ok; ++c, ++acc) {
                    ok = mbar_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    for (int g = 0; g < n8; ++g) {
                        float v[8];
                        load8(lane_base + (acc & 1) * half, g, false, c > c_lo, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&m->acc_empty[acc & 1]));
                }
                if (!ok) continue;
            }
            ok = mbar_wait(smem_u32(&m->acc_full[acc & 1]), (acc >> 1) & 1, abort, fault);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            const uint32_t base = lane_base + (acc & 1) * half;
            const bool join = SPLIT && c_hi - c_lo > 1;
            if (a.ksplit == 1) {
                for (int g = 0; g < n8; ++g) {
                    float v[8];
                    load8(base, g, true, join, v);
                    finish8(a, m, 8 * g, t.n, row, v);
                }
            } else {
                // group g of 8 columns is finished by rank g % ksplit, which receives the other ranks' sums
                const int ks = a.ksplit, per = (a.tile_n / 8 + ks - 1) / ks;
                if (item > 0) {
                    ok = mbar_wait_cluster(smem_u32(&m->red_empty), (item - 1) & 1, abort, fault);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                }
                for (int g = 0; g < n8; ++g) {
                    const uint32_t to = (uint32_t)(g % ks);
                    if (to == rank) continue;
                    float v[8];
                    load8(base, g, true, join, v);
                    const int from = (int)rank - (rank > to ? 1 : 0);
                    const uint32_t at = map_shared_rank(red_addr + (uint32_t)(((from * per + g / ks) * 8 * kTileRows + warp * 32 + lane) * 4), to);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_cluster_f32(at + j * (kTileRows * 4), v[j]);
                }
                __syncwarp();
                if (lane < ks && lane != (int)rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_full), (uint32_t)lane));
                ok = mbar_wait_cluster(smem_u32(&m->red_full), item & 1, abort, fault);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                for (int g = (int)rank; g < n8; g += ks) {
                    float v[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    load8(base, g, true, join, v);
                    for (int r = 0; r < ks; ++r) {
                        if (r == (int)rank) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] += v[j];
                        } else {
                            const int from = r - (r > (int)rank ? 1 : 0);
                            const float *src = red + (from * per + g / ks) * 8 * kTileRows + warp * 32 + lane;
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] += src[j * kTileRows];
                        }
                    }
                    finish8(a, m, 8 * g, t.n, row, o);
                }
                __syncwarp();
                if (lane < ks && lane != (int)rank) mbar_arrive_remote(map_shared_rank(smem_u32(&m->red_empty), (uint32_t)lane));
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

struct PrepArgs {
    const void *x;
    __half *hi, *lo;                // lo: f32 only
    int32_t *x_exp;
    long long x_rows, cols;
    int dtype;
    // grouping
    const int32_t *ids;
    long long n_slots, n_mats;
    int tile_n;
    int32_t *order, *n_tiles;
    TileRec *tiles;
    void *y;                        // rows of slots whose id is out of range get NaN
    long long y_cols;
    int y_dtype;
    // adapters
    const int32_t *adapter_ids;
    const uint16_t *A;
    const float *scales;
    long long n_adapters, n_tokens;
    int rank, rank_pad;
    float *u;
    uint32_t *fault;
    int plan_blocks;                // 1: block 0 groups
    int pack_blocks;                // blocks that convert x
};

__device__ __forceinline__ float load_elem(const void *x, long long i, int dtype) {
    if (dtype == HQ_DT_F32) return static_cast<const float *>(x)[i];
    if (dtype == HQ_DT_F16) return __half2float(static_cast<const __half *>(x)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
}

// Sum of `v` over the threads before this one, and over all of them.
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
    int before = 0, total = 0;
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) before += red[w];
        total += red[w];
    }
    *all = total;
    return before + inc - v;
}

// One block: counts the experts' slots, lays them out expert after expert and
// cuts each expert's slots into tiles.  (The order within an expert is whatever the
// counters give; an output does not depend on it.)
__device__ void plan_block(const PrepArgs &a) {
    extern __shared__ int count[];                          // [n_mats]
    __shared__ int red[kPrepThreads / 32];
    __shared__ int carry[2];
    for (int e = threadIdx.x; e < a.n_mats; e += kPrepThreads) count[e] = 0;
    __syncthreads();
    for (long long s = threadIdx.x; s < a.n_slots; s += kPrepThreads) {
        const int e = a.ids[s];
        if (e >= 0 && e < a.n_mats) atomicAdd(&count[e], 1);
    }
    if (threadIdx.x == 0) carry[0] = carry[1] = 0;
    __syncthreads();
    for (long long e0 = 0; e0 < a.n_mats; e0 += kPrepThreads) {
        const long long e = e0 + threadIdx.x;
        const int n = e < a.n_mats ? count[e] : 0;
        int size = 0, nt = 0;
        if (n) {
            nt = (n + a.tile_n - 1) / a.tile_n;
            size = round16((n + nt - 1) / nt);
            nt = (n + size - 1) / size;
        }
        int all_n, all_t;
        const int at = carry[0] + block_scan(n, red, &all_n);
        const int tile = carry[1] + block_scan(nt, red, &all_t);
        for (int i = 0; i < nt; ++i) {
            TileRec r = {(int)e, at + i * size, min(size, n - i * size), tile, nt, 0, 0, 0};
            a.tiles[tile + i] = r;
        }
        if (e < a.n_mats) count[e] = at;
        __syncthreads();
        if (threadIdx.x == 0) { carry[0] += all_n; carry[1] += all_t; }
        __syncthreads();
    }
    if (threadIdx.x == 0) *a.n_tiles = carry[1];
    for (long long s = threadIdx.x; s < a.n_slots; s += kPrepThreads) {
        const int e = a.ids[s];
        if (e >= 0 && e < a.n_mats) {
            a.order[atomicAdd(&count[e], 1)] = (int)s;
        } else {
            atomicOr(a.fault, kFaultExpertId);
            for (long long i = 0; i < a.y_cols; ++i) store_elem(a.y, s * a.y_cols + i, a.y_dtype, __int_as_float(0x7fc00000));
        }
    }
}

// Rows of x to f16 terms, each row scaled so that its largest finite element
// lies in [2^13, 2^14).
__device__ void pack_row(const PrepArgs &a, long long r) {
    __shared__ float red[kPrepThreads / 32];
    const long long base = r * a.cols;
    float top = 0.f;
    for (long long j = threadIdx.x; j < a.cols; j += kPrepThreads) {
        const float v = fabsf(load_elem(a.x, base + j, a.dtype));
        if (v < INFINITY) top = fmaxf(top, v);
    }
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kPrepThreads / 32; ++w) top = fmaxf(top, red[w]);
    int e = 0;
    if (top > 0.f) { frexpf(top, &e); e -= 14; }
    if (threadIdx.x == 0) a.x_exp[r] = e;
    const float s1 = pow2(-(e / 2)), s2 = pow2(-(e - e / 2));
    for (long long j = threadIdx.x; j < a.cols; j += kPrepThreads) {
        const float v = load_elem(a.x, base + j, a.dtype) * s1 * s2;
        const __half h = __float2half_rn(v);
        a.hi[base + j] = h;
        if (a.lo) a.lo[base + j] = __hisinf(h) ? __float2half_rn(0.f) : __float2half_rn(v - __half2float(h));
    }
}

// u[t][k] = scale (A[adapter][k] . x[t]), zero for the padded ranks: one warp per value.
__device__ void adapter_down(const PrepArgs &a, long long o) {
    const long long t = o / a.rank_pad;
    const int k = (int)(o % a.rank_pad), lane = threadIdx.x & 31;
    const int ad = a.adapter_ids[t];
    if (ad < 0 || ad >= a.n_adapters) return;
    float s = 0.f;
    if (k < a.rank) {
        const uint16_t *A = a.A + ((long long)ad * a.rank + k) * a.cols;
        for (long long j = lane; j < a.cols; j += 32)
            s = fmaf(__uint_as_float((uint32_t)A[j] << 16), load_elem(a.x, t * a.cols + j, a.dtype), s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scales[ad];
    }
    if (lane == 0) a.u[o] = s;
}

__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(PrepArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    int b = blockIdx.x;
    if (b < a.plan_blocks) { plan_block(a); return; }
    b -= a.plan_blocks;
    if (b < a.pack_blocks) {
        for (long long r = b; r < a.x_rows; r += a.pack_blocks) pack_row(a, r);
        return;
    }
    b -= a.pack_blocks;
    const long long blocks = gridDim.x - a.plan_blocks - a.pack_blocks;
    for (long long o = b * (kPrepThreads / 32) + (threadIdx.x >> 5); o < a.n_tokens * a.rank_pad; o += blocks * (kPrepThreads / 32))
        adapter_down(a, o);
}

// y[t][i] = sum_k router_w[t][k] part[t][k][i]
__global__ void __launch_bounds__(256) combine_kernel(const float *part, const float *router_w, void *y, long long n_tokens,
                                                      int n_active, long long rows, int dtype) {
    griddep_launch_dependents();
    griddep_wait();
    for (long long o = blockIdx.x * 256ll + threadIdx.x; o < n_tokens * rows; o += gridDim.x * 256ll) {
        const long long t = o / rows, i = o % rows;
        float s = 0.f;
        for (int k = 0; k < n_active; ++k) s = fmaf(router_w[t * n_active + k], part[(t * n_active + k) * rows + i], s);
        store_elem(y, o, dtype, s);
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
    int64_t hi = 0, lo = 0, x_exp = 0, order = 0, n_tiles = 0, tiles = 0, part = 0, u = 0, total = 0;
};

int64_t x_rows(const MatmulArgs &a) { return a.moe && a.x_per_slot ? a.n_tokens * a.n_active : a.n_tokens; }
int rank_pad(const MatmulArgs &a) { return (a.rank + 7) / 8 * 8; }

Layout layout(const MatmulArgs &a) {
    Layout l;
    const int64_t slots = a.n_tokens * a.n_active;
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t p = at; at += up256(bytes); return p; };
    if (a.n_tokens == 0) return l;
    if (a.dtype != HQ_DT_F16) {
        l.hi = take(x_rows(a) * a.cols * 2);
        if (a.dtype == HQ_DT_F32) l.lo = take(x_rows(a) * a.cols * 2);
        l.x_exp = take(x_rows(a) * 4);
    }
    if (a.moe) {
        l.n_tiles = take(4);
        l.order = take(slots * 4);
        l.tiles = take((slots / 16 + std::min(slots, a.n_mats) + 1) * (int64_t)sizeof(TileRec));
        if (a.epilogue == HQ_MOE_EPI_COMBINE) l.part = take(slots * a.rows * 4);
    } else if (a.rank > 0) {
        l.u = take(a.n_tokens * rank_pad(a) * 4);
    }
    l.total = at;
    return l;
}

struct TcPlan { int tile_n, ksplit, grid, x_slots, raw_slots, tmem_cols; size_t smem; uint32_t off_x, off_raw, off_red, off_meta; };

// Memory of a launch with tiles of p->tile_n tokens and the columns split over p->ksplit CTAs; false if it does not fit.
bool fit_smem(const DeviceInfo &dev, int fmt, bool split, TcPlan *p) {
    const int terms = split ? 2 : 1;
    const int chunk = (fmt == 8 ? Fmt<8>::kChunk : Fmt<4>::kChunk) * kTileRows;
    const int per = (p->tile_n / 8 + p->ksplit - 1) / p->ksplit;
    const size_t red = p->ksplit > 1 ? (size_t)(p->ksplit - 1) * per * 8 * kTileRows * 4 : 0;
    const size_t fixed = (size_t)kASlots * kABytes * terms + red + sizeof(Meta) + 128;
    const size_t room = (size_t)dev.max_smem_optin;
    const size_t xb = (size_t)p->tile_n * 128 * terms;
    p->x_slots = 3;
    p->raw_slots = 1;
    if (fixed + p->x_slots * xb + chunk > room) return false;
    while (p->raw_slots < 3 && fixed + p->x_slots * xb + (size_t)(p->raw_slots + 1) * chunk <= room) ++p->raw_slots;
    while (p->x_slots < kMaxX && fixed + (p->x_slots + 1) * xb + (size_t)p->raw_slots * chunk <= room) ++p->x_slots;
    uint32_t at = (uint32_t)(kASlots * kABytes * terms);
    p->off_x = at;
    at += (uint32_t)(p->x_slots * xb);
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

template <int FMT, bool SPLIT>
hq_status launch_tc(const TcArgs &t, const TcPlan &p, cudaStream_t stream) {
    auto kern = matmul_tc_kernel<FMT, SPLIT>;
    static int configured[64] = {0};
    int d = 0;
    cudaGetDevice(&d);
    if (d < 0 || d >= 64 || !configured[d]) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        if (d >= 0 && d < 64) configured[d] = 1;
    }
    return launch(kern, p.grid, kThreads, p.smem, p.ksplit, stream, "matmul", t);
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
    if ((slots / 16 + std::min(slots, a.n_mats) + 1) * n_rt > 0x7fffffffLL)
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
    q.n_tokens = a.n_tokens;
    const bool pack = a.dtype != HQ_DT_F16;
    if (pack) {
        q.x_rows = x_rows(a);
        q.hi = reinterpret_cast<__half *>(ws + l.hi);
        q.lo = split ? reinterpret_cast<__half *>(ws + l.lo) : nullptr;
        q.x_exp = reinterpret_cast<int32_t *>(ws + l.x_exp);
        q.pack_blocks = (int)std::min<int64_t>(q.x_rows, dev->num_sms * 4);
    }
    if (a.moe) {
        q.plan_blocks = 1;
        q.ids = a.idx;
        q.n_slots = slots;
        q.n_mats = a.n_mats;
        q.tile_n = p.tile_n;
        q.order = reinterpret_cast<int32_t *>(ws + l.order);
        q.n_tiles = reinterpret_cast<int32_t *>(ws + l.n_tiles);
        q.tiles = reinterpret_cast<TileRec *>(ws + l.tiles);
        const bool comb = a.epilogue == HQ_MOE_EPI_COMBINE;
        q.y = comb ? ws + l.part : a.y;
        q.y_dtype = comb ? HQ_DT_F32 : a.dtype;
        q.y_cols = a.epilogue == HQ_MOE_EPI_SWIGLU ? a.rows / 2 : a.rows;
    }
    int down_blocks = 0;
    if (!a.moe && a.n_adapters > 0) {
        q.adapter_ids = a.idx;
        q.A = a.A;
        q.scales = a.scales;
        q.n_adapters = a.n_adapters;
        q.rank = a.rank;
        q.rank_pad = rank_pad(a);
        q.u = reinterpret_cast<float *>(ws + l.u);
        down_blocks = (int)std::min<int64_t>((a.n_tokens * q.rank_pad + 15) / 16, dev->num_sms * 4);
    }
    const int prep_grid = q.plan_blocks + q.pack_blocks + down_blocks;
    if (prep_grid > 0) {
        st = launch(prepare_kernel, prep_grid, kPrepThreads, a.moe ? (size_t)a.n_mats * 4 : 0, 1, stream, "prepare", q);
        if (st != HQ_OK) return st;
    }

    TcArgs t = {};
    st = encode(&t.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT16, a.W, (uint64_t)n_chunks * chunk / 2, (uint64_t)(a.n_mats * a.rows),
                (uint64_t)n_chunks * chunk, (uint32_t)chunk / 2, kTileRows, false);
    if (st != HQ_OK) return st;
    const void *xh = pack ? (const void *)(ws + l.hi) : a.x;
    const uint32_t box = a.moe ? 1u : (uint32_t)p.tile_n;
    st = encode(&t.map_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xh, (uint64_t)a.cols, (uint64_t)x_rows(a), (uint64_t)a.cols * 2, 64, box, true);
    if (st == HQ_OK && split)
        st = encode(&t.map_xlo, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws + l.lo, (uint64_t)a.cols, (uint64_t)x_rows(a), (uint64_t)a.cols * 2, 64, box, true);
    if (st != HQ_OK) return st;
    t.w_exp = a.w_exp;
    t.x_exp = q.x_exp;
    t.order = q.order;
    t.tiles = q.tiles;
    t.n_tiles = q.n_tiles;
    t.adapter_ids = q.adapter_ids;
    t.B = a.B;
    t.u = q.u;
    t.n_adapters = a.n_adapters;
    t.rank = a.rank;
    t.rank_pad = q.rank_pad;
    t.y = a.moe ? q.y : a.y;
    t.fault = dev->fault;
    t.rows = a.rows;
    t.n_tokens = (int)a.n_tokens;
    t.n_tt = (int)((a.n_tokens + p.tile_n - 1) / p.tile_n);
    t.n_rt = (int)n_rt;
    t.n_items = t.n_tt * t.n_rt;
    t.n_chunks = n_chunks;
    t.x_div = a.moe && !a.x_per_slot ? a.n_active : 1;
    t.tile_n = p.tile_n;
    t.x_slots = p.x_slots;
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
        const int grid = (int)std::min<int64_t>((a.n_tokens * a.rows + 255) / 256, dev->num_sms * 16);
        st = launch(combine_kernel, grid, 256, 0, 1, stream, "combine", (const float *)(ws + l.part), a.router_w, a.y,
                    (long long)a.n_tokens, a.n_active, (long long)a.rows, a.dtype);
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
