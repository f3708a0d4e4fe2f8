// hq_attention_tile.cu -- attention over the quantized key/value cache for many
// query rows a key/value head (prompts, wide groups of verified drafts), 16-bit
// tokens, on the tensor cores.
//
// A tile is 128 query rows (tokens with their group's heads), a unit 128 positions.  Per unit, with the shared memory of a block
// holding one tile of Q, K and V^T as 16-bit floats:
//   4 + 4 warps      the stored bytes, from global memory to registers, become K [128 positions][D] and V^T [D][128 positions]
//   1 thread         S = Q K^T and O += P V, tcgen05.mma with accumulators in tensor memory (P is an operand there)
//   4 softmax warps  a thread a row: maxima, weights into tensor memory, rescaling of O where the maximum has risen
//   1 walker warp    finds the parts and the addresses of their cells, and asks for them ahead into L2
// Two blocks a multiprocessor (D 256: one) fill each other's gaps.
//
// f16 tokens: K and V^T in two terms, units of 64 positions, whose second terms take the tiles' other half; the same weights meet both of V's.
// With one term f16 outputs were off by 3.9e-4 (Q4_0) to 6.9e-4 (Q8_0) of their norm, where their own rounding is 2.1e-4: keys 2.5 and 5.9, values 1.6 and
// 2.1, weights 1.7; with two by 2.9e-4.  bf16 outputs' own rounding is 1.7e-3, and one term stays.
//
// Measured: Q4_0, heads of 128, 4096 tokens behind 12289 positions, 32 on 8 heads (962 GFLOP): f16 1838 us, with one term 1131 us = 851 TFLOP/s, 44 % of what a
// large bf16 product reaches.  A prompt of 2011 tokens, Q8_0 (33 GFLOP): 126 us.  Bound by the chain of a unit, S, softmax, O: the weights take the
// place of the scores in tensor memory, so the next unit's S waits for O, and two blocks hide part of that (tensor pipe 36 % busy, issue slots
// 57 %).  The short prompt: 14 units a block, among them the start and end of two or three tiles, then 12 us of joins.  On the way, of these
// two: keys and values decoded by the same four warps 1843 and 332 us; tensor memory read 16 columns at a time 1670 and 303; hidden
// columns masked in the loop of all columns 1344 and 197; Q prepared by the softmax warps 1210 and 197; joins of eight groups a row 1167 and
// 152.  Not kept: units of 64 positions with scores and weights side by side, 1366 and 266 where this had 1344 and 201.
//
// Ranges.  Q rows are scaled as in the kernel for few rows.  K and V^T of 32 neighbouring positions are scaled by
// the power of two that takes their largest scale to the top of what 16 bits hold (2^-6 or 2^-2 for the largest element), so an element
// is rounded to 11 bits, or, where its scale is so far below that the offset's product is subnormal, to 2^-17 (Q4_0) or 2^-20 (Q8_0) of the
// largest near it: two roundings of half the finest step, 2^-25, of at least 2^-7 or 2^-3.  Scores of those 32 columns get K's power back in fp32; V's joins
// the exponent of the weights, whose reference is thus the largest weight times value, and the sum of the weights leaves it out.
#include <algorithm>
#include <atomic>

#include "hq_attention.cuh"
#include "hq_tc.cuh"

namespace hq {
namespace {

constexpr int kRows = 128, kTile = 128;                     // query rows, and rows of K (columns of V^T) that a tile holds
constexpr int kSoftmax = 4, kDecode = 4;                    // warps: softmax, then of keys, of values
constexpr int kValues = kSoftmax + kDecode, kWalker = kValues + kDecode, kProducts = kWalker + 1;
constexpr int kThreads = 32 * (kProducts + 1);
constexpr int kSlots = 4;                                   // units whose addresses are known ahead
constexpr float kSlack = 8.f, kWeight = 6.f;                // weights up to 2^(slack + weight); 2^weight at the reference

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const int a = min(max(lo, 0), 32), b = min(max(hi, a), 32);
    return (uint32_t)((1ull << b) - (1ull << a));
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }     // 2^e
__device__ __forceinline__ __half2 power_h2(int e) {        // 2^e, -14 <= e <= 15
    return __half2half2(__ushort_as_half((uint16_t)((15 + e) << 10)));
}

// D[128][N] (+)= A[128][16] B[N][16]^T, both in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// This warp's 32 lanes x 32 columns, waited for.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr) : "memory");
}
// 16 columns' pairs of 16-bit floats.
__device__ __forceinline__ void tmem_st8u(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(addr) : "memory");
}

// 16 bytes into shared memory, zeros without `live`; this thread's, waited for by copy_async_wait.
__device__ __forceinline__ void copy_async16(uint32_t to, const void *from, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Plain loads: the cells may have been written by the kernel in front of this one while this block was already there, which the wait at the
// start orders for plain loads, not for those of memory that nobody writes (times as before: 4096 tokens 1132 us).
template <int WORDS>
__device__ __forceinline__ void load_global(const uint8_t *p, uint32_t *v) {
    if constexpr (WORDS == 1) asm volatile("ld.global.u32 %0, [%1];" : "=r"(v[0]) : "l"(p));
    else if constexpr (WORDS == 2) asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
    else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]) : "l"(p + 4 * i));
    }
}

template <int BITS, int D, int TERMS_>
struct Tile {
    using L = CellLayout<BITS, D>;
    static constexpr int TERMS = TERMS_;                    // of keys and values
    static constexpr int UNIT = kTile / TERMS, CELLS = UNIT / kCell;        // positions of a unit
    static constexpr int GROUPS = kDecode / TERMS;          // 32 positions that one warp, or two, decode
    static constexpr int NB = L::NB;
    static constexpr int MIN_BLOCKS = tile_blocks(D);
    static constexpr uint32_t TMEM = D == 256 ? 512 : 256;  // columns: scores (and in their place weights) 0..127, outputs from 128
    static constexpr int Q_BYTES = kRows * D * 2, K_BYTES = kTile * D * 2, V_BYTES = kTile * D * 2;
    struct Shared {
        WalkShared walk;
        Part part[2];
        uint64_t part_full[2], part_empty[2], cell_full[kSlots], cell_empty[kSlots];
        uint64_t q_full, k_full, v_full, s_full, p_full, pv_done;
        uint64_t cell[kSlots][CELLS];                       // addresses; 0: no position that is seen, 1: page out of range
        float factor[2][kRows];                             // of the queries of a part
        int k_exp[2][GROUPS], v_exp[2][GROUPS];             // of 32 positions: the stored value is the tile's times 2^exp
        uint32_t any_bad[2][GROUPS];                        // some value block of the 32 positions is no number
        uint8_t bad[2][UNIT];                               // then: of each position, bit b: block b
        uint32_t tmem;
        int abort;
    };
    static constexpr int FIXED = ((int)sizeof(Shared) + 1023) / 1024 * 1024;
    static constexpr int SMEM = FIXED + Q_BYTES + K_BYTES + V_BYTES;
    static_assert(SMEM <= (228 / MIN_BLOCKS - 1) * 1024, "shared memory");
};

// Raw 16-bit floats of unsigned quants: pairs 0 and 2 times 2^-24, pairs 1 and 3 times 2^-20 (4 bits) or 2^-24 (8 bits).
template <int BITS, uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ void raw_pairs(const uint32_t *w, uint32_t (&h)[4]) {
    if constexpr (BITS == 4) {
        const uint32_t v = w[0] >> 8;
        h[0] = w[0] & 0x000f000fu;
        h[1] = w[0] & 0x00f000f0u;
        h[2] = v & 0x000f000fu;
        h[3] = v & 0x00f000f0u;
    } else {
        h[0] = prmt(w[0], 0, SEL0);
        h[1] = prmt(w[0], 0, SEL1);
        h[2] = prmt(w[1], 0, SEL0);
        h[3] = prmt(w[1], 0, SEL1);
    }
}

// raw quants times scale d (normalised): 4 bits: d 2^-20 (n - 8), 8 bits: d 2^-24 (u - 128); one rounding each, and one
// of the offset's product where that is subnormal.
struct Scale {                                              // of two blocks, or of two positions
    __half2 d, off, big;
    template <int BITS>
    static __device__ __forceinline__ Scale of(__half2 d) {
        return {d, __hmul2(d, __half2half2(__ushort_as_half(0x8080))), BITS == 4 ? __hmul2(d, power_h2(4)) : d};       // -2^-17
    }
    __device__ __forceinline__ Scale block(int b) const {
        return b ? Scale{__high2half2(d), __high2half2(off), __high2half2(big)} : Scale{__low2half2(d), __low2half2(off), __low2half2(big)};
    }
};
template <int BITS>
__device__ __forceinline__ void scaled_pairs(uint32_t (&h)[4], const Scale &s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = h2_bits(__hfma2(bits_h2(h[i]), BITS == 4 && (i & 1) == 0 ? s.big : s.d, s.off));
}

// Term t of a scale d.  Two: its first bits, so few that their product with any quant has 11 bits, and the rest: Q4_0 values are exact
// then, Q8_0 ones rounded to 2^-4 2^-11 of themselves.  Scales below 2^3, whose products are subnormal, stay whole: two more roundings
// of 2^-25 would cost what the rest adds.
template <int BITS, int TERMS>
__device__ __forceinline__ __half2 term(__half2 d, int t) {
    if (TERMS == 1) return d;
    const uint32_t large = __hge2_mask(__habs2(d), __half2half2(__ushort_as_half(0x4800)));
    const __half2 first = bits_h2(h2_bits(d) & (~large | (BITS == 4 ? 0xfff8fff8u : 0xff80ff80u)));
    return t == 0 ? first : __hsub2(d, first);
}

// ------------------------------------------------------------------ the walker

template <int BITS, int D, int TERMS>
__device__ __forceinline__ void walk(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, long long total, long long x0, long long end) {
    using L = CellLayout<BITS, D>;
    constexpr int UNIT = Tile<BITS, D, TERMS>::UNIT, CELLS = Tile<BITS, D, TERMS>::CELLS, AHEAD = 32 / CELLS;
    const int lane = threadIdx.x & 31;
    volatile int *abort = &s.abort;
    int slot = 0;
    uint32_t phase = 1;
    for (long long x = x0, n = 0;; ++n) {
        const int at = (int)n & 1;
        if (!tc_wait(smem_u32(&s.part_empty[at]), (uint32_t)(n >> 1 & 1) ^ 1, abort, a.c.fault)) return;
        if (x >= end) {
            if (lane == 0) {
                s.part[at].take = 0;
                mbar_arrive(smem_u32(&s.part_full[at]));
            }
            return;
        }
        if (x >= s.walk.walk.next) walk_to<32>(a, x, s.walk.walk.r + 1, s.walk.walk.next, s.walk);
        tell_part(a, s.walk.walk, x, x0, end, total, s.part[at]);
        const Part &p = s.part[at];
        if (lane == 0) mbar_arrive(smem_u32(&s.part_full[at]));
        uint64_t cell = 0;
        for (int u = 0; u < p.take; ++u) {
            if (u % AHEAD == 0) {                           // lane i: cell i of the next units
                const int pos = p.begin + u * UNIT + lane * kCell;
                cell = 0;
                if (lane / CELLS + u < p.take && pos < p.span.hi && pos + kCell > p.span.lo) {
                    uint8_t *cells = page_cells(a.c, s.walk.walk.r, pos, p.item.kv_head);
                    cell = cells ? reinterpret_cast<uint64_t>(cell_of<L>(a.c, cells, pos)) : 1;
                    if (cells) prefetch_l2(reinterpret_cast<const void *>(cell), L::BYTES);
                }
            }
            if (!tc_wait(smem_u32(&s.cell_empty[slot]), phase, abort, a.c.fault)) return;
            if (lane / CELLS == u % AHEAD) s.cell[slot][lane % CELLS] = cell;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.cell_full[slot]));
            if (++slot == kSlots) { slot = 0; phase ^= 1; }
        }
        x += p.take;
    }
}

// ------------------------------------------------------------------ decoding

// The addresses of a decode warp's cells, unit after unit.
template <int BITS, int D, int TERMS>
struct Cells {
    typename Tile<BITS, D, TERMS>::Shared &s;
    uint32_t at;                                            // slot, and below it the phase of its barrier
    __device__ __forceinline__ bool next(const AttnArgs &a, int group, uint64_t (&cell)[2]) {
        const uint32_t slot = at >> 1;
        if (!tc_wait(smem_u32(&s.cell_full[slot]), at & 1, &s.abort, a.c.fault)) return false;
        cell[0] = s.cell[slot][2 * group];
        cell[1] = s.cell[slot][2 * group + 1];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&s.cell_empty[slot]));
        at = slot == kSlots - 1 ? (at & 1) ^ 1 : at + 2;
        return true;
    }
};

// The decode warps prepare the tile of Q at a part's start, 16 rows each, while the softmax warps may still write the part before:
// rows times a power of two that takes their largest element to [2^14, 2^15), and the scale's sign.
template <int BITS, int D, int TERMS>
__device__ __forceinline__ void prepare_queries(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, uint8_t *q_tile, int at) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, MINE = kRows / (2 * kDecode);       // lanes of a row, rows at once, rows of a warp
    const Part &part = s.part[at];
    const int lane = threadIdx.x & 31, col = lane % LANES, row0 = MINE * ((threadIdx.x >> 5) - kSoftmax) + lane / LANES;
    auto place = [&](int row) { return q_tile + (col / 8) * (kRows * 128) + row * 128 + ((col % 8 ^ (row & 7)) << 4); };
    // all of the warp's rows on their way into the tile at once, then scaled in place, each lane what it copied
#pragma unroll 1
    for (int i = 0; i < MINE; i += ROWS) {
        int token, head;
        const bool live = row_of(a, part.q, part.item, row0 + i, token, head);
        const long long from = live ? ((long long)part.q.first + token) * a.q_stride + (long long)head * D + 8 * col : 0;
        copy_async16(smem_u32(place(row0 + i)), static_cast<const uint16_t *>(a.q) + from, live);
    }
    copy_async_wait();
#pragma unroll 1
    for (int i = 0; i < MINE; i += ROWS) {
        const int row = row0 + i;
        float v[8];
        if (a.dtype == HQ_DT_F16) load8(reinterpret_cast<const __half *>(place(row)), v);
        else load8(reinterpret_cast<const __nv_bfloat16 *>(place(row)), v);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = min(253, 268 - (int)(top >> 23));
        const float up = __uint_as_float((uint32_t)e << 23) * (a.scale < 0.f ? -1.f : 1.f);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = h2_bits(__floats2half2_rn(v[2 * k] * up, v[2 * k + 1] * up));
        *reinterpret_cast<uint4 *>(place(row)) = make_uint4(h[0], h[1], h[2], h[3]);
        if (col == 0) {                                     // as in the kernel for few rows
            const float f = fabsf(a.scale) * kLog2e * __uint_as_float((uint32_t)(254 - e) << 23);
            s.factor[at][row] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fmaf_rn(f, 0.f, f);
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.q_full));
}

// A key warp has 32 positions of a unit: two cells (two terms: one of them, and a power of two with the warp of the other).  Four neighbouring lanes have a row; rows x and x ^ 5 lie side by
// side, so that the stores do not meet in a bank.  The next unit's bytes are asked for while this one's products run.
template <int BITS, int D, int TERMS>
__device__ __forceinline__ void decode_keys(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, uint8_t *q_tile, uint32_t k_tile) {
    using T = Tile<BITS, D, TERMS>;
    using L = typename T::L;
    constexpr int NB = T::NB, WB = BITS / 4, BLOCKS = NB / L::UNITS;        // words of a block, blocks of a unit
    constexpr int SCALES = NB / 2;                          // words of a lane's share of the scales: 16 lanes a cell
    constexpr int TO = BITS == 4 ? 25 : 29;                 // scales go to [2^10, 2^11) or [2^14, 2^15)
    constexpr int UNIT = T::UNIT, ROWS = 4 / TERMS;         // of a lane, 8 apart
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kSoftmax, group = w / TERMS, half = w % TERMS;
    const int c = lane & 3, kr = (lane >> 3) ^ (lane & 4 ? 5 : 0);
    volatile int *abort = &s.abort;
    Cells<BITS, D, TERMS> cells = {s, 0};
    uint32_t n = 0;                                         // units so far
    uint64_t cell[2] = {0, 0};
    uint32_t raw[ROWS][L::UW], ks[ROWS][BLOCKS / 2], tk[SCALES];
    auto load_unit = [&](int u) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {                    // rows 8 i + kr (and 16 half)
            const uint64_t from = cell[TERMS == 1 ? i >> 1 : half];
            const uint8_t *p = reinterpret_cast<const uint8_t *>(from);
#pragma unroll
            for (int k = 0; k < L::UW; ++k) raw[i][k] = 0;
#pragma unroll
            for (int k = 0; k < BLOCKS / 2; ++k) ks[i][k] = from ? 0x7fff7fffu : 0u;        // a page out of range: NaN
            if (from > 1) {
                load_global<L::UW>(p + L::k_word(8 * (i & 1) + kr, c, u * L::UW), raw[i]);
                load_global<BLOCKS / 2>(p + L::k_scale(8 * (i & 1) + kr, u * BLOCKS), ks[i]);
            }
        }
    };
    auto load = [&]() {
        load_unit(0);
        const uint8_t *p = reinterpret_cast<const uint8_t *>(cell[lane >> 4]);
#pragma unroll
        for (int k = 0; k < SCALES; ++k) {
            tk[k] = 0;
            if (cell[lane >> 4] > 1) load_global<1>(p + L::KS + 4 * ((lane & 15) * SCALES + k), &tk[k]);
        }
    };
    for (int part_n = 0;; ++part_n) {
        const int at = part_n & 1;
        if (!tc_wait(smem_u32(&s.part_full[at]), (uint32_t)(part_n >> 1 & 1), abort, a.c.fault)) return;
        if (s.part[at].take == 0) return;
        if (n > 0 && !tc_wait(smem_u32(&s.s_full), (n - 1) & 1, abort, a.c.fault)) return;          // the tile of Q is free
        prepare_queries<BITS, D, TERMS>(a, s, q_tile, at);
        if (!cells.next(a, group, cell)) return;
        load();
        for (int u = 0; u < s.part[at].take; ++u, ++n) {
            const int p0 = s.part[at].begin + u * UNIT + 32 * group;        // of this warp's positions
            const int lo = s.part[at].span.lo, hi = s.part[at].span.hi;
            uint32_t top = 0;                               // of what is a number and seen by some row
#pragma unroll
            for (int k = 0; k < SCALES; ++k) {
                const int p = p0 + kCell * (lane >> 4) + ((lane & 15) * SCALES + k) / (NB / 2);
                if (p >= lo && p < hi) {
                    const uint32_t x = tk[k] & 0x7fffu, y = tk[k] >> 16 & 0x7fffu;
                    top = max(top, max(x < 0x7c00u ? x : 0u, y < 0x7c00u ? y : 0u));
                }
            }
            const int e = (int)(__reduce_max_sync(0xffffffffu, top) >> 10);
            if (n > 0 && !tc_wait(smem_u32(&s.s_full), (n - 1) & 1, abort, a.c.fault)) return;      // the tile is free
            if (lane == 0 && half == 0) s.k_exp[n & 1][group] = e - 5;
            const int x = TO - e, x1 = min(x, 15);
            const __half2 up1 = power_h2(x1), up2 = power_h2(x - x1);
#pragma unroll 1
            for (int v = 0; v < L::UNITS; ++v) {
                if (v > 0) load_unit(v);
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    const int row = 32 * group + 16 * half + 8 * i + kr;
                    Scale d[TERMS];
#pragma unroll
                    for (int k = 0; k < BLOCKS; ++k) {
                        const int b = v * BLOCKS + k;
                        if (k % 2 == 0) {
                            const __half2 both = __hmul2(__hmul2(bits_h2(ks[i][k / 2]), up1), up2);
#pragma unroll
                            for (int t = 0; t < TERMS; ++t) d[t] = Scale::of<BITS>(term<BITS, TERMS>(both, t));
                        }
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) {
                            uint32_t h[4];
                            raw_pairs<BITS, 0x4140, 0x4342>(&raw[i][k * WB], h);
                            scaled_pairs<BITS>(h, d[t].block(k & 1));
                            const uint32_t to = k_tile + (b >> 1) * (kTile * 128) + (row + t * UNIT) * 128 + (((4 * (k & 1) + c) ^ (row & 7)) << 4);
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                        }
                    }
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&s.k_full));
                mbar_arrive(smem_u32(&s.s_full));           // (the softmax warps read the exponents)
            }
            if (u + 1 < s.part[at].take) {
                if (!cells.next(a, group, cell)) return;
                load();
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.part_empty[at]));
    }
}

// A value warp has 32 positions of a unit (two terms: half of the blocks of them).  A lane turns eight positions' elements g, 8 + g, .. into rows of V^T: 16 bytes
// each, the rows of eight neighbouring lanes in different banks.
template <int BITS, int D, int TERMS>
__device__ __forceinline__ void decode_values(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, uint8_t *q_tile, uint32_t v_tile) {
    using T = Tile<BITS, D, TERMS>;
    using L = typename T::L;
    constexpr int NB = T::NB, WB = BITS / 4;                // words of a block
    constexpr int UNIT = T::UNIT, MINE = NB / TERMS;        // blocks of a warp
    constexpr int STEP = MINE == 1 || (BITS == 8 && D == 128) ? 1 : 2;      // blocks at a time (two are more than 72 registers there)
    constexpr int SCALES = NB / 2;
    constexpr int TO = BITS == 4 ? 25 : 29;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kValues, group = w / TERMS, half = w % TERMS, first = half * MINE;
    const int q = lane >> 3, g = lane & 7;                  // eight positions from 8 q, elements g of each eight
    volatile int *abort = &s.abort;
    Cells<BITS, D, TERMS> cells = {s, 0};
    uint32_t n = 0;
    uint64_t cell[2] = {0, 0};
    uint32_t raw[4][STEP * WB], vs[4][STEP], tv[SCALES];
    auto load_step = [&](int b) {                           // blocks b .. + STEP - 1
        const uint64_t from = cell[q >> 1];
        const uint8_t *p = reinterpret_cast<const uint8_t *>(from);
#pragma unroll
        for (int i = 0; i < 4; ++i) {                       // pairs 4 (q % 2) + i
#pragma unroll
            for (int k = 0; k < STEP * WB; ++k) raw[i][k] = 0;
#pragma unroll
            for (int k = 0; k < STEP; ++k) vs[i][k] = 0;
            if (from > 1) {
                load_global<STEP * WB>(p + L::v_word(4 * (q & 1) + i, g, b * WB), raw[i]);
                load_global<STEP>(p + L::v_scale(8 * (q & 1) + 2 * i, b), vs[i]);
            }
        }
    };
    auto load = [&]() {
        load_step(first);
        const uint8_t *p = reinterpret_cast<const uint8_t *>(cell[lane >> 4]);
#pragma unroll
        for (int k = 0; k < SCALES; ++k) {
            tv[k] = 0;
            if (cell[lane >> 4] > 1) load_global<1>(p + L::VS + 4 * ((lane & 15) * SCALES + k), &tv[k]);
        }
    };
    for (int part_n = 0;; ++part_n) {
        const int at = part_n & 1;
        if (!tc_wait(smem_u32(&s.part_full[at]), (uint32_t)(part_n >> 1 & 1), abort, a.c.fault)) return;
        if (s.part[at].take == 0) return;
        if (n > 0 && !tc_wait(smem_u32(&s.s_full), (n - 1) & 1, abort, a.c.fault)) return;          // the tile of Q is free
        prepare_queries<BITS, D, TERMS>(a, s, q_tile, at);
        if (!cells.next(a, group, cell)) return;
        load();
        for (int u = 0; u < s.part[at].take; ++u, ++n) {
            const int p0 = s.part[at].begin + u * UNIT + 32 * group;
            const int lo = s.part[at].span.lo, hi = s.part[at].span.hi, par = n & 1;
            const bool edge = p0 < lo || p0 + 32 > hi;
            uint32_t top = 0;
            bool odd = false;                               // a block that is no number
#pragma unroll
            for (int k = 0; k < SCALES; ++k) {
                const int p = p0 + kCell * (lane >> 4) + 2 * (((lane & 15) * SCALES + k) / NB);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = tv[k] >> (16 * h) & 0x7fffu;
                    if (p + h >= lo && p + h < hi) {
                        if (x < 0x7c00u) top = max(top, x); else odd = true;
                    }
                }
            }
            const int e = (int)(__reduce_max_sync(0xffffffffu, top) >> 10);
            odd = __any_sync(0xffffffffu, odd);
            if (n > 0 && !tc_wait(smem_u32(&s.s_full), (n - 1) & 1, abort, a.c.fault)) return;
            if (lane == 0) {
                if (half == 0) s.v_exp[par][group] = e - 5;
                mbar_arrive(smem_u32(&s.s_full));           // (the softmax warps read the exponents)
            }
            if (n > 0 && !tc_wait(smem_u32(&s.pv_done), (n - 1) & 1, abort, a.c.fault)) return;     // the tile is free
            if (lane == 0 && half == 0) s.any_bad[par][group] = odd;         // (the softmax warps are done with those of two units before)
            if (odd && half == 0) {                         // a lane a position: marks of its blocks
                uint32_t marks = 0;
                const uint64_t from = cell[lane >> 4];
#pragma unroll 1
                for (int b = 0; b < NB && from > 1 && p0 + lane >= lo && p0 + lane < hi; ++b) {
                    const uint16_t d = *reinterpret_cast<const uint16_t *>(reinterpret_cast<const uint8_t *>(from) + L::v_scale(lane & 15, b));
                    if ((d & 0x7c00u) == 0x7c00u) marks |= 1u << b;
                }
                s.bad[par][32 * group + lane] = (uint8_t)marks;
            }
            const int x = TO - e, x1 = min(x, 15);
            const __half2 up1 = power_h2(x1), up2 = power_h2(x - x1);
#pragma unroll 1
            for (int b = first; b < first + MINE; b += STEP) {
                if (b > first) load_step(b);
                if (edge) {                                 // positions that no row sees are zeros
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = p0 + 8 * q + 2 * i;
                        const uint32_t keep = (p >= lo && p < hi ? 0xffffu : 0u) | (p + 1 >= lo && p + 1 < hi ? 0xffff0000u : 0u);
#pragma unroll
                        for (int k = 0; k < STEP; ++k) vs[i][k] &= keep;
                    }
                }
                if (odd) {                                  // blocks that are no numbers leave the product
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < STEP; ++k) vs[i][k] &= ~__vcmpeq2(vs[i][k] & 0x7c007c00u, 0x7c007c00u);
                }
#pragma unroll
                for (int k = 0; k < STEP; ++k)
#pragma unroll 1
                for (int t = 0; t < TERMS; ++t) {
                    uint32_t h[4][4];                       // [pair][j]
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        raw_pairs<BITS, 0x4240, 0x4341>(&raw[i][k * WB], h[i]);
                        scaled_pairs<BITS>(h[i], Scale::of<BITS>(term<BITS, TERMS>(__hmul2(__hmul2(bits_h2(vs[i][k]), up1), up2), t)));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = 32 * (b + k) + 8 * j + g, column = t * UNIT + 32 * group + 8 * q;       // of 128, 64 to a row of 128 bytes
                        const uint32_t to = v_tile + column / 64 * (D * 128) + row * 128 + ((column / 8 % 8 ^ g) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(h[0][j]), "r"(h[1][j]), "r"(h[2][j]), "r"(h[3][j]) : "memory");
                    }
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.v_full));
            if (u + 1 < s.part[at].take) {
                if (!cells.next(a, group, cell)) return;
                load();
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.part_empty[at]));
    }
}

// ------------------------------------------------------------------ products

template <int BITS, int D, int TERMS>
__device__ __forceinline__ void products(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, uint32_t q_tile, uint32_t k_tile,
                                         uint32_t v_tile, uint32_t tmem) {
    volatile int *abort = &s.abort;
    constexpr int UNIT = Tile<BITS, D, TERMS>::UNIT;
    const uint32_t qk = tc_idesc(UNIT, false), pv = tc_idesc(D, false);
    const uint32_t scores = tmem, outputs = tmem + 128;
    uint32_t n = 0;
    bool fine = true;
    for (uint32_t part_n = 0; fine; ++part_n) {
        const int at = part_n & 1;
        if (!tc_wait(smem_u32(&s.part_full[at]), part_n >> 1 & 1, abort, a.c.fault)) break;
        const int take = s.part[at].take;
        if (take == 0) break;
        if (!tc_wait(smem_u32(&s.q_full), part_n & 1, abort, a.c.fault)) break;
        for (int u = 0; u < take; ++u, ++n) {
            if (!tc_wait(smem_u32(&s.k_full), n & 1, abort, a.c.fault) ||
                (n > 0 && !tc_wait(smem_u32(&s.pv_done), (n - 1) & 1, abort, a.c.fault))) { fine = false; break; }
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_ss(scores, tc_desc_sw128(q_tile + k / 4 * (kRows * 128) + k % 4 * 32),
                              tc_desc_sw128(k_tile + k / 4 * (kTile * 128) + t * UNIT * 128 + k % 4 * 32), qk, t + k > 0);
            tc_commit(smem_u32(&s.s_full));
            if (!tc_wait(smem_u32(&s.v_full), n & 1, abort, a.c.fault) ||
                !tc_wait(smem_u32(&s.p_full), n & 1, abort, a.c.fault)) { fine = false; break; }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)            // (of each term's columns the weights are the same)
                tc_mma(outputs, scores + 8 * (k % (UNIT / 16)), tc_desc_sw128(v_tile + k / 4 * (D * 128) + k % 4 * 32), pv, u > 0 || k > 0);
            tc_commit(smem_u32(&s.pv_done));
        }
        if (fine) mbar_arrive(smem_u32(&s.part_empty[at]));
    }
    if (!fine || *abort) {
        // after a time-out: what was issued ends before the tensor memory is given back
        tc_commit(smem_u32(&s.pv_done));
        for (int k = 0; k < 1000 && !mbar_try_wait_sleep(smem_u32(&s.pv_done), n & 1, 20000u); ++k) {}
    }
}

// ------------------------------------------------------------------ softmax

template <int BITS, int D, int TERMS>
__device__ __forceinline__ void softmax(const AttnArgs &a, typename Tile<BITS, D, TERMS>::Shared &s, uint32_t tmem) {
    constexpr int UNIT = Tile<BITS, D, TERMS>::UNIT, GROUPS = Tile<BITS, D, TERMS>::GROUPS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = threadIdx.x;
    volatile int *abort = &s.abort;
    const uint32_t scores = tmem + ((uint32_t)(32 * warp) << 16), outputs = scores + 128;
    uint32_t n = 0;
    for (uint32_t part_n = 0;; ++part_n) {
        const int at = part_n & 1;
        if (!tc_wait(smem_u32(&s.part_full[at]), part_n >> 1 & 1, abort, a.c.fault)) return;
        const Part &part = s.part[at];
        const int take = part.take;
        if (take == 0) return;
        float factor = 0.f;                                 // (known with the part's first scores)
        int token, head;
        const bool live = row_of(a, part.q, part.item, me, token, head);
        const bool work = __any_sync(0xffffffffu, live);    // some row of the warp
        const Range see = seen_by(a, part.q, min(token, part.q.n - 1));
        float ref = -INFINITY, l = 0.f;                     // the reference of the weights, their sum
        uint32_t bad = 0;
        int p0 = part.begin;
        // value blocks of a unit that are no numbers and that the row sees
        auto look_at_bad = [&](uint32_t unit, int first) {
            const uint32_t *f = s.any_bad[unit & 1];
            uint32_t any = 0;
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) any |= f[k];
            if (any == 0) return;
            for (int k = 0; k < UNIT; ++k)
                if (f[k >> 5] && first + k >= see.lo && first + k < see.hi && first + k >= part.span.lo && first + k < part.span.hi)
                    bad |= s.bad[unit & 1][k];
        };
        for (int u = 0; u < take; ++u, ++n, p0 += UNIT) {
            if (!tc_wait(smem_u32(&s.s_full), n & 1, abort, a.c.fault)) return;
            tc_fence_after();
            if (u == 0) factor = see.hi > see.lo ? s.factor[at][me] : 0.f;      // (a row that sees nothing is zeros, whatever its query)
            if (work) {
                if (u > 0) look_at_bad(n - 1, p0 - UNIT);
                const int first = see.lo - p0, last = see.hi - p0;          // columns that the row sees: [first, last)
                const bool edge = __any_sync(0xffffffffu, first > 0 || last < UNIT);
                const int *ke = s.k_exp[n & 1], *ve = s.v_exp[n & 1];       // of 32 columns
                // (Loops that stay loops, and the hidden columns in a pass of their own: the warps of a multiprocessor run many
                // different paths, and what they do not find in the instruction caches they wait for.)
                if (edge) {
#pragma unroll 1
                    for (int c = 0; c < UNIT; c += 8) {
                        float v[8];
                        tmem_ld8(scores + c, v);
                        tmem_wait_ld(v);
                        const uint32_t seen = bits_between(first - c, last - c);
#pragma unroll
                        for (int k = 0; k < 8; ++k) if (!(seen >> k & 1u)) v[k] = -INFINITY;
                        tmem_st8(scores + c, v);
                    }
                    tmem_wait_st();
                }
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < GROUPS; ++c) {
                    float v[32], m[4];
                    tmem_load32(scores + 32 * c, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) m[k] = v[k];
#pragma unroll
                    for (int k = 4; k < 32; ++k) m[k & 3] = fmaxf(m[k & 3], v[k]);
                    m[0] = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                    if (m[0] > -INFINITY) top = fmaxf(top, fmaf(m[0], factor * power(ke[c]), (float)ve[c]));
                }
                const bool raise = top > ref + kSlack;
                if (__any_sync(0xffffffffu, raise)) {
                    const float now = raise ? top : ref, f = raise ? ex2(ref - now) : 1.f;         // 0 from -inf
                    l *= f;
                    ref = now;
                    if (u > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 8) {
                            float y[8];
                            tmem_ld8(outputs + c, y);
                            tmem_wait_ld(y);
#pragma unroll
                            for (int k = 0; k < 8; ++k) y[k] *= f;
                            tmem_st8(outputs + c, y);
                        }
                    }
                }
                const float base = kWeight - fmaxf(ref, -3e38f);            // nothing seen yet: all columns are hidden
                // weights into tensor memory, in place of scores that are in registers by then
#pragma unroll 1
                for (int c = 0; c < GROUPS; ++c) {
                    float v[32], fk = factor * power(ke[c]);
                    if (fk == 0.f) fk = 1e-37f;             // a hidden column's -inf stays one
                    const float b = base + (float)ve[c];
                    const float2 f2 = make_float2(fk, fk), b2 = make_float2(b, b);
                    tmem_load32(scores + 32 * c, v);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int at = 16 * h + 2 * k;
                            float2 z = ffma2(make_float2(v[at], v[at + 1]), f2, b2);
                            z = make_float2(ex2(z.x), ex2(z.y));
                            sum[k & 1] = fadd2(sum[k & 1], z);
                            x[k] = h2_bits(__floats2half2_rn(z.x, z.y));
                        }
                        tmem_st8u(scores + 16 * c + 8 * h, x);
                    }
                    sum[0] = fadd2(sum[0], sum[1]);
                    l = fmaf(sum[0].x + sum[0].y, power(-ve[c]), l);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.p_full));
        }
        // ---- the tile's outputs
        if (!tc_wait(smem_u32(&s.pv_done), (n - 1) & 1, abort, a.c.fault)) return;
        tc_fence_after();
        if (work) {
            look_at_bad(n - 1, p0 - UNIT);
            const float f = part.slot >= 0 ? 1.f : l == 0.f ? 0.f : __fdiv_rn(1.f, l);
            const long long r = (long long)part.slot * kRows + me;
            const long long to = ((long long)part.q.first + token) * a.out_stride + (long long)head * D;
            if (live && part.slot >= 0) a.stat[r] = make_float2(ref - kWeight, l);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float v[32];
                tmem_load32(outputs + 32 * c, v);
                const bool gone = bad >> c & 1u;
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = gone ? __uint_as_float(0x7fffffffu) : v[k + i] * f;
                    if (!live) continue;
                    if (part.slot >= 0) store8(a.partial + r * D + 32 * c + k, y);
                    else store_row8<false>(a, to + 32 * c + k, y);
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.part_empty[at]));
    }
}

template <int BITS, int D, int TERMS>
__global__ void __launch_bounds__(kThreads, (Tile<BITS, D, TERMS>::MIN_BLOCKS)) attention_tile_kernel(const __grid_constant__ AttnArgs a) {
    using T = Tile<BITS, D, TERMS>;
    extern __shared__ __align__(1024) uint8_t memory[];
    typename T::Shared &s = *reinterpret_cast<typename T::Shared *>(memory);
    uint8_t *q_tile = memory + T::FIXED;
    const uint32_t q = smem_u32(q_tile), k = q + T::Q_BYTES, v = k + T::K_BYTES;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.part_full[i]), 1);
            mbar_init(smem_u32(&s.part_empty[i]), kSoftmax + 2 * kDecode + 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&s.cell_full[i]), 1);
            mbar_init(smem_u32(&s.cell_empty[i]), 2 * kDecode);
        }
        mbar_init(smem_u32(&s.q_full), 2 * kDecode);
        mbar_init(smem_u32(&s.k_full), kDecode);
        mbar_init(smem_u32(&s.v_full), kDecode);
        mbar_init(smem_u32(&s.s_full), 1 + 2 * kDecode);         // the products, and the exponents of K and V
        mbar_init(smem_u32(&s.p_full), kSoftmax);
        mbar_init(smem_u32(&s.pv_done), 1);
        fence_mbar_init();
        s.abort = 0;
    }
    // Tensor memory is taken after what precedes is done and before what follows may start: neither can hold it while it
    // waits for this kernel, or the other way round.
    griddep_wait();
    if (warp == 0) tmem_alloc(smem_u32(&s.tmem), T::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = s.tmem;
    long long total, x0, end;
    deal<kThreads>(a, total, x0, end, s.walk);
    if (x0 >= end) {
    } else if (warp < kSoftmax) {
        softmax<BITS, D, TERMS>(a, s, tmem);
    } else if (warp < kValues) {
        decode_keys<BITS, D, TERMS>(a, s, q_tile, k);
    } else if (warp < kWalker) {
        decode_values<BITS, D, TERMS>(a, s, q_tile, v);
    } else if (warp == kWalker) {
        walk<BITS, D, TERMS>(a, s, total, x0, end);
    } else if (elect_one()) {
        products<BITS, D, TERMS>(a, s, q, k, v, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, T::TMEM);
}

template <int BITS, int D, int TERMS>
hq_status run(AttnArgs a, int num_sms, cudaStream_t stream) {
    using T = Tile<BITS, D, TERMS>;
    static std::atomic<bool> done[64];
    hq_status st = allow_smem(attention_tile_kernel<BITS, D, TERMS>, T::SMEM, done);
    if (st != HQ_OK) return st;
    static_assert(T::UNIT == 1 << (8 - TERMS), "unit_shift");
    deal_rows(a, kRows, D, 8 - TERMS, std::min(kSms, num_sms) * T::MIN_BLOCKS);
    st = launch_blocks(attention_tile_kernel<BITS, D, TERMS>, dim3((unsigned)a.blocks), kThreads, T::SMEM, stream, "attention", a);
    return st != HQ_OK ? st : run_attention_combine(a, kRows, D, stream);
}

template <int TERMS>
hq_status run_fmt(const AttnArgs &a, int fmt, int dim, int num_sms, cudaStream_t stream) {
    if (fmt == HQ_FMT_Q8_0)
        return dim == 64    ? run<8, 64, TERMS>(a, num_sms, stream)
               : dim == 128 ? run<8, 128, TERMS>(a, num_sms, stream)
                            : run<8, 256, TERMS>(a, num_sms, stream);
    return dim == 64    ? run<4, 64, TERMS>(a, num_sms, stream)
           : dim == 128 ? run<4, 128, TERMS>(a, num_sms, stream)
                        : run<4, 256, TERMS>(a, num_sms, stream);
}

}  // namespace

hq_status run_attention_tile(const AttnArgs &a, int fmt, int dim, int num_sms, cudaStream_t stream) {
    return a.dtype == HQ_DT_F16 ? run_fmt<2>(a, fmt, dim, num_sms, stream) : run_fmt<1>(a, fmt, dim, num_sms, stream);
}

}  // namespace hq
