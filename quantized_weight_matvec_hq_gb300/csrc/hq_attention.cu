// hq_attention.cu -- attention of a batch's tokens over the quantized key/value
// cache: few query rows a key/value head (single tokens, verified drafts).
//
// For 8 or 16 query rows of one key/value head the cache's bytes are the work, and the loads go straight from global
// memory to the registers that decode them.  The layout of a cell is made for that: with mma.sync m16n8k16, scores are
// S^T = K Q^T, 16 positions by 8 rows, and a lane's unit of a key's row is its part of the K operand; outputs are O^T = V^T P^T,
// and a lane's unit of a pair of positions is its part of the V^T operand (halves of a register are neighbouring positions).
// Quants enter as exact 16-bit integers.  A key block's scale multiplies that block's sum in fp32; a value block's scale
// multiplies the weights, which go from one operand's layout to the other's by movmatrix.
//
// Weights are exp2(z - m) with m within 2^5 of the row's running maximum: it is raised, and the outputs so far
// are rescaled, only when a score passes it by that much.  Values' scales are brought to [2^8, 2^9) by a power of two that a
// warp holds, so that 16 bits keep the products' relative precision down to 2^-23 of the largest.
#include <type_traits>

#include <algorithm>

#include "hq_attention.cuh"

namespace hq {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr float kSlack = 5.f;

// ------------------------------------------------------------------ operands

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// A word of eight nibbles n -> four pairs n - 8: the magic 0x6400 | n is 1024 + n (0x6400 | n << 4: 1024 + 16 n), exact.
__device__ __forceinline__ void decode_q4(uint32_t w, uint32_t (&h)[4]) {
    const __half2 off = __half2half2(__ushort_as_half(0xe408));                     // -1032
    const __half2 r16 = __half2half2(__ushort_as_half(0x2c00)), off16 = __half2half2(__ushort_as_half(0xd480));   // 1/16, -72
    const uint32_t v = w >> 8;
    h[0] = h2_bits(__hadd2(bits_h2((w & 0x000f000fu) | 0x64006400u), off));
    h[1] = h2_bits(__hfma2(bits_h2((w & 0x00f000f0u) | 0x64006400u), r16, off16));
    h[2] = h2_bits(__hadd2(bits_h2((v & 0x000f000fu) | 0x64006400u), off));
    h[3] = h2_bits(__hfma2(bits_h2((v & 0x00f000f0u) | 0x64006400u), r16, off16));
}

// Two words of bytes u -> four pairs u - 128; SEL0 and SEL1 pick a word's first and second pair.
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ void decode_q8(uint32_t w0, uint32_t w1, uint32_t (&h)[4]) {
    const __half2 off = __half2half2(__ushort_as_half(0xe480));                     // -1152
    h[0] = h2_bits(__hadd2(bits_h2(prmt(w0, 0x64646464u, SEL0)), off));
    h[1] = h2_bits(__hadd2(bits_h2(prmt(w0, 0x64646464u, SEL1)), off));
    h[2] = h2_bits(__hadd2(bits_h2(prmt(w1, 0x64646464u, SEL0)), off));
    h[3] = h2_bits(__hadd2(bits_h2(prmt(w1, 0x64646464u, SEL1)), off));
}

// WORDS 32-bit words that nothing writes while the kernel runs.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *v) {
    if constexpr (WORDS == 1) {
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v[0]) : "l"(p));
    } else if constexpr (WORDS == 2) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]) : "l"(p + 4 * i));
    }
}

// ------------------------------------------------------------------ the kernel

template <bool WIDE_, int BITS, int D, int NT>
struct Stream {
    using L = CellLayout<BITS, D>;
    static constexpr bool WIDE = WIDE_;                     // q and the weights in two terms
    static constexpr int TERMS = WIDE ? 2 : 1;
    static constexpr int ROWS = 8 * NT, NB = L::NB, LW = L::LANE / 4;
    static constexpr int CELLS = L::LANE <= 16 && NT == 1 ? 2 : 1;          // of an iteration of a warp
    static constexpr int STEP = kCell * CELLS;
    // by the registers that a thread needs: loaded cells, outputs, operands and the rest
    static constexpr int REGS = CELLS * (4 * LW + 3 * NB) + 8 * NB * NT + 12 * NT + (WIDE ? 24 : 0) + 52;
    static constexpr int MIN_BLOCKS = REGS <= 128 ? 4 : REGS <= 168 ? 3 : 2;

    struct Shared {
        WalkShared walk;
        uint4 q[TERMS][NT][NB][32];                         // the Q operand: lane (row g, c) has elements 8 c .. + 7 of a block
        float factor[ROWS];                                 // scores = sum * factor, in powers of two
        Range seen[ROWS], part;
        float m[kWarps][ROWS], l[kWarps][ROWS];
        uint32_t bad[ROWS];                                 // value blocks that are no numbers and that the row sees
        alignas(16) float o[kWarps][ROWS][D + 4];           // read as float4
    };

    struct Raw {                                            // what a lane loads of an iteration's cells
        uint32_t k[CELLS][2][LW], v[CELLS][2][LW], ks[CELLS][2][NB / 2], vs[CELLS][2][NB];
    };

    static __device__ __forceinline__ void load_keys(const uint64_t (&cell)[CELLS], Raw &w) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int j = 0; j < CELLS; ++j) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(cell[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (cell[j] > 1) {
#pragma unroll
                    for (int u = 0; u < L::UNITS; ++u)
                        load_words<L::UW>(p + L::k_word(g + 8 * h, c, u * L::UW), &w.k[j][h][u * L::UW]);
                    load_words<NB / 2>(p + L::k_scale(g + 8 * h, 0), w.ks[j][h]);
                } else {                                    // nothing there: masked; a page out of range: NaN
#pragma unroll
                    for (int i = 0; i < LW; ++i) w.k[j][h][i] = 0;
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) w.ks[j][h][i] = cell[j] ? 0x7fff7fffu : 0u;
                }
            }
        }
    }
    static __device__ __forceinline__ void load_values(const uint64_t (&cell)[CELLS], Raw &w) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int j = 0; j < CELLS; ++j) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(cell[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (cell[j] > 1) {
#pragma unroll
                    for (int u = 0; u < L::UNITS; ++u)
                        load_words<L::UW>(p + L::v_word(c + 4 * h, g, u * L::UW), &w.v[j][h][u * L::UW]);
                    load_words<NB>(p + L::v_scale(2 * (c + 4 * h), 0), w.vs[j][h]);
                } else {
#pragma unroll
                    for (int i = 0; i < LW; ++i) w.v[j][h][i] = 0;
#pragma unroll
                    for (int i = 0; i < NB; ++i) w.vs[j][h][i] = 0;
                }
            }
        }
    }

    // The query rows of an item, each times a power of two that takes its largest element to [2^14, 2^15), as 16-bit terms.
    static __device__ __forceinline__ void prepare_rows(const AttnArgs &a, Shared &s) {
        const Walk &w = s.walk.walk;
        const Item &it = s.walk.item;
        constexpr int LANES = D / 8;                        // lanes of a row
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % LANES;
#pragma unroll
        for (int r0 = 0; r0 < ROWS; r0 += kThreads / LANES) {
            const int row = r0 + warp * (32 / LANES) + lane / LANES;
            int token = 0, head = 0;
            const bool live = row < ROWS && row_of(a, w.q, it, row, token, head);
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) load_row8<WIDE>(a, ((long long)w.q.first + token) * a.q_stride + (long long)head * D + 8 * at, v);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int e = min(253, 268 - (int)(top >> 23));        // exponent field of the power: its value 2^(e - 127)
            const float up = __uint_as_float((uint32_t)e << 23);
            uint32_t h[4], r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 x = __floats2half2_rn(v[2 * i] * up, v[2 * i + 1] * up);
                h[i] = h2_bits(x);
                const float2 f = __half22float2(x);
                r[i] = h2_bits(__floats2half2_rn(v[2 * i] * up - f.x, v[2 * i + 1] * up - f.y));
            }
            if (row < ROWS) {
                const int to = (row & 7) * 4 + (at & 3);
                s.q[0][row >> 3][at >> 2][to] = make_uint4(h[0], h[1], h[2], h[3]);
                if (WIDE) s.q[TERMS - 1][row >> 3][at >> 2][to] = make_uint4(r[0], r[1], r[2], r[3]);
                if (at == 0) {
                    // a row that holds no number makes all its scores NaN
                    s.factor[row] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                                       : a.scale * kLog2e * __uint_as_float((uint32_t)(254 - e) << 23);
                    s.bad[row] = 0;
                    s.seen[row] = seen_by(a, w.q, min(token, w.q.n - 1));
                }
            }
        }
    }
};

// An item's part: `take` units from the one that the walk is at.
template <bool WIDE, int BITS, int D, int NT>
__device__ __forceinline__ void stream_part(const AttnArgs &a, int take, int slot, typename Stream<WIDE, BITS, D, NT>::Shared &s) {
    using S = Stream<WIDE, BITS, D, NT>;
    using L = typename S::L;
    constexpr int NB = S::NB, CELLS = S::CELLS, STEP = S::STEP, ROWS = S::ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    // Every row of the tile sees [last_lo, first_hi) of its part; some row sees [begin, end), which is in shared memory.
    int first_hi, last_lo, p_begin;
    {
        const Walk &w = s.walk.walk;
        const Item &it = s.walk.item;
        const int t0 = it.tile * a.tokens, t1 = min(t0 + a.tokens, w.q.n) - 1;
        const Range first = seen_by(a, w.q, t0), last = seen_by(a, w.q, t1);
        first_hi = first.hi;
        last_lo = last.lo;
        p_begin = (first.lo / kUnit + it.unit) * kUnit;
        if (threadIdx.x == 0) s.part = {first.lo, min(p_begin + take * kUnit, last.hi)};
        __syncthreads();
    }
    constexpr int ITS = kUnit / (kWarps * STEP);
    const int n_it = take * ITS;

    // Lane i knows cell i % CELLS of iteration (of 32 / CELLS) i / CELLS: its address, 0 where there is none, 1 where the page is out of range.
    uint64_t mine = 0;
    auto place = [&](int i) { return p_begin + (i * kWarps + warp) * STEP; };
    auto look_up = [&](int i0) {
        const int p = place(i0 + lane / CELLS) + kCell * (lane % CELLS);
        mine = 0;
        if (i0 + lane / CELLS < n_it && p < s.part.hi && p + kCell > s.part.lo) {
            uint8_t *cells = page_cells(a.c, s.walk.walk.r, p, s.walk.item.kv_head);
            mine = cells ? reinterpret_cast<uint64_t>(cell_of<L>(a.c, cells, p)) : 1;
        }
    };
    auto cells_of = [&](int i, uint64_t (&cell)[CELLS]) {
#pragma unroll
        for (int j = 0; j < CELLS; ++j) cell[j] = __shfl_sync(0xffffffffu, mine, (i * CELLS + j) & 31);
    };
    typename S::Raw raw;
    look_up(0);
    bool here = false;                                      // the iteration has a cell (the whole warp)
    {
        uint64_t cell[CELLS];
        cells_of(0, cell);
#pragma unroll
        for (int j = 0; j < CELLS; ++j) here |= cell[j] != 0;
        S::load_keys(cell, raw);
        S::load_values(cell, raw);
    }

    __syncthreads();                                        // the part before is done with the shared memory
    S::prepare_rows(a, s);
    __syncthreads();

    float o[NT][NB][2][4], m[NT][2], l[NT][2], factor[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[n][i] = -INFINITY;
            l[n][i] = 0.f;
            factor[n][i] = s.factor[8 * n + 2 * c + i];
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][b][0][i] = o[n][b][1][i] = 0.f;
    }
    int up = 23;                                            // the values' scales are taken times 2^up

    for (int i = 0; i < n_it; ++i) {
        const int p0 = place(i);
        if ((i + 1) % (32 / CELLS) == 0) look_up(i + 1);
        uint64_t next[CELLS];
        cells_of(i + 1, next);                              // past the last iteration: not loaded below
        const bool more = i + 1 < n_it;
        const bool now = here;
        here = false;
#pragma unroll
        for (int j = 0; j < CELLS; ++j) here |= next[j] != 0;
        if (!now) {
            if (more) { S::load_keys(next, raw); S::load_values(next, raw); }
            continue;
        }
        // ---- scores
        float z[NT][CELLS][4];
#pragma unroll
        for (int j = 0; j < CELLS; ++j) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][j][e] = 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t ka[4], kb[4];
                if constexpr (BITS == 4) {
                    decode_q4(raw.k[j][0][b], ka);
                    decode_q4(raw.k[j][1][b], kb);
                } else {
                    decode_q8<0x4140, 0x4342>(raw.k[j][0][2 * b], raw.k[j][0][2 * b + 1], ka);
                    decode_q8<0x4140, 0x4342>(raw.k[j][1][2 * b], raw.k[j][1][2 * b + 1], kb);
                }
                const __half2 d0 = bits_h2(raw.ks[j][0][b / 2]), d1 = bits_h2(raw.ks[j][1][b / 2]);
                const float f0 = b % 2 ? __high2float(d0) : __low2float(d0), f1 = b % 2 ? __high2float(d1) : __low2float(d1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int t = S::TERMS - 1; t >= 0; --t) {
                        const uint4 q = s.q[t][n][b][lane];
                        mma16816(acc, ka[0], kb[0], ka[1], kb[1], q.x, q.y);
                        mma16816(acc, ka[2], kb[2], ka[3], kb[3], q.z, q.w);
                    }
                    z[n][j][0] = fmaf(acc[0], f0, z[n][j][0]);
                    z[n][j][1] = fmaf(acc[1], f0, z[n][j][1]);
                    z[n][j][2] = fmaf(acc[2], f1, z[n][j][2]);
                    z[n][j][3] = fmaf(acc[3], f1, z[n][j][3]);
                }
            }
        }
        if (more) S::load_keys(next, raw);
        // ---- softmax: lane (g, c) has positions g and g + 8 of each cell, of rows 2 c and 2 c + 1
        const bool edge = p0 < last_lo || p0 + STEP > first_hi;
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < CELLS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[n][j][e] *= factor[n][e & 1];
                    if (edge) {
                        const int p = p0 + kCell * j + g + 8 * (e >> 1);
                        const Range x = s.seen[8 * n + 2 * c + (e & 1)];
                        if (p < x.lo || p >= x.hi) z[n][j][e] = -INFINITY;
                    }
                    raise |= z[n][j][e] > m[n][e & 1] + kSlack;
                }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float t = m[n][k];
#pragma unroll
                    for (int j = 0; j < CELLS; ++j) t = fmaxf(t, fmaxf(z[n][j][k], z[n][j][k + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                    const float f = t == m[n][k] ? 1.f : ex2(m[n][k] - t);      // 0 from -inf
                    m[n][k] = t;
                    l[n][k] *= f;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            o[n][b][h][k] *= f;
                            o[n][b][h][k + 2] *= f;
                        }
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < CELLS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[n][j][e] = ex2(z[n][j][e] - fmaxf(m[n][e & 1], -3e38f));    // nothing seen yet: 0
                    l[n][e & 1] += z[n][j][e];
                }
        // ---- the power of two of the values' scales, and blocks that are no numbers
        if (edge) {                                         // positions that no row sees count for nothing
            const int begin = s.part.lo, end = s.part.hi;
#pragma unroll
            for (int j = 0; j < CELLS; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = p0 + kCell * j + 2 * (c + 4 * h);
                    const uint32_t keep = (p >= begin && p < end ? 0xffffu : 0u) | (p + 1 >= begin && p + 1 < end ? 0xffff0000u : 0u);
#pragma unroll
                    for (int b = 0; b < NB; ++b) raw.vs[j][h][b] &= keep;
                }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < CELLS; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < NB; ++b) top = __vmaxu2(top, raw.vs[j][h][b] & 0x7fff7fffu);
        top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        if (top >= 0x7c00u) {                               // an infinity or a NaN: its block leaves the product, its rows are marked
            top = 0;
#pragma unroll
            for (int j = 0; j < CELLS; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t d = raw.vs[j][h][b] >> (16 * k) & 0x7fffu;
                            if (d < 0x7c00u) { top = max(top, d); continue; }
                            raw.vs[j][h][b] &= k ? 0x0000ffffu : 0xffff0000u;
                            const int p = p0 + kCell * j + 2 * (c + 4 * h) + k;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const Range x = s.seen[8 * n + g];
                                if (p >= x.lo && p < x.hi) atomicOr(&s.bad[8 * n + g], 1u << b);
                            }
                        }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        const int want = 23 - (int)(top >> 10);
        if (want < up) {
            const float f = __uint_as_float((uint32_t)(127 + want - up) << 23);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) { o[n][b][0][e] *= f; o[n][b][1][e] *= f; }
            up = want;
        }
        const __half2 up1 = __half2half2(__ushort_as_half((uint16_t)((15 + min(up, 15)) << 10)));
        const __half2 up2 = __half2half2(__ushort_as_half((uint16_t)((15 + up - min(up, 15)) << 10)));
        // ---- outputs
#pragma unroll
        for (int j = 0; j < CELLS; ++j) {
            uint32_t ph[NT][2], pr[NT][2];                  // the weights, positions along a register: pairs c and c + 4
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2 x = __floats2half2_rn(z[n][j][2 * h], z[n][j][2 * h + 1]);
                    ph[n][h] = transpose8x8(h2_bits(x));
                    if (S::WIDE) {
                        const float2 f = __half22float2(x);
                        pr[n][h] = transpose8x8(h2_bits(__floats2half2_rn((z[n][j][2 * h] - f.x) * 2048.f,
                                                                          (z[n][j][2 * h + 1] - f.y) * 2048.f)));
                    }
                }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t va[4], vb[4];
                if constexpr (BITS == 4) {
                    decode_q4(raw.v[j][0][b], va);
                    decode_q4(raw.v[j][1][b], vb);
                } else {
                    decode_q8<0x4240, 0x4341>(raw.v[j][0][2 * b], raw.v[j][0][2 * b + 1], va);
                    decode_q8<0x4240, 0x4341>(raw.v[j][1][2 * b], raw.v[j][1][2 * b + 1], vb);
                }
                __half2 d[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    d[h] = __hmul2(bits_h2(raw.vs[j][h][b]), up1);
                    if (up > 15) d[h] = __hmul2(d[h], up2);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t p[2], r[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (S::WIDE) {
                            const float2 x = __half22float2(bits_h2(ph[n][h])), y = __half22float2(bits_h2(pr[n][h]));
                            const float2 e = __half22float2(d[h]);
                            const float u0 = fmaf(y.x, 0x1p-11f, x.x) * e.x, u1 = fmaf(y.y, 0x1p-11f, x.y) * e.y;
                            const __half2 t = __floats2half2_rn(u0, u1);
                            const float2 f = __half22float2(t);
                            p[h] = h2_bits(t);
                            r[h] = h2_bits(__floats2half2_rn(u0 - f.x, u1 - f.y));
                        } else {
                            p[h] = h2_bits(__hmul2(bits_h2(ph[n][h]), d[h]));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (S::WIDE) mma16816(o[n][b][t], va[2 * t], va[2 * t + 1], vb[2 * t], vb[2 * t + 1], r[0], r[1]);
                        mma16816(o[n][b][t], va[2 * t], va[2 * t + 1], vb[2 * t], vb[2 * t + 1], p[0], p[1]);
                    }
                }
            }
        }
        if (more) S::load_values(next, raw);
    }

    // ---- the warps' results together
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], d);
            if (g == 0) {
                s.m[warp][8 * n + 2 * c + k] = m[n][k];
                s.l[warp][8 * n + 2 * c + k] = l[n][k];
            }
        }
    __syncthreads();
    const float down = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = 8 * n + 2 * c + k;
            float t = s.m[0][row];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) t = fmaxf(t, s.m[i][row]);
            const float f = (m[n][k] == t ? 1.f : ex2(m[n][k] - t)) * down;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s.o[warp][row][32 * b + 16 * h + g] = o[n][b][h][k] * f;
                    s.o[warp][row][32 * b + 16 * h + 8 + g] = o[n][b][h][k + 2] * f;
                }
        }
    __syncthreads();
    constexpr int CHUNKS = D / 8;                           // 8 columns a thread
    const Walk &w = s.walk.walk;
    for (int i = threadIdx.x; i < ROWS * CHUNKS; i += kThreads) {
        const int row = i / CHUNKS, at = i % CHUNKS;
        int token, head;
        if (!row_of(a, w.q, s.walk.item, row, token, head)) continue;
        float t = s.m[0][row], sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 1; k < kWarps; ++k) t = fmaxf(t, s.m[k][row]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            sum += s.l[k][row] * (s.m[k][row] == t ? 1.f : ex2(s.m[k][row] - t));
            const float4 x = *reinterpret_cast<const float4 *>(&s.o[k][row][8 * at]);
            const float4 y = *reinterpret_cast<const float4 *>(&s.o[k][row][8 * at + 4]);
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w; v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
        if (s.bad[row] >> (at / 4) & 1u)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(0x7fffffffu);
        if (slot < 0) {
            const float f = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);         // a row that sees nothing: zeros
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= f;
            store_row8<WIDE>(a, ((long long)w.q.first + token) * a.out_stride + (long long)head * D + 8 * at, v);
        } else {
            const long long r = (long long)slot * ROWS + row;
            store8(a.partial + r * D + 8 * at, v);
            if (at == 0)
                *reinterpret_cast<float2 *>(a.partial + 2ll * a.blocks * ROWS * D + 2 * r) = make_float2(t, sum);
        }
    }
}

template <bool WIDE, int BITS, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Stream<WIDE, BITS, D, NT>::MIN_BLOCKS)) attention_stream_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ typename Stream<WIDE, BITS, D, NT>::Shared s;
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < a.c.n_req; r += kThreads)
            if (request_of(a.c, r).bad) atomicOr(a.c.fault, kFaultCache);
    const long long total = batch_units<kThreads>(a, s.walk);
    const long long x0 = first_unit(a, total, blockIdx.x), end = first_unit(a, total, blockIdx.x + 1);
    if (x0 >= end) return;
    walk_to<kThreads>(a, x0, 0, 0, s.walk);
    for (long long x = x0; x < end;) {
        if (threadIdx.x == 0) s.walk.item = item_at(a, s.walk.walk, x);
        __syncthreads();
        const int units = s.walk.item.units, take = (int)min((long long)(units - s.walk.item.unit), end - x);
        const int slot = take == units ? -1 : 2 * (int)blockIdx.x + (x == x0 ? 0 : 1);
        stream_part<WIDE, BITS, D, NT>(a, take, slot, s);
        __syncthreads();
        x += take;
        if (x < end && x >= s.walk.walk.next) walk_to<kThreads>(a, x, s.walk.walk.r + 1, s.walk.walk.next, s.walk);
    }
}

// Joins the partial results of one item: block b has that of the item that goes on past the end of block b's units and does
// not begin before them.
template <bool WIDE, int D>
__global__ void __launch_bounds__(kThreads) attention_combine_kernel(const __grid_constant__ AttnArgs a, int rows) {
    __shared__ WalkShared s;
    griddep_launch_dependents();
    griddep_wait();
    const long long total = batch_units<kThreads>(a, s);
    const int b = blockIdx.x;
    const long long x0 = first_unit(a, total, b), x = first_unit(a, total, b + 1);
    if (x == x0 || x >= total) return;
    walk_to<kThreads>(a, x, 0, 0, s);
    const Item it = item_at(a, s.walk, x);
    if (it.unit == 0 || it.first < x0) return;              // it begins with this unit, or in a block before
    const long long end = it.first + it.units;
    int last = b;                                           // the last block that has a part
    while (first_unit(a, total, last + 1) < end) ++last;
    const float *stat = a.partial + 2ll * a.blocks * rows * D;
    constexpr int CHUNKS = D / 8;
    for (int i = threadIdx.x; i < rows * CHUNKS; i += kThreads) {
        const int row = i / CHUNKS, at = i % CHUNKS;
        int token, head;
        if (!row_of(a, s.walk.q, it, row, token, head)) continue;
        float t = -INFINITY, sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k = b; k <= last; ++k) {
            const long long r = (2ll * k + (k == b && it.first != x0 ? 1 : 0)) * rows + row;
            const float2 ml = *reinterpret_cast<const float2 *>(stat + 2 * r);
            float y[8];
            load8(a.partial + r * D + 8 * at, y);
            const float t1 = fmaxf(t, ml.x);
            const float f0 = t == t1 ? 1.f : ex2(t - t1), f1 = ml.x == t1 ? 1.f : ex2(ml.x - t1);
            sum = sum * f0 + ml.y * f1;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * f0 + y[e] * f1;
            t = t1;
        }
        const float f = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f;
        store_row8<WIDE>(a, ((long long)s.walk.q.first + token) * a.out_stride + (long long)head * D + 8 * at, v);
    }
}

// ------------------------------------------------------------------ host side

template <class K, class... A>
hq_status launch(K kern, unsigned grid, cudaStream_t stream, const char *what, const A &... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
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

constexpr int kMaxBlocks = 608;                             // the workspace holds two partial results of each

// Rows of a tile: the mean request's query rows a key/value head decide.
int stream_tiles(const AttentionArgs &x) {
    const int64_t rows = (x.cache.n_tokens + x.cache.n_req - 1) / x.cache.n_req * (x.n_heads / x.cache.n_kv_heads);
    return x.cache.head_dim == 256 || rows <= 8 ? 1 : 2;
}

template <bool WIDE, int BITS, int D, int NT>
hq_status run_stream(const AttentionArgs &x, AttnArgs a, int num_sms, cudaStream_t stream) {
    using S = Stream<WIDE, BITS, D, NT>;
    a.tokens = a.group <= S::ROWS ? S::ROWS / a.group : 1;
    a.part_heads = a.group <= S::ROWS ? a.group : S::ROWS;
    a.parts = (a.group + a.part_heads - 1) / a.part_heads;
    // no more blocks than there can be units
    const int64_t tiles = std::min(x.cache.n_tokens, x.cache.n_tokens / a.tokens + x.cache.n_req);
    const int64_t per_tile = (x.cache.table_width * x.cache.page_size + kUnit - 1) / kUnit;
    const double most = (double)tiles * a.c.n_kv_heads * a.parts * per_tile;
    a.blocks = std::min(kMaxBlocks, num_sms * S::MIN_BLOCKS);
    if (most < a.blocks) a.blocks = (int)most;
    a.min_units = 1;
    hq_status st = launch(attention_stream_kernel<WIDE, BITS, D, NT>, (unsigned)a.blocks, stream, "attention", a);
    if (st != HQ_OK || a.blocks < 2 || per_tile < 2) return st;             // an item of one unit is never divided
    return launch(attention_combine_kernel<WIDE, D>, (unsigned)(a.blocks - 1), stream, "attention combine", a, S::ROWS);
}

template <bool WIDE, int BITS>
hq_status run_dim(const AttentionArgs &x, const AttnArgs &a, int num_sms, cudaStream_t stream) {
    const int nt = stream_tiles(x);
    if (x.cache.head_dim == 256) return run_stream<WIDE, BITS, 256, 1>(x, a, num_sms, stream);
    if (x.cache.head_dim == 128)
        return nt == 1 ? run_stream<WIDE, BITS, 128, 1>(x, a, num_sms, stream) : run_stream<WIDE, BITS, 128, 2>(x, a, num_sms, stream);
    return nt == 1 ? run_stream<WIDE, BITS, 64, 1>(x, a, num_sms, stream) : run_stream<WIDE, BITS, 64, 2>(x, a, num_sms, stream);
}

template <bool WIDE>
hq_status run_fmt(const AttentionArgs &x, const AttnArgs &a, int num_sms, cudaStream_t stream) {
    return x.cache.fmt == HQ_FMT_Q8_0 ? run_dim<WIDE, 8>(x, a, num_sms, stream) : run_dim<WIDE, 4>(x, a, num_sms, stream);
}

}  // namespace

#if HQ_PART == 1

hq_status run_attention_f32(const AttentionArgs &x, const AttnArgs &a, int num_sms, cudaStream_t stream) {
    return run_fmt<true>(x, a, num_sms, stream);
}

#else

hq_status run_attention_f32(const AttentionArgs &x, const AttnArgs &a, int num_sms, cudaStream_t stream);

int64_t attention_workspace(const AttentionArgs &x) {
    const int64_t rows = 8 * stream_tiles(x);
    return 2ll * kMaxBlocks * rows * (x.cache.head_dim + 2) * 4;
}

hq_status launch_attention(const AttentionArgs &x, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    AttnArgs a = {};
    a.c = cache_view(x.cache, dev->fault);
    a.q = x.q;
    a.out = x.out;
    a.q_stride = x.q_stride;
    a.out_stride = x.out_stride;
    a.n_heads = x.n_heads;
    a.group = x.n_heads / x.cache.n_kv_heads;
    a.causal = x.causal;
    a.scale = x.scale;
    a.window = x.window;
    a.partial = static_cast<float *>(x.workspace);
    a.dtype = x.cache.dtype;
    return a.dtype == HQ_DT_F32 ? run_attention_f32(x, a, dev->num_sms, stream) : run_fmt<false>(x, a, dev->num_sms, stream);
}

#endif

}  // namespace hq
