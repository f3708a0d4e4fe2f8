// hq_attention.cu -- attention of a batch's tokens over the quantized key/value
// cache: few query rows a key/value head (single tokens, verified drafts).
//
// For 8 or 16 query rows of one key/value head the cache's bytes are the work.  A producer warp copies cells into a ring in
// shared memory, four to a unit, and each of four warps takes a cell of every unit.  The layout of a cell is made for that: with mma.sync
// m16n8k16, scores are S^T = K Q^T, 16 positions by 8 rows, and a lane's unit of a key's row is its part of the K operand; outputs
// are O^T = V^T P^T, and a lane's unit of a pair of positions is its part of the V^T operand (halves of a register are neighbouring
// positions).  So a cell is used where it lies, without a pass that lays its quants out anew; tcgen05 would want them as a tile of
// 128 positions in shared memory, for a product of which 8 of 128 rows are used.  Quants enter as exact 16-bit floats.  A key
// block's scale multiplies that block's sum in fp32; a value block's scale multiplies the weights, which go from one operand's
// layout to the other's by movmatrix.
//
// Weights are exp2(z - m) with m at most 5 below the row's running maximum: it is raised, and the outputs so far
// are rescaled, only when a score passes it by that much.
//
// Measured (Q4_0, heads of 128): 64 requests of 100 to 8191 positions, 8 key/value heads, 4 query heads each (133 MB), 56 us = 2.4 TB/s, of
// which 7 the joins: bound by instructions (335 a cell and warp at 0.50 to 0.67 a cycle and scheduler; tensor pipe 22 %), and by what a block
// does before its first unit, 15 of its 90 thousand cycles.  Q8_0: one request of 131071 positions (143 MB) 38 us = 3.8 TB/s, whose
// loop keeps up with 4 of 5 bytes of the copy rate; 10 us are the start and the joins.  Steps on the way, of these two: 6235 and 164011 with
// a thread an output; 72 and 81 with loads from global memory to registers; 60 and 43 with the ring; 56 and 37 with units of 64
// positions and quants that stay unsigned.
#include <type_traits>

#include "hq_attention.cuh"

namespace hq {
namespace {

constexpr int kWarps = 4, kConsumers = 32 * kWarps, kThreads = kConsumers + 32;     // the last warp is the producer
constexpr int kUnit = kCell * kWarps;                       // a consumer warp has a cell of every unit
constexpr int kCombineThreads = 256;
constexpr float kSlack = 5.f;

// ------------------------------------------------------------------ operands

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// As mma16816, with what is added to: c0 in columns 0 and c1 in columns 1 of a thread's pairs.
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// A word of eight nibbles n -> four pairs n - 8: the magic 0x6400 | n is 1024 + n (0x6400 | n << 4: 1024 + 16 n), exact.
template <class = void>
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

// The same with the quants left unsigned, as 16-bit floats of n 2^-24 (pairs 0 and 2) and n 2^-20, or of u 2^-24: subnormal numbers,
// which the bits are already.
template <class = void>
__device__ __forceinline__ void decode_q4_raw(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t v = w >> 8;
    h[0] = w & 0x000f000fu;
    h[1] = w & 0x00f000f0u;
    h[2] = v & 0x000f000fu;
    h[3] = v & 0x00f000f0u;
}
template <uint32_t SEL0, uint32_t SEL1>
__device__ __forceinline__ void decode_q8_raw(uint32_t w0, uint32_t w1, uint32_t (&h)[4]) {
    h[0] = prmt(w0, 0, SEL0);
    h[1] = prmt(w0, 0, SEL1);
    h[2] = prmt(w1, 0, SEL0);
    h[3] = prmt(w1, 0, SEL1);
}

// WORDS 32-bit words of shared memory.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&v)[WORDS]) {
    if constexpr (WORDS == 1) {
        v[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (WORDS == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        v[0] = x.x; v[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
            v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
    }
}

// ------------------------------------------------------------------ the kernel

template <bool WIDE_, int BITS, int D, int NT>
struct Stream {
    using L = CellLayout<BITS, D>;
    static constexpr bool WIDE = WIDE_;                     // q and the weights in two terms
    static constexpr int TERMS = WIDE ? 2 : 1;
    // Keys unsigned: the offset's part of a block's sum, -8 or -128 times the sum of q, is where the sum starts.  Its rounding is 2^-22 of
    // the largest key times the sum of |q|; f32 decodes the signed quants instead.
    // The values' offset is a second product, with the negative offset for a quant (elements g of a block times 2^-24, g + 8 times 2^-20 or
    // 2^-24): each cell's is taken off at once, so that no large sum of offsets builds up.
    static constexpr bool RAW = !WIDE;
    static constexpr uint32_t LESS0 = BITS == 4 ? 0x80088008u : 0x80808080u, LESS1 = 0x80808080u;       // -8 2^-24 or -128 2^-24; -8 2^-20
    static constexpr float BACK0 = RAW ? 0x1p24f : 1.f, BACK1 = RAW ? BITS == 4 ? 0x1p20f : 0x1p24f : 1.f;
    static constexpr int ROWS = 8 * NT, NB = L::NB;
    static constexpr int STAGE = kWarps * L::BYTES;     // a stage of the ring is a unit
    static constexpr int MIN_BLOCKS = stream_blocks(WIDE, D, ROWS);
    static constexpr int MAX_STAGES = 6;

    // The power of two for scales with this largest exponent field (the value is in [2^(e - 15), 2^(e - 14))).
    // 16 bits: none between 2^-12 and 2: with weights of up to 2^15 (2^10 at the running maximum) the products stay in range,
    // and keep their 11 bits down to 2^-12 of the largest at least.  f32: to [2^8, 2^9), for its second terms.
    static constexpr float WEIGHT = WIDE ? 0.f : 10.f;      // weights are exp2(z - m + WEIGHT)
    static __device__ __forceinline__ int shift_of(int e) { return WIDE ? 23 - e : e > 15 ? 15 - e : e < 3 ? 10 : 0; }

    struct Shared {
        WalkShared walk;
        uint4 q[TERMS][NT][NB][32];                         // the Q operand: lane (row g, c) has elements 8 c .. + 7 of a block
        Part part[2];                                       // this part and the one the producer is ahead with
        alignas(8) float offset[NB][ROWS];
        alignas(8) float factor[ROWS];                                // scores = sum * factor, in powers of two
        Range seen[ROWS];
        float m[kWarps][ROWS], l[kWarps][ROWS];
        uint32_t bad[ROWS];                                 // value blocks that are no numbers and that the row sees
        alignas(16) float o[kWarps / 2][ROWS][D + 4];       // read as float4
        alignas(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], part_full[2], part_empty[2];
        uint32_t cells[MAX_STAGES];                         // of a stage: bit i: cell i is there; bit 16 + i: its page is out of range
        int abort;
    };
    static constexpr int FIXED = ((int)sizeof(Shared) + 127) / 128 * 128;
    static constexpr int LIMIT = (228 / MIN_BLOCKS - 1) * 1024;
    static constexpr int STAGES = (LIMIT - FIXED) / STAGE < MAX_STAGES ? (LIMIT - FIXED) / STAGE : MAX_STAGES;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(STAGES >= 2, "the ring needs two stages");

    // The query rows of an item, each times a power of two that takes its largest element to [2^14, 2^15), as 16-bit terms.
    static __device__ __forceinline__ void prepare_rows(const AttnArgs &a, const Part &part, Shared &s) {
        constexpr int LANES = D / 8;                        // lanes of a row
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = lane % LANES;
#pragma unroll
        for (int r0 = 0; r0 < ROWS; r0 += kConsumers / LANES) {
            const int row = r0 + warp * (32 / LANES) + lane / LANES;
            int token = 0, head = 0;
            const bool live = row < ROWS && row_of(a, part.q, part.item, row, token, head);
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) load_row8<WIDE>(a, ((long long)part.q.first + token) * a.q_stride + (long long)head * D + 8 * at, v);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int e = min(253, 268 - (int)(top >> 23)); // exponent field of the power: its value is 2^(e - 127)
            const float up = __uint_as_float((uint32_t)e << 23);
            uint32_t h[4], r[4];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 x = __floats2half2_rn(v[2 * i] * up, v[2 * i + 1] * up);
                h[i] = h2_bits(x);
                const float2 f = __half22float2(x);
                sum += f.x + f.y;
                if (RAW && BITS == 4 && (i & 1)) h[i] = h2_bits(__hmul2(x, __half2half2(__ushort_as_half(0x2c00))));      // times 1/16, for quants times 16
                r[i] = h2_bits(__floats2half2_rn(v[2 * i] * up - f.x, v[2 * i + 1] * up - f.y));
            }
            if (RAW) {                                      // of the block: four lanes
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (row < ROWS && (at & 3) == 0) s.offset[at >> 2][row] = sum * (BITS == 4 ? -0x1p-21f : -0x1p-17f);
            }
            if (row < ROWS) {
                const int to = (row & 7) * 4 + (at & 3);
                s.q[0][row >> 3][at >> 2][to] = make_uint4(h[0], h[1], h[2], h[3]);
                if (WIDE) s.q[TERMS - 1][row >> 3][at >> 2][to] = make_uint4(r[0], r[1], r[2], r[3]);
                if (at == 0) {
                    // a row that holds no number, or a factor past the largest, makes all scores NaN
                    const float f = a.scale * kLog2e * (RAW ? 0x1p24f : 1.f) * __uint_as_float((uint32_t)(254 - e) << 23);
                    s.factor[row] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fmaf_rn(f, 0.f, f);
                    s.bad[row] = 0;
                    s.seen[row] = seen_by(a, part.q, min(token, part.q.n - 1));
                }
            }
        }
    }
};

// The producer warp: tells the consumers the parts, one after another, and copies their cells into the ring, a cell a lane.
template <bool WIDE, int BITS, int D, int NT>
__device__ __forceinline__ void stream_produce(const AttnArgs &a, typename Stream<WIDE, BITS, D, NT>::Shared &s, uint32_t ring,
                                               long long total, long long x0, long long end) {
    using S = Stream<WIDE, BITS, D, NT>;
    using L = typename S::L;
    constexpr int AHEAD = 32 / kWarps;                  // units whose cells are looked up at once
    const int lane = threadIdx.x & 31;
    volatile int *abort = &s.abort;
    const uint64_t policy = l2_evict_first_policy();
    int n = 0, stage = 0;                                   // parts and units so far
    uint32_t phase = 1;
    for (long long x = x0;; ++n) {
        const int at = n & 1;
        if (!mbar_wait(smem_u32(&s.part_empty[at]), (n >> 1 & 1) ^ 1, abort, a.c.fault)) break;
        if (x >= end) {                                     // the end
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
            if (u % AHEAD == 0) {                           // lane i: cell i of the next units; 0: none, 1: its page is out of range
                const int pos = p.begin + u * kUnit + lane * kCell;
                cell = 0;
                if (pos < p.span.hi && pos + kCell > p.span.lo) {
                    uint8_t *cells = page_cells(a.c, s.walk.walk.r, pos, p.item.kv_head);
                    cell = cells ? reinterpret_cast<uint64_t>(cell_of<L>(a.c, cells, pos)) : 1;
                }
            }
            if (!mbar_wait(smem_u32(&s.empty[stage]), phase, abort, a.c.fault)) goto drain;
            const int first = u % AHEAD * kWarps;
            const uint32_t there = __ballot_sync(0xffffffffu, cell > 1) >> first & ((1u << kWarps) - 1);
            const uint32_t bad = __ballot_sync(0xffffffffu, cell == 1) >> first & ((1u << kWarps) - 1);
            const uint32_t full = smem_u32(&s.full[stage]);
            if (lane == 0) {
                s.cells[stage] = there | bad << 16;
                mbar_arrive_expect_tx(full, __popc(there) * L::BYTES);
            }
            __syncwarp();
            if (lane / kWarps == u % AHEAD && cell > 1)
                bulk_load(ring + stage * S::STAGE + lane % kWarps * L::BYTES, reinterpret_cast<const void *>(cell), L::BYTES, full, policy);
            if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
        }
        x += p.take;
    }
drain:
    // after a time-out: the copies under way end before the block does
    for (int i = 0; i < S::STAGES; ++i) {
        const bool lapped = i < stage;
        const uint32_t parity = lapped ? phase ^ 1 : phase;
        for (int k = 0; k < 100000 && !mbar_try_wait_sleep(smem_u32(&s.full[i]), parity, 20000u); ++k) {}
    }
}

// A consumer warp's way through a part: a cell of every unit.  False after a time-out.
template <bool WIDE, int BITS, int D, int NT>
__device__ __forceinline__ bool stream_consume(const AttnArgs &a, const Part &part, typename Stream<WIDE, BITS, D, NT>::Shared &s,
                                               const uint8_t *ring, uint32_t &lap) {
    using S = Stream<WIDE, BITS, D, NT>;
    using L = typename S::L;
    constexpr int NB = S::NB, ROWS = S::ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

    named_barrier(1, kConsumers);                           // the part before is done with the shared memory
    S::prepare_rows(a, part, s);
    named_barrier(1, kConsumers);

    float o[NT][NB][2][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[n][i] = -INFINITY;
            l[n][i] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][b][0][i] = o[n][b][1][i] = 0.f;
    }
    int up = S::shift_of(0);                                // the values' scales are taken times 2^up
    for (int u = 0; u < part.take; ++u) {
        const uint32_t stage = lap >> 1;                    // the ring's stage, and below it the phase of its barrier
        if (!mbar_wait(smem_u32(&s.full[stage]), lap & 1, &s.abort, a.c.fault)) break;
        const uint32_t states = s.cells[stage];
        const uint32_t state = states >> warp & 0x10001u;
        if (state != 0) {                                   // the whole warp
            const uint8_t *cell = ring + stage * S::STAGE + warp * L::BYTES;
            const int p0 = part.begin + u * kUnit + warp * kCell;
            // ---- scores
            float z[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][e] = 0.f;
            uint32_t ks0[NB / 2], ks1[NB / 2];
            load_words(cell + L::k_scale(g, 0), ks0);
            load_words(cell + L::k_scale(g + 8, 0), ks1);
#pragma unroll
            for (int v = 0; v < L::UNITS; ++v) {
                uint32_t k0[L::UW], k1[L::UW];
                load_words(cell + L::k_word(g, c, v * L::UW), k0);
                load_words(cell + L::k_word(g + 8, c, v * L::UW), k1);
                constexpr int BLOCKS = NB / L::UNITS;       // of a unit
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    const int b = v * BLOCKS + i;
                    uint32_t ka[4], kb[4];
                    if constexpr (S::RAW && BITS == 4) {
                        decode_q4_raw(k0[i], ka);
                        decode_q4_raw(k1[i], kb);
                    } else if constexpr (S::RAW) {
                        decode_q8_raw<0x4140, 0x4342>(k0[2 * i], k0[2 * i + 1], ka);
                        decode_q8_raw<0x4140, 0x4342>(k1[2 * i], k1[2 * i + 1], kb);
                    } else if constexpr (BITS == 4) {
                        decode_q4(k0[i], ka);
                        decode_q4(k1[i], kb);
                    } else {
                        decode_q8<0x4140, 0x4342>(k0[2 * i], k0[2 * i + 1], ka);
                        decode_q8<0x4140, 0x4342>(k1[2 * i], k1[2 * i + 1], kb);
                    }
                    const __half2 d0 = bits_h2(ks0[b / 2]), d1 = bits_h2(ks1[b / 2]);
                    const float f0 = b % 2 ? __high2float(d0) : __low2float(d0), f1 = b % 2 ? __high2float(d1) : __low2float(d1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float acc[4];
                        const float2 start = S::RAW ? *reinterpret_cast<const float2 *>(&s.offset[b][8 * n + 2 * c]) : make_float2(0.f, 0.f);
#pragma unroll
                        for (int t = S::TERMS - 1; t >= 0; --t) {
                            const uint4 q = s.q[t][n][b][lane];
                            if (t == S::TERMS - 1) mma16816_from(acc, ka[0], kb[0], ka[1], kb[1], q.x, q.y, start.x, start.y);
                            else mma16816(acc, ka[0], kb[0], ka[1], kb[1], q.x, q.y);
                            mma16816(acc, ka[2], kb[2], ka[3], kb[3], q.z, q.w);
                        }
                        const float2 z0 = ffma2(make_float2(acc[0], acc[1]), make_float2(f0, f0), make_float2(z[n][0], z[n][1]));
                        const float2 z1 = ffma2(make_float2(acc[2], acc[3]), make_float2(f1, f1), make_float2(z[n][2], z[n][3]));
                        z[n][0] = z0.x;
                        z[n][1] = z0.y;
                        z[n][2] = z1.x;
                        z[n][3] = z1.y;
                    }
                }
            }
            // ---- softmax: lane (g, c) has positions g and g + 8, of rows 2 c and 2 c + 1
            uint32_t vs[2][NB];
            load_words(cell + L::v_scale(2 * c, 0), vs[0]);
            load_words(cell + L::v_scale(2 * c + 8, 0), vs[1]);
            const bool gone = state >> 16;                  // a page out of range: NaN
            if (gone)
#pragma unroll
                for (int b = 0; b < NB; ++b) vs[0][b] = vs[1][b] = 0;
            const bool edge = p0 < part.all_lo || p0 + kCell > part.all_hi;
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 factor = *reinterpret_cast<const float2 *>(&s.factor[8 * n + 2 * c]);
                // A sum is infinite through an infinite scale alone (quants and q are at most 2^15): 0 times it takes the row to NaN, where its
                // sign could make it a score of -inf, the mark of what is not seen.
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 sums = make_float2(z[n][e], z[n][e + 1]), none = make_float2(0.f, 0.f);
                    const float2 x = ffma2(sums, factor, ffma2(sums, none, none));
                    z[n][e] = x.x;
                    z[n][e + 1] = x.y;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (gone) z[n][e] = __uint_as_float(0x7fffffffu);
                    if (edge) {
                        const int p = p0 + g + 8 * (e >> 1);
                        const Range x = s.seen[8 * n + 2 * c + (e & 1)];
                        if (p < x.lo || p >= x.hi) z[n][e] = -INFINITY;
                    }
                    raise |= z[n][e] > m[n][e & 1] + kSlack;
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float t = fmaxf(m[n][k], fmaxf(z[n][k], z[n][k + 2]));
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
                for (int e = 0; e < 4; ++e) {
                    z[n][e] = ex2(z[n][e] - (fmaxf(m[n][e & 1], -3e38f) - S::WEIGHT));      // nothing seen yet: 0
                    l[n][e & 1] += z[n][e];
                }
            // ---- the power of two of the values' scales, and blocks that are no numbers: a word (two positions' scale) a lane
            constexpr int WORDS = (8 * NB + 31) / 32;
            uint32_t mine[WORDS], top = 0;
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const int at = (lane + 32 * i) % (8 * NB);
                mine[i] = *reinterpret_cast<const uint32_t *>(cell + L::VS + 4 * at) & 0x7fff7fffu;
                if (edge) {                                 // positions that no row sees count for nothing
                    const int p = p0 + 2 * (at / NB);
                    mine[i] &= (p >= part.span.lo && p < part.span.hi ? 0xffffu : 0u) |
                               (p + 1 >= part.span.lo && p + 1 < part.span.hi ? 0xffff0000u : 0u);
                }
                top = max(top, max(mine[i] & 0xffffu, mine[i] >> 16));
            }
            top = gone ? 0u : __reduce_max_sync(0xffffffffu, top);
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = p0 + 2 * (c + 4 * h);
                    const uint32_t keep = (p >= part.span.lo && p < part.span.hi ? 0xffffu : 0u) |
                                          (p + 1 >= part.span.lo && p + 1 < part.span.hi ? 0xffff0000u : 0u);
#pragma unroll
                    for (int b = 0; b < NB; ++b) vs[h][b] &= keep;
                }
            }
            if (top >= 0x7c00u) {                           // an infinity or a NaN: its block leaves the product, its rows are marked
                top = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t d = vs[h][b] >> (16 * k) & 0x7fffu;
                            if (d < 0x7c00u) { top = max(top, d); continue; }
                            vs[h][b] &= k ? 0x0000ffffu : 0xffff0000u;
                            const int p = p0 + 2 * (c + 4 * h) + k;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const Range x = s.seen[8 * n + g];
                                if (p >= x.lo && p < x.hi) atomicOr(&s.bad[8 * n + g], 1u << b);
                            }
                        }
                top = __reduce_max_sync(0xffffffffu, top);
            }
            const int want = S::shift_of((int)(top >> 10));
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
            if (up != 0) {
                const int part1 = min(max(up, -14), 15);    // two factors that are normal numbers
                const __half2 up1 = __half2half2(__ushort_as_half((uint16_t)((15 + part1) << 10)));
                const __half2 up2 = __half2half2(__ushort_as_half((uint16_t)((15 + up - part1) << 10)));
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b) vs[h][b] = h2_bits(__hmul2(__hmul2(bits_h2(vs[h][b]), up1), up2));
            }
            // ---- outputs
            // The weights, positions along a register: pairs c and c + 4; what their rounding left joins the product with the scale, so
            // that 16-bit tokens have one rounding (64 requests 55 to 56 us; f16 outputs of 131071 positions 3.4e-4 off without it).
            uint32_t ph[NT][2], pr[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2 x = __floats2half2_rn(z[n][2 * h], z[n][2 * h + 1]);
                    ph[n][h] = transpose8x8(h2_bits(x));
                    const float2 f = __half22float2(x);
                    const float up = S::WIDE ? 2048.f : 1.f;
                    pr[n][h] = transpose8x8(h2_bits(__floats2half2_rn((z[n][2 * h] - f.x) * up, (z[n][2 * h + 1] - f.y) * up)));
                }
#pragma unroll
            for (int v = 0; v < L::UNITS; ++v) {
                uint32_t v0[L::UW], v1[L::UW];
                load_words(cell + L::v_word(c, g, v * L::UW), v0);
                load_words(cell + L::v_word(c + 4, g, v * L::UW), v1);
                constexpr int BLOCKS = NB / L::UNITS;
#pragma unroll
                for (int i = 0; i < BLOCKS; ++i) {
                    const int b = v * BLOCKS + i;
                    uint32_t va[4], vb[4];
                    if constexpr (S::RAW && BITS == 4) {
                        decode_q4_raw(v0[i], va);
                        decode_q4_raw(v1[i], vb);
                    } else if constexpr (S::RAW) {
                        decode_q8_raw<0x4240, 0x4341>(v0[2 * i], v0[2 * i + 1], va);
                        decode_q8_raw<0x4240, 0x4341>(v1[2 * i], v1[2 * i + 1], vb);
                    } else if constexpr (BITS == 4) {
                        decode_q4(v0[i], va);
                        decode_q4(v1[i], vb);
                    } else {
                        decode_q8<0x4240, 0x4341>(v0[2 * i], v0[2 * i + 1], va);
                        decode_q8<0x4240, 0x4341>(v1[2 * i], v1[2 * i + 1], vb);
                    }
                    const __half2 d[2] = {bits_h2(vs[0][b]), bits_h2(vs[1][b])};
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
                                p[h] = h2_bits(__hfma2(bits_h2(ph[n][h]), d[h], __hmul2(bits_h2(pr[n][h]), d[h])));
                            }
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (S::RAW) mma16816(o[n][b][t], S::LESS0, S::LESS1, S::LESS0, S::LESS1, p[0], p[1]);
                            if (S::WIDE) mma16816(o[n][b][t], va[2 * t], va[2 * t + 1], vb[2 * t], vb[2 * t + 1], r[0], r[1]);
                            mma16816(o[n][b][t], va[2 * t], va[2 * t + 1], vb[2 * t], vb[2 * t + 1], p[0], p[1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.empty[stage]));
        lap = stage == S::STAGES - 1 ? (lap & 1) ^ 1 : lap + 2;
    }

    // ---- the warps' results together: the upper half's to the lower half's, then those
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
    named_barrier(1, kConsumers);
    const float down = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        if (warp / (kWarps / 2) == 1 - turn) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = 8 * n + 2 * c + k;
                    float t = s.m[0][row];
#pragma unroll
                    for (int i = 1; i < kWarps; ++i) t = fmaxf(t, s.m[i][row]);
                    const float f = (m[n][k] == t ? 1.f : ex2(m[n][k] - t)) * down;
                    float *to = s.o[warp % (kWarps / 2)][row] + g;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float *x = to + 32 * b + 16 * h;
                            x[0] = (turn ? x[0] : 0.f) + o[n][b][h][k] * f * S::BACK0;
                            x[8] = (turn ? x[8] : 0.f) + o[n][b][h][k + 2] * f * S::BACK1;
                        }
                }
        }
        named_barrier(1, kConsumers);
    }
    constexpr int CHUNKS = D / 8;                           // 8 columns a thread
    for (int i = threadIdx.x; i < ROWS * CHUNKS; i += kConsumers) {
        const int row = i / CHUNKS, at = i % CHUNKS;
        int token, head;
        if (!row_of(a, part.q, part.item, row, token, head)) continue;
        float t = s.m[0][row], sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 1; k < kWarps; ++k) t = fmaxf(t, s.m[k][row]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += s.l[k][row] * (s.m[k][row] == t ? 1.f : ex2(s.m[k][row] - t));
#pragma unroll
        for (int k = 0; k < kWarps / 2; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(&s.o[k][row][8 * at]);
            const float4 y = *reinterpret_cast<const float4 *>(&s.o[k][row][8 * at + 4]);
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w; v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
        if (s.bad[row] >> (at / 4) & 1u)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(0x7fffffffu);
        if (part.slot < 0) {
            const float f = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);         // a row that sees nothing: zeros
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= f;
            store_row8<WIDE>(a, ((long long)part.q.first + token) * a.out_stride + (long long)head * D + 8 * at, v);
        } else {
            const long long r = (long long)part.slot * ROWS + row;
            store8(a.partial + r * D + 8 * at, v);
            if (at == 0)
                a.stat[r] = make_float2(t, sum);
        }
    }
    return *(volatile int *)&s.abort == 0;
}

template <bool WIDE, int BITS, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Stream<WIDE, BITS, D, NT>::MIN_BLOCKS)) attention_stream_kernel(const __grid_constant__ AttnArgs a) {
    using S = Stream<WIDE, BITS, D, NT>;
    extern __shared__ __align__(128) uint8_t memory[];
    typename S::Shared &s = *reinterpret_cast<typename S::Shared *>(memory);
    uint8_t *ring = memory + S::FIXED;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.part_full[i]), 1);
            mbar_init(smem_u32(&s.part_empty[i]), kWarps);
        }
        fence_mbar_init();
        s.abort = 0;
    }
    griddep_launch_dependents();
    griddep_wait();
    long long total, x0, end;
    deal<kThreads>(a, total, x0, end, s.walk);              // (with barriers, which the mbarriers' set-up needs)
    if (x0 >= end) return;
    if (threadIdx.x >= kConsumers) {
        stream_produce<WIDE, BITS, D, NT>(a, s, smem_u32(ring), total, x0, end);
        return;
    }
    uint32_t lap = 0;
    for (int n = 0;; ++n) {
        const int at = n & 1;
        if (!mbar_wait(smem_u32(&s.part_full[at]), n >> 1 & 1, &s.abort, a.c.fault)) break;
        if (s.part[at].take == 0) break;
        const bool ok = stream_consume<WIDE, BITS, D, NT>(a, s.part[at], s, ring, lap);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&s.part_empty[at]));
        if (!ok) break;
    }
}

// Joins the partial results of the item that block blockIdx.x tells of, AT_ONCE rows at a time (gridDim.y blocks share them).  D / 8
// lanes a row of a partial result, the groups of them that a row has take every GROUPS-th block's.
// It is bound by the latency of its loads, so its shape is a matter of how many are under way.  Few rows: two at a time with 4 to 16 groups
// (7 us of 64 requests' 56, from a cold start; eight rows a block 61 in all); an item may lie on many blocks (131071 positions of 4 heads: 152
// each).  Tiles: mostly two or three blocks an item, and 128 rows, so a group a row and nothing to exchange; eight groups a row,
// with two barriers for every two rows, took 43 us of a prompt of 2011 tokens (152 in all) where this takes 11.6 (126).
template <bool WIDE, int D, int AT_ONCE>
__global__ void __launch_bounds__(kCombineThreads) attention_combine_kernel(const __grid_constant__ AttnArgs a, int rows) {
    constexpr int LANES = D / 8, GROUPS = kCombineThreads / LANES / AT_ONCE;
    __shared__ float gm[AT_ONCE][GROUPS], gl[AT_ONCE][GROUPS];
    __shared__ alignas(16) float go[GROUPS > 1 ? AT_ONCE : 1][GROUPS][D];
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x;
    if (!a.joins[b].valid) return;
    const Join join = a.joins[b];
    const int mine = threadIdx.x / (LANES * GROUPS), group = threadIdx.x / LANES % GROUPS, at = threadIdx.x % LANES;
    for (int row0 = blockIdx.y * AT_ONCE; row0 < rows; row0 += gridDim.y * AT_ONCE) {
        const int row = row0 + mine;
        int token, head;
        const bool live = row_of(a, join.q, join.item, row, token, head);
        float t = -INFINITY, sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live) {
#pragma unroll 4
            for (int k = b + group; k <= join.last; k += GROUPS) {
                const long long r = (long long)(k == b ? join.slot : 2 * k) * rows + row;
                const float2 ml = a.stat[r];
                float y[8];
                load8(a.partial + r * D + 8 * at, y);
                const float t1 = fmaxf(t, ml.x);
                const float f0 = t == t1 ? 1.f : ex2(t - t1), f1 = ml.x == t1 ? 1.f : ex2(ml.x - t1);
                sum = sum * f0 + ml.y * f1;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * f0 + y[e] * f1;
                t = t1;
            }
        }
        if constexpr (GROUPS > 1) {
            if (at == 0) { gm[mine][group] = t; gl[mine][group] = sum; }
            store8(&go[mine][group][8 * at], v);
            __syncthreads();
            if (group == 0 && live) {
                for (int k = 0; k < GROUPS; ++k) t = fmaxf(t, gm[mine][k]);
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
                for (int k = 0; k < GROUPS; ++k) {
                    const float f = gm[mine][k] == t ? 1.f : ex2(gm[mine][k] - t);
                    float y[8];
                    load8(&go[mine][k][8 * at], y);
                    sum += gl[mine][k] * f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += y[e] * f;
                }
            }
        }
        if (group == 0 && live) {
            const float f = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= f;
            store_row8<WIDE>(a, ((long long)join.q.first + token) * a.out_stride + (long long)head * D + 8 * at, v);
        }
        if constexpr (GROUPS > 1) __syncthreads();
    }
}

// ------------------------------------------------------------------ host side

// Query rows a key/value head of the mean request.
int64_t mean_rows(const AttentionArgs &x) {
    return (x.cache.n_tokens + x.cache.n_req - 1) / x.cache.n_req * (x.n_heads / x.cache.n_kv_heads);
}
// Tiles above 16 rows (bf16) or 32 (f16, whose tiles take two terms).  32 requests of 500 to 4000 positions, few rows / tiles, us at 16 and 32
// rows: bf16, heads of 128 30 / 35, 47 / 36; of 64 34 / 45, 54 / 46; of 256 33 / 47, 52 / 48.  f16, at 32 and 48 rows: 48 / 50, 66 / 51; 54 / 62, 75 / 62;
// 52 / 66, 72 / 69.
[[maybe_unused]] bool on_tiles(const AttentionArgs &x) {
    return x.cache.dtype != HQ_DT_F32 && mean_rows(x) > (x.cache.dtype == HQ_DT_F16 ? 32 : 16);
}
int stream_rows(const AttentionArgs &x) { return mean_rows(x) <= 8 || x.cache.head_dim == 256 ? 8 : 16; }

// MANY rows at once, or two where there are so few items that each may lie on more than 32 blocks.
template <bool WIDE, int D, int MANY>
hq_status run_combine(const AttnArgs &a, int rows, cudaStream_t stream) {
    if (a.blocks < 2 || a.most_units < 2) return HQ_OK;     // an item of one unit is never divided
    const long long items = (a.c.n_tokens / a.tokens + a.c.n_req) * a.c.n_kv_heads * a.parts;  // at most
    const bool few = 32 * items < a.blocks;
    return launch_blocks(few ? attention_combine_kernel<WIDE, D, 2> : attention_combine_kernel<WIDE, D, MANY>,
                         dim3((unsigned)(a.blocks - 1), rows / (few ? 2 : MANY)), kCombineThreads, 0, stream, "attention combine", a, rows);
}

template <bool WIDE, int BITS, int D, int NT>
hq_status run_stream(AttnArgs a, int num_sms, cudaStream_t stream) {
    using S = Stream<WIDE, BITS, D, NT>;
    static std::atomic<bool> done[64];
    hq_status st = allow_smem(attention_stream_kernel<WIDE, BITS, D, NT>, S::SMEM, done);
    if (st != HQ_OK) return st;
    static_assert(kUnit == 1 << 6, "unit_shift");
    deal_rows(a, S::ROWS, D, 6, std::min(kSms, num_sms) * S::MIN_BLOCKS);
    st = launch_blocks(attention_stream_kernel<WIDE, BITS, D, NT>, dim3((unsigned)a.blocks), kThreads, S::SMEM, stream, "attention", a);
    return st != HQ_OK ? st : run_combine<WIDE, D, 2>(a, S::ROWS, stream);
}

template <bool WIDE, int BITS>
hq_status run_dim(const AttentionArgs &x, const AttnArgs &a, int num_sms, cudaStream_t stream) {
    const bool few = stream_rows(x) == 8;
    if (x.cache.head_dim == 256) return run_stream<WIDE, BITS, 256, 1>(a, num_sms, stream);
    if (x.cache.head_dim == 128)
        return few ? run_stream<WIDE, BITS, 128, 1>(a, num_sms, stream) : run_stream<WIDE, BITS, 128, 2>(a, num_sms, stream);
    return few ? run_stream<WIDE, BITS, 64, 1>(a, num_sms, stream) : run_stream<WIDE, BITS, 64, 2>(a, num_sms, stream);
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

// Of tiles: a group of lanes a row.
hq_status run_attention_combine(const AttnArgs &a, int rows, int dim, cudaStream_t stream) {
    return dim == 64    ? run_combine<false, 64, kCombineThreads / 8>(a, rows, stream)
           : dim == 128 ? run_combine<false, 128, kCombineThreads / 16>(a, rows, stream)
                        : run_combine<false, 256, kCombineThreads / 32>(a, rows, stream);
}

// Of the batch and of every one of fewer tokens or requests, whose mean request has group to n_tokens * group query rows a key/value
// head: a buffer for the largest batch serves the others.
int64_t attention_workspace(const AttentionArgs &x) {
    const int dim = x.cache.head_dim;
    const bool wide = x.cache.dtype == HQ_DT_F32;
    auto bytes = [&](int64_t rows, int blocks) {
        return (int64_t)kSms * blocks * (2 * rows * (dim + 2) * 4 + (int64_t)sizeof(Join));
    };
    AttentionArgs least = x, most = x;
    least.cache.n_req = least.cache.n_tokens;
    most.cache.n_req = 1;
    int64_t need = 0;
    for (const int rows : {8, 16})
        if (stream_rows(least) <= rows && rows <= stream_rows(most)) need = std::max(need, bytes(rows, stream_blocks(wide, dim, rows)));
    return on_tiles(most) ? std::max(need, bytes(128, tile_blocks(dim))) : need;
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
    a.window = window_of(x.window, a.c);
    a.partial = static_cast<float *>(x.workspace);
    a.dtype = x.cache.dtype;
    if (on_tiles(x)) return run_attention_tile(a, x.cache.fmt, x.cache.head_dim, dev->num_sms, stream);
    return a.dtype == HQ_DT_F32 ? run_attention_f32(x, a, dev->num_sms, stream) : run_fmt<false>(x, a, dev->num_sms, stream);
}

#endif

}  // namespace hq
