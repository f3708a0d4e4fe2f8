// hq_cache.cu -- rows of new positions into the quantized key/value cache, and
// back out as values.
//
// A lane takes 8 neighbouring elements of a row (16 bytes of a 16-bit type), so a block of 32 is four lanes c = 0..3, and a
// row head_dim / 8 of them.  A key's lane is one word (8 bits: two) of the cell; of the values, element 8 c + g lies
// with the other c of the same g, so four lanes exchange what they hold.
//
// Measured, Q8_0, 8 heads of 128.  Written: 11296 tokens of three prompts, f16 (71 MB in and out), 32 us from a cold start, 2.2 TB/s: bound by
// instructions (0.71 a cycle and scheduler), of which the quotients are the largest part; a division each took 38 us.  Written and
// read back, 62 us with a head a block, 51 with four, 44 without divisions.  Read: the positions of 16 requests, bf16 (563 MB), 120 us = 4.7 TB/s, 0.70 of the copy rate (0.62 a cycle and scheduler, otherwise
// waits for loads of the cells' 2- and 8-byte pieces, four heads' under way at once); a head a block 158.
#include <type_traits>

#include "hq_cache.cuh"

namespace hq {
namespace {

constexpr int kThreads = 256;
constexpr int kFewBlocks = 304;                             // two a multiprocessor

struct RowsArgs {
    CacheView c;
    void *k, *v;                        // token tensors
    long long k_stride, v_stride;
};

// The request of token t, or -1: the last r with offsets[r] <= t, if they rise.  A whole warp, 32 offsets a step.
__device__ __forceinline__ int request_at(const CacheView &c, long long t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = c.n_req;                                // it is in [lo, lo + n), if anywhere
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool in = lane * step < n && c.offsets[lo + min(lane * step, n - 1)] <= t;
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        if (m == 0) return -1;
        const int k = 31 - __clz(m);                        // the last probe at or before t
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Quants of 8 elements of a block of which four neighbouring lanes hold the rest: the scale as it is stored, and the
// unsigned quants, four to a word.  Every operation is fp32, and correctly rounded.
template <int BITS>
__device__ __forceinline__ void quantize8(const float (&w)[8], __half &scale, uint32_t (&q)[2]) {
    float top = 0.f, m = 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(w[i]);
        odd |= !(a < INFINITY);
        if (a > top) { top = a; m = w[i]; }                 // the first of the largest
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        const float ot = __shfl_xor_sync(0xffffffffu, top, d), om = __shfl_xor_sync(0xffffffffu, m, d);
        odd |= __shfl_xor_sync(0xffffffffu, (int)odd, d) != 0;
        if (ot > top || (ot == top && (threadIdx.x & d))) { top = ot; m = om; }
    }
    const float d = BITS == 8 ? fminf(__fdiv_rn(top, 127.f), 65504.f)
                              : fminf(fmaxf(__fdiv_rn(m, -8.f), -65504.f), 65504.f);
    const bool none = odd || d == 0.f;
    // Quotients by the reciprocal and one correction by the remainder are correctly rounded, as the reciprocal is (P. Markstein, IBM Journal of
    // Research and Development 34, 1990, theorem 7), where nothing on the way leaves the normal range; a third of the division's instructions.
    const float inverse = __frcp_rn(d);
    const bool plain = fabsf(d) > 1e-30f;
    scale = odd ? __ushort_as_half(0x7fff) : __float2half_rn(d);
    q[0] = q[1] = 0;
    auto code = [&](int i, float z) {
        uint32_t u;
        if (BITS == 8) u = (uint32_t)(max(-127, min(127, (int)roundf(z))) + 128);
        else u = (uint32_t)max(0, min(15, (int)floorf(__fadd_rn(z, 8.5f))));
        q[i / 4] |= (none ? (BITS == 8 ? 128u : 8u) : u) << (8 * (i % 4));
    };
    if (__all_sync(0xffffffffu, plain || none)) {           // the whole warp
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float z = __fmul_rn(w[i], inverse);
            code(i, __fmaf_rn(__fmaf_rn(-z, d, w[i]), inverse, z));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) code(i, __fdiv_rn(w[i], d));
    }
}

// The rows that a warp handles: R tokens of one head, a row D / 8 lanes.
template <int D>
struct Rows {
    static constexpr int LANES = D / 8, R = 32 / LANES, BLOCK = kThreads / 32 * R;
};

// The search above is for offsets that rise.  Where they do not, it may have passed a good request: then all are looked at, 32 a
// step, and the lowest that has the lane's token counts (r = -1: none).  A whole warp, LANES neighbouring lanes a token.  Not inlined: no call
// with rising offsets comes here but for rows that are no request's, which cost a look at the offsets (16384 such rows behind 64 requests
// written in 41.8 us, 40.0 without the look).
struct Place { int r, p; };
template <int LANES>
__device__ __noinline__ Place place_of(const CacheView &c, long long t) {
    const int lane = threadIdx.x & 31;
    bool falls = false;
#pragma unroll 8
    for (int i = lane; i < c.n_req; i += 32) falls |= c.offsets[i] > c.offsets[i + 1];
    Place at = {-1, 0};
    if (!__any_sync(0xffffffffu, falls)) return at;
    for (int r0 = 0; r0 < c.n_req; r0 += 32) {
        Request q = {0, 0, 0, false};
        if (r0 + lane < c.n_req) q = request_of(c, r0 + lane);
        for (int i = 0; i < 32; i += LANES) {
            const long long x = __shfl_sync(0xffffffffu, t, i);
            const uint32_t m = __ballot_sync(0xffffffffu, x >= q.first && x < (long long)q.first + q.n);
            if (m == 0) continue;
            const int from = __ffs(m) - 1, less = __shfl_sync(0xffffffffu, q.length - q.n - q.first, from);
            if (lane / LANES == i / LANES && at.r < 0) {
                at.r = r0 + from;
                at.p = less + (int)t;
            }
        }
    }
    return at;
}

// Finds the position of this lane's token: request r and position p, or false.
template <int D>
__device__ __forceinline__ bool find_row(const CacheView &c, long long &t, int &r, int &p) {
    using W = Rows<D>;
    const int lane = threadIdx.x & 31, mine = lane / W::LANES;
    const long long t0 = (long long)blockIdx.x * W::BLOCK + (threadIdx.x >> 5) * W::R;
    t = t0 + mine;
    if (t0 >= c.n_tokens) return false;
    int at = request_at(c, t0);
    bool ok = false;
    r = p = 0;
#pragma unroll
    for (int i = 0; i < W::R; ++i) {
        if (i > 0 && t0 + i < c.n_tokens && !(at >= 0 && t0 + i < c.offsets[at + 1])) at = request_at(c, t0 + i);
        if (mine == i && at >= 0 && t < c.n_tokens) {
            const Request q = request_of(c, at);
            ok = !q.bad && t >= q.first && t < (long long)q.first + q.n;
            r = at;
            p = q.length - q.n + (int)(t - q.first);
        }
    }
    if (__any_sync(0xffffffffu, !ok && t < c.n_tokens)) {
        const Place place = place_of<W::LANES>(c, t);
        if (!ok && place.r >= 0 && t < c.n_tokens) {
            ok = true;
            r = place.r;
            p = place.p;
        }
    }
    return ok;
}

// Descriptors out of range are reported once a launch (a request may have no token that looks for it).
__device__ __forceinline__ void check_requests(const CacheView &c) {
    if (blockIdx.x + blockIdx.y != 0) return;
    for (int r = threadIdx.x; r < c.n_req; r += kThreads)
        if (request_of(c, r).bad) atomicOr(c.fault, kFaultCache);
}

// 16 bytes (fp32: 32) of a token's row, as they come.
template <class T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const { load8(reinterpret_cast<const T *>(w), v); }
};

// A warp's rows, of HEADS heads: what finding them costs is paid once, and the heads' loads are under way together.
template <class T, int BITS, int D, int HEADS>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 4 : 2)) cache_write_kernel(const __grid_constant__ RowsArgs a) {
    using L = CellLayout<BITS, D>;
    griddep_launch_dependents();
    griddep_wait();
    check_requests(a.c);
    long long t;
    int r, p;
    const bool ok = find_row<D>(a.c, t, r, p) && p >= 0;
    const int head = blockIdx.y * HEADS, heads = min(HEADS, a.c.n_kv_heads - head);
    uint8_t *cell0 = nullptr;
    if (ok) {
        uint8_t *cells = page_cells(a.c, r, p, head);
        if (cells) cell0 = cell_of<L>(a.c, cells, p);
    }
    const int at = threadIdx.x & (Rows<D>::LANES - 1), b = at / 4, g = at % 4, pos = p & (kCell - 1);
    Raw8<T> k[HEADS], v[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
        if (cell0 && h < heads) {
            k[h].load(static_cast<const T *>(a.k) + t * a.k_stride + (head + h) * D + 8 * at);
            v[h].load(static_cast<const T *>(a.v) + t * a.v_stride + (head + h) * D + 8 * at);
        }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        uint8_t *cell = cell0 && h < heads ? cell0 + h * a.c.head_bytes : nullptr;
        float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        __half scale;
        uint32_t q[2];
        if (cell) k[h].values(w);
        quantize8<BITS>(w, scale, q);
        if (cell) {
            if (BITS == 8) {
                *reinterpret_cast<uint2 *>(cell + L::k_word(pos, g, 2 * b)) = make_uint2(q[0], q[1]);
            } else {
                // bytes e0 e1 e2 e3 | e4 .. e7 -> nibbles e0 e2 e4 e6 e1 e3 e5 e7
                const uint32_t lo = q[0] | (q[0] >> 12), hi = q[1] | (q[1] >> 12);  // byte 0: e0 | e2 << 4, byte 1: e1 | e3 << 4
                *reinterpret_cast<uint32_t *>(cell + L::k_word(pos, g, b)) = prmt(lo, hi, 0x5140);
            }
            if (g == 0) *reinterpret_cast<__half *>(cell + L::k_scale(pos, b)) = scale;
            v[h].values(w);
        }
        quantize8<BITS>(w, scale, q);
        // lane c holds elements 8 c + g, g = 0..7; it gets those of g = 2 c and 2 c + 1, of all four lanes:
        // a 4 x 4 transposition of pairs of bytes
        const uint32_t s0 = __shfl_xor_sync(0xffffffffu, (g & 2) ? q[0] : q[1], 2);
        const uint32_t own = (g & 2) ? q[1] : q[0];         // bytes g = 4 (c / 2) .. + 3 of this lane and of lane c ^ 2
        const uint32_t x0 = (g & 2) ? s0 : own, x1 = (g & 2) ? own : s0;            // of j = c % 2, and of j = 2 + c % 2
        const uint32_t give = (g & 1) ? prmt(x0, x1, 0x5410) : prmt(x0, x1, 0x7632);
        const uint32_t keep = (g & 1) ? prmt(x0, x1, 0x7632) : prmt(x0, x1, 0x5410);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
        const uint32_t j0 = (g & 1) ? got : keep, j1 = (g & 1) ? keep : got;        // bytes: j0: (j 0: g, g+1; j 2: g, g+1), j1: j 1 and 3
        if (cell) {
            const int odd = pos & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t j = prmt(j0, j1, i == 0 ? 0x6240 : 0x7351);          // bytes j = 0, 1, 2, 3 of g = 2 c + i
                if (BITS == 8) {
                    *reinterpret_cast<uint16_t *>(cell + L::v_word(pos / 2, 2 * g + i, 2 * b) + 2 * odd) = (uint16_t)j;
                    *reinterpret_cast<uint16_t *>(cell + L::v_word(pos / 2, 2 * g + i, 2 * b + 1) + 2 * odd) = (uint16_t)(j >> 16);
                } else {
                    const uint32_t n = j | (j >> 4);        // bytes 0 and 2: j 0 | j 1 << 4, j 2 | j 3 << 4
                    *reinterpret_cast<uint16_t *>(cell + L::v_word(pos / 2, 2 * g + i, b) + 2 * odd) = (uint16_t)prmt(n, 0, 0x4420);
                }
            }
            if (g == 0) *reinterpret_cast<__half *>(cell + L::v_scale(pos, b)) = scale;
        }
    }
}

template <class T, int BITS, int D, int HEADS>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 4 : 2)) cache_read_kernel(const __grid_constant__ RowsArgs a) {
    using L = CellLayout<BITS, D>;
    griddep_launch_dependents();
    griddep_wait();
    check_requests(a.c);
    long long t;
    int r, p;
    const bool ok = find_row<D>(a.c, t, r, p);
    const int head = blockIdx.y * HEADS, heads = min(HEADS, a.c.n_kv_heads - head);
    const uint8_t *cell = nullptr;
    float other = 0.f;                                      // what a row without a cell reads as
    if (ok && p >= 0) {
        uint8_t *cells = page_cells(a.c, r, p, head);
        if (cells) cell = cell_of<L>(a.c, cells, p);
        else other = __uint_as_float(0x7fffffffu);
    }
    const int at = threadIdx.x & (Rows<D>::LANES - 1), b = at / 4, g = at % 4, pos = p & (kCell - 1), odd = pos & 1;
    __half ks[HEADS], vs[HEADS];
    uint2 k[HEADS];
    uint16_t v[HEADS][2][BITS / 4];                         // the values' halves of words of g = 2 c and 2 c + 1
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        k[h] = make_uint2(0, 0);
        ks[h] = vs[h] = __ushort_as_half(0);
#pragma unroll
        for (int i = 0; i < BITS / 2; ++i) v[h][i / (BITS / 4)][i % (BITS / 4)] = 0;
        if (cell && h < heads) {
            const uint8_t *from = cell + h * a.c.head_bytes;
            ks[h] = *reinterpret_cast<const __half *>(from + L::k_scale(pos, b));
            vs[h] = *reinterpret_cast<const __half *>(from + L::v_scale(pos, b));
            if (BITS == 8) k[h] = *reinterpret_cast<const uint2 *>(from + L::k_word(pos, g, 2 * b));
            else k[h].x = *reinterpret_cast<const uint32_t *>(from + L::k_word(pos, g, b));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < BITS / 4; ++n)
                    v[h][i][n] = *reinterpret_cast<const uint16_t *>(from + L::v_word(pos / 2, 2 * g + i, BITS / 4 * b + n) + 2 * odd);
        }
    }
    constexpr float kMid = BITS == 8 ? 128.f : 8.f;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        uint32_t q[2] = {k[h].x, k[h].y};
        if (BITS == 4) {                                    // nibbles e0 e2 e4 e6 e1 e3 e5 e7 -> bytes e0..e3, e4..e7
            const uint32_t n = prmt(q[0], 0, 0x3120);       // bytes: e0 e2 | e1 e3 | e4 e6 | e5 e7
            const uint32_t lo = n & 0x0f0f0f0fu, hi = (n >> 4) & 0x0f0f0f0fu;
            q[0] = prmt(lo, hi, 0x5410);                    // lo: e0 e1 e4 e5, hi: e2 e3 e6 e7
            q[1] = prmt(lo, hi, 0x7632);
        }
        float w[8];
        const float dk = __half2float(ks[h]), dv = __half2float(vs[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = cell ? ((float)((q[i / 4] >> (8 * (i % 4))) & 0xffu) - kMid) * dk : other;
        if (ok && h < heads) store8(static_cast<T *>(a.k) + t * a.k_stride + (head + h) * D + 8 * at, w);
        uint32_t j[2];                                      // j[i]: bytes j = 0..3 of g = 2 c + i
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t n = v[h][i][0];
            j[i] = BITS == 8 ? n | (uint32_t)v[h][i][BITS / 4 - 1] << 16
                             : (n & 0xfu) | ((n & 0xf0u) << 4) | ((n & 0xf00u) << 8) | ((n & 0xf000u) << 12);
        }
        // the transposition of the write, backwards
        const uint32_t j0 = prmt(j[0], j[1], 0x6240), j1 = prmt(j[0], j[1], 0x7351);    // (j 0: g, g+1; j 2: g, g+1), (j 1; j 3)
        const uint32_t got = __shfl_xor_sync(0xffffffffu, (g & 1) ? j0 : j1, 1);
        const uint32_t keep = (g & 1) ? j1 : j0;
        const uint32_t x0 = (g & 1) ? prmt(got, keep, 0x5410) : prmt(keep, got, 0x5410);
        const uint32_t x1 = (g & 1) ? prmt(got, keep, 0x7632) : prmt(keep, got, 0x7632);
        const uint32_t s0 = __shfl_xor_sync(0xffffffffu, (g & 2) ? x0 : x1, 2);
        q[0] = (g & 2) ? s0 : x0;
        q[1] = (g & 2) ? x1 : s0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = cell ? ((float)((q[i / 4] >> (8 * (i % 4))) & 0xffu) - kMid) * dv : other;
        if (ok && h < heads) store8(static_cast<T *>(a.v) + t * a.v_stride + (head + h) * D + 8 * at, w);
    }
}

template <class T, int BITS, int D, int HEADS>
hq_status launch_rows(bool write, const RowsArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.c.n_tokens + Rows<D>::BLOCK - 1) / Rows<D>::BLOCK), (unsigned)((a.c.n_kv_heads + HEADS - 1) / HEADS));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, write ? cache_write_kernel<T, BITS, D, HEADS> : cache_read_kernel<T, BITS, D, HEADS>, a);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "cache %s launch: %s", write ? "write" : "read", cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

// Four heads a block where that leaves blocks for every multiprocessor (16 requests read 120 us, a head a block 158); few rows spread over
// more blocks (64 tokens: a block each of 8 tokens and a head).
template <class T, int BITS, int D>
hq_status launch_heads(bool write, const RowsArgs &a, cudaStream_t stream) {
    const long long blocks = (a.c.n_tokens + Rows<D>::BLOCK - 1) / Rows<D>::BLOCK * a.c.n_kv_heads;
    return blocks > 4 * kFewBlocks ? launch_rows<T, BITS, D, 4>(write, a, stream) : launch_rows<T, BITS, D, 1>(write, a, stream);
}

template <class T, int BITS>
hq_status launch_dim(bool write, int dim, const RowsArgs &a, cudaStream_t stream) {
    if (dim == 64) return launch_heads<T, BITS, 64>(write, a, stream);
    if (dim == 128) return launch_heads<T, BITS, 128>(write, a, stream);
    return launch_heads<T, BITS, 256>(write, a, stream);
}

template <class T>
hq_status launch_bits(bool write, const CacheArgs &c, const RowsArgs &a, cudaStream_t stream) {
    return c.fmt == HQ_FMT_Q8_0 ? launch_dim<T, 8>(write, c.head_dim, a, stream) : launch_dim<T, 4>(write, c.head_dim, a, stream);
}

hq_status launch_all(bool write, const CacheArgs &c, void *k, int64_t k_stride, void *v, int64_t v_stride,
                     cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    const RowsArgs a = {cache_view(c, dev->fault), k, v, k_stride, v_stride};
    switch (c.dtype) {
        case HQ_DT_F32: return launch_bits<float>(write, c, a, stream);
        case HQ_DT_F16: return launch_bits<__half>(write, c, a, stream);
        default: return launch_bits<__nv_bfloat16>(write, c, a, stream);
    }
}

}  // namespace

hq_status launch_cache_write(const CacheArgs &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             cudaStream_t stream) {
    return launch_all(true, c, const_cast<void *>(k), k_stride, const_cast<void *>(v), v_stride, stream);
}

hq_status launch_cache_read(const CacheArgs &c, void *k, int64_t k_stride, void *v, int64_t v_stride,
                            cudaStream_t stream) {
    return launch_all(false, c, k, k_stride, v, v_stride, stream);
}

}  // namespace hq
