// hq_cache.cuh -- the key/value cache in memory (see include/hq.h), and which
// positions of it a request's tokens are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hq_device.cuh"
#include "hq_internal.h"

namespace hq {

constexpr int kCell = 16;                                   // positions that lie together

// Offsets (bytes) in a cell of BITS-bit quants and heads of D.  A lane's bytes, LANE, are those of a quarter of a key's row, or
// of an eighth of the values of two neighbouring positions; words of a lane follow the blocks (8 bits: two words a block).
template <int BITS, int D>
struct CellLayout {
    static constexpr int NB = D / 32;                       // blocks of a row
    static constexpr int RB = D * BITS / 8;                 // bytes of a row's quants
    static constexpr int LANE = RB / 4;
    static constexpr int UB = LANE < 16 ? LANE : 16;        // a unit: what a lane loads at once
    static constexpr int UNITS = LANE / UB;
    static constexpr int UW = UB / 4;                       // words of a unit
    static constexpr int V0 = kCell * RB, KS = 2 * kCell * RB, VS = KS + kCell * NB * 2;
    static constexpr int BYTES = VS + kCell * NB * 2;
    static __device__ __forceinline__ int k_word(int pos, int c, int w) {
        return pos * RB + w / UW * (4 * UB) + c * UB + w % UW * 4;
    }
    static __device__ __forceinline__ int v_word(int pair, int g, int w) {
        return V0 + pair * (2 * RB) + w / UW * (8 * UB) + g * UB + w % UW * 4;
    }
    static __device__ __forceinline__ int k_scale(int pos, int b) { return KS + (pos * NB + b) * 2; }
    static __device__ __forceinline__ int v_scale(int pos, int b) { return VS + ((pos / 2 * NB + b) * 2 + pos % 2) * 2; }
};

// What a kernel gets of a cache and its batch.
struct CacheView {
    uint8_t *pool;
    const int32_t *page_table, *offsets, *lengths;
    long long n_pages, table_width, head_bytes;             // head_bytes: of a page's cells of one head
    long long n_tokens;
    int n_req, page_shift, n_kv_heads;
    uint32_t *fault;
};

inline CacheView cache_view(const CacheArgs &c, uint32_t *fault) {
    CacheView v;
    v.pool = c.pool;
    v.page_table = c.page_table;
    v.offsets = c.offsets;
    v.lengths = c.lengths;
    v.n_pages = c.n_pages;
    v.table_width = c.table_width;
    v.head_bytes = (long long)c.page_size * 2 * (c.head_dim * (c.fmt == HQ_FMT_Q8_0 ? 8 : 4) / 8 + c.head_dim / 16);
    v.n_tokens = c.n_tokens;
    v.n_req = (int)c.n_req;
    v.page_shift = 0;
    while ((16 << v.page_shift) < c.page_size) ++v.page_shift;
    v.page_shift += 4;
    v.n_kv_heads = c.n_kv_heads;
    v.fault = fault;
    return v;
}

// A request's tokens and positions; n = 0 where the descriptor is out of range (`bad`) or it brings none.
struct Request {
    int first, n, length;
    bool bad;
};
__device__ __forceinline__ Request request_of(const CacheView &c, int r) {
    const int o0 = c.offsets[r], o1 = c.offsets[r + 1], len = c.lengths[r];
    Request q;
    q.bad = o0 < 0 || o1 < o0 || o1 > c.n_tokens || len < 0 || len > c.table_width << c.page_shift;
    q.first = q.bad ? 0 : o0;
    q.n = q.bad ? 0 : o1 - o0;
    q.length = q.bad ? 0 : len;
    return q;
}

// The cells of `head` of the page that holds position p of request r, or null (and the fault) for a page out of range.
__device__ __forceinline__ uint8_t *page_cells(const CacheView &c, int r, int p, int head) {
    const int page = c.page_table[r * c.table_width + (p >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) {
        atomicOr(c.fault, kFaultCache);
        return nullptr;
    }
    return c.pool + ((long long)page * c.n_kv_heads + head) * c.head_bytes;
}

// A position's cell in its page.
template <class L>
__device__ __forceinline__ uint8_t *cell_of(const CacheView &c, uint8_t *cells, int p) {
    return cells + (long long)((p & ((1 << c.page_shift) - 1)) / kCell) * L::BYTES;
}

// 8 neighbouring elements of a token's row <-> fp32.
template <class T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            else f = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <class T>
__device__ __forceinline__ T to_elem(float v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

template <class T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T e[2] = {to_elem<T>(v[2 * i]), to_elem<T>(v[2 * i + 1])};
            u[i] = *reinterpret_cast<const uint32_t *>(e);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

}  // namespace hq
