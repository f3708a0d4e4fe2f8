// hq_verify.cu -- probabilities of logits (one temperature per row) and the
// verification of drafted tokens against them.
//
// Both read a row of the vocabulary (0.5 MB) once and are bound by that read, or at few rows by
// the chain of latencies around it.  A thread-block cluster takes a row, a contiguous part per
// CTA, so that few rows still occupy several SMs; the parts' results are exchanged
// through distributed shared memory.
//
// Measured: softmax of 512 rows of 128256 fp32 columns 155 us, 3.4 TB/s read and written, at half the issue
// slots (43 instructions a column, most of them the accurate power) and with phases that do not overlap inside a block; 5 rows of
// 151936 10 us, three passes over a part and an exchange, on the 40 multiprocessors that clusters of eight occupy.
// Verification of 64 requests of 0 to 7 drafts 31 us, 2.1 TB/s; of one 11 us.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "hq_device.cuh"
#include "hq_internal.h"

namespace hq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kPartCols = 25600;            // softmax: columns of a row's part that shared memory keeps (100 KB)

// ------------------------------------------------------------------ softmax

template <class T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void get8(const float *p, float (&v)[8]) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <> struct Elem<__half> {
    static __device__ __forceinline__ float get(const __half *p) { return __half2float(*p); }
    static __device__ __forceinline__ void get8(const __half *p, float (&v)[8]) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void get8(const __nv_bfloat16 *p, float (&v)[8]) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

struct SoftmaxArgs {
    const void *logits;
    const float *temperature;
    float *p;
    int vocab, cluster, part;       // columns of a CTA's part, a multiple of 8
    int vector;                     // both pointers are 16-byte aligned
};

// The first maximum over the block of (value, column); every thread gets it.
__device__ __forceinline__ void block_first_max(float &m, int &at, float *red, int *redi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int round = 0; round < 2; ++round) {
        for (int d = 16; d > 0; d >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, d);
            const int oa = __shfl_xor_sync(0xffffffffu, at, d);
            if (om > m || (om == m && oa < at)) { m = om; at = oa; }
        }
        if (round == 0) {
            if (lane == 0) { red[warp] = m; redi[warp] = at; }
            __syncthreads();
            m = lane < kWarps ? red[lane] : -INFINITY;
            at = lane < kWarps ? redi[lane] : 0x7fffffff;
        }
    }
}

// A row: the part's maximum m_c, e = exp((l - m_c) / t) and their sum s_c; with the row's maximum M and
// sum S = sum_c s_c exp((m_c - M) / t) of the cluster, p = e exp((m_c - M) / t) / S.  One exponential an element, and
// the part stays in shared memory (CACHED) between the steps; a row too long for that is read three times.
// 8 neighbouring columns a thread, aligned in memory: column i is at virtual place i + head.
template <class T, bool CACHED>
__global__ void __launch_bounds__(kThreads) softmax_kernel(SoftmaxArgs a) {
    extern __shared__ float keep[];
    __shared__ float red[kWarps], red2[kWarps], peer_m[kMaxCluster], peer_s[kMaxCluster];
    __shared__ int redi[kWarps], peer_at[kMaxCluster];
    if (a.cluster > 1) cluster_arrive_relaxed();
    griddep_launch_dependents();
    griddep_wait();
    const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
    const long long row = blockIdx.x / a.cluster;
    const T *l = static_cast<const T *>(a.logits) + row * a.vocab;
    float *o = a.p + row * a.vocab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const int head = (int)(row * a.vocab & 7);
    const int lo = rank * a.part - head, hi = lo + a.part;  // columns of this part, cut to [0, vocab) below

    auto load = [&](int i, float (&v)[8]) {
        if (a.vector && i >= 0 && i + 8 <= a.vocab) {
            Elem<T>::get8(l + i, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k >= 0 && i + k < a.vocab ? Elem<T>::get(l + i + k) : -INFINITY;
        }
    };
    auto put8 = [&](int i, const float (&v)[8]) {           // to shared memory
        float4 *q = reinterpret_cast<float4 *>(keep + (i - lo));
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    };
    auto take8 = [&](int i, float (&v)[8]) {
        const float4 *q = reinterpret_cast<const float4 *>(keep + (i - lo));
        const float4 x = q[0], y = q[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    };
    auto store = [&](int i, const float (&v)[8]) {
        if (a.vector && i >= 0 && i + 8 <= a.vocab) {
            float4 *q = reinterpret_cast<float4 *>(o + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) if (i + k >= 0 && i + k < a.vocab) o[i + k] = v[k];
        }
    };
    const int end = min(hi, a.vocab);
    const bool greedy = !(t > 0.f);
    float m = -INFINITY;
    int at = 0x7fffffff;
    if (greedy) {
        for (int i = lo + 8 * (int)threadIdx.x; i < end; i += 8 * kThreads) {
            float v[8];
            load(i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) if (v[k] > m) { m = v[k]; at = i + k; }
        }
    } else {
#pragma unroll 2
        for (int i = lo + 8 * (int)threadIdx.x; i < end; i += 8 * kThreads) {
            float v[8];
            load(i, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k]);
            if (CACHED) put8(i, v);
        }
    }
    block_first_max(m, at, red, redi);

    float s = 0.f;
    const float mc = m == -INFINITY ? 0.f : m;
    // e^((v - mc) / t) of 8 columns.  Mode 0: t is 1.  Otherwise the quotient is a product with 1/t and one correction by its
    // remainder, three instructions for a division's ten; z is cut at -200 t, whose power is 0 as well, so that the
    // remainder of -inf is no NaN (a NaN stays).  Mode 2 keeps 1/t and the cut in range: a large t is taken in units of 2^64, and
    // so are the values, whose difference may be too large a float and still count (an infinite t: 1e30 of them, which makes
    // every finite difference 0); for a small t the differences are taken in units of 2^-64.
    const bool large = t >= 1e18f;
    const int mode = t == 1.f ? 0 : t > 1e-18f && !large ? 1 : 2;
    const float unit = large ? 0x1p-64f : 1.f, back = mode == 2 && !large ? 0x1p64f : 1.f;
    const float ut = large ? fminf(t * 0x1p-64f, 1e30f) : t * back, rt = __frcp_rn(ut), least = -200.f * ut;
    auto power = [&](auto which, float (&v)[8]) {
        constexpr int MODE = decltype(which)::value;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float z = MODE == 2 ? (v[k] * unit - mc * unit) * back : v[k] - mc;
            if constexpr (MODE > 0) {
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(z) : "f"(least));
                const float q = z * rt;
                z = fmaf(fmaf(-q, ut, z), rt, q);
            }
            v[k] = expf(z);
        }
    };
    auto sum = [&](auto which) {
        for (int i = lo + 8 * (int)threadIdx.x; i < end; i += 8 * kThreads) {
            float v[8];
            if (CACHED) take8(i, v); else load(i, v);
            power(which, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
            if (CACHED) put8(i, v);
        }
    };
    if (!greedy) {
        if (mode == 0) sum(std::integral_constant<int, 0>());
        else if (mode == 1) sum(std::integral_constant<int, 1>());
        else sum(std::integral_constant<int, 2>());
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) red2[warp] = s;
        __syncthreads();
        s = lane < kWarps ? red2[lane] : 0.f;
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    float M = m, S = s, mine = 1.f;
    if (a.cluster > 1) {
        cluster_wait();                                     // the peers run: their shared memory may be written
        if (threadIdx.x < a.cluster) {
            st_shared_cluster_f32(map_shared_rank(smem_u32(&peer_m[rank]), threadIdx.x), m);
            st_shared_cluster_f32(map_shared_rank(smem_u32(&peer_s[rank]), threadIdx.x), s);
            st_shared_cluster_s32(map_shared_rank(smem_u32(&peer_at[rank]), threadIdx.x), at);
        }
        cluster_sync();
        for (int r = 0; r < a.cluster; ++r)
            if (peer_m[r] > M || (peer_m[r] == M && peer_at[r] < at)) { M = peer_m[r]; at = peer_at[r]; }
        S = 0.f;
        // a part of nothing but -inf (m_c = -inf) has the sum 0, or NaN
        for (int r = 0; r < a.cluster; ++r) {
            const float f = peer_m[r] == -INFINITY ? 1.f : expf(__fdiv_rn((peer_m[r] * unit - M * unit) * back, ut));
            if (r == rank) mine = f;
            S += greedy ? 0.f : peer_s[r] * f;
        }
    }
    if (greedy) {
        for (int i = lo + 8 * (int)threadIdx.x; i < end; i += 8 * kThreads) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k == at ? 1.f : 0.f;
            store(i, v);
        }
        return;
    }
    const float scale = S == 0.f ? 0.f : __fdiv_rn(mine, S);
    auto finish = [&](auto which) {
        for (int i = lo + 8 * (int)threadIdx.x; i < end; i += 8 * kThreads) {
            float v[8];
            if (CACHED) take8(i, v); else { load(i, v); power(which, v); }
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= scale;
            store(i, v);
        }
    };
    if (CACHED || mode == 0) finish(std::integral_constant<int, 0>());
    else if (mode == 1) finish(std::integral_constant<int, 1>());
    else finish(std::integral_constant<int, 2>());
}

// ------------------------------------------------------------------ verification

// floor(2^40 s), s clamped to [0, 1], NaN as 0: integer sums do not depend on their order
__device__ __forceinline__ unsigned long long fixed40(float s) {
    const float c = fminf(fmaxf(s, 0.f), 1.f);          // fmaxf(NaN, 0) = 0
    return (unsigned long long)(c * 1099511627776.f);   // the product by 2^40 is exact
}

struct VerifyArgs {
    const float *p, *q;
    const int32_t *drafts, *off;
    const float *u_accept, *u_sample;
    int32_t *n_accepted, *tokens;
    int n_req, n_drafts, vocab, cluster, vector;
    uint32_t *fault;
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// A cluster takes a request.  Every warp finds the accepted drafts by itself (a lane a draft), and owns a contiguous
// part of the vocabulary, of which it sums the integers of the residual.  The sums tell which warp holds the
// sampled token; that warp reads its part again (from L1 or L2) and finds it.  One request: that chain of reads and two
// exchanges, 11 us (17 us with nothing in L2 or the instruction caches).  64 requests, whose rows of p and q are 66 MB: 31 us; of their 512
// blocks 456 fit at once (40 registers a thread), so that seven clusters run behind the others.
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
    __shared__ unsigned long long sums[kWarps], peer[2][kMaxCluster];
    if (a.cluster > 1) cluster_arrive_relaxed();
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
    const long long r = blockIdx.x / a.cluster;
    const long long o0 = a.off[r], o1 = a.off[r + 1];
    const bool lead = rank == 0 && threadIdx.x == 0;
    const float us = a.u_sample[r] * 16777216.f;
    if (o0 < 0 || o1 < o0 || o1 > a.n_drafts || (r == 0 && o0 != 0) || (r == a.n_req - 1 && o1 != a.n_drafts)) {
        if (lead) atomicOr(a.fault, kFaultDraft);
        if (a.cluster > 1) cluster_wait();
        return;                                             // the whole cluster
    }
    const int n = (int)(o1 - o0);
    int acc = n, refused = -1;                              // the first refused draft and its token
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        bool ok = true, bad = false;
        int d = -1;
        if (i < n) {
            d = a.drafts[o0 + i];
            bad = d < 0 || d >= a.vocab;
            ok = false;
            if (!bad) {
                const float qd = a.q ? a.q[(o0 + i) * a.vocab + d] : 1.f;
                ok = __fmul_rn(a.u_accept[o0 + i], qd) < a.p[(o0 + r + i) * a.vocab + d];
            }
        }
        const uint32_t no = __ballot_sync(0xffffffffu, !ok);
        if (no) {
            const int f = __ffs(no) - 1;
            acc = i0 + f;
            refused = __shfl_sync(0xffffffffu, d, f);
            bad = __shfl_sync(0xffffffffu, bad, f);
            if (lead && bad) atomicOr(a.fault, kFaultDraft);
            break;
        }
    }
    const float *p = a.p + (o0 + r + acc) * a.vocab;
    const float *q = acc < n && a.q ? a.q + (o0 + acc) * a.vocab : nullptr;
    const int sure = acc < n && !a.q ? refused : -1;
    // parts of a multiple of 128 columns
    const int part = ((a.vocab + a.cluster * kWarps - 1) / (a.cluster * kWarps) + 127) & ~127;
    const int lo = (int)min((long long)(rank * kWarps + warp) * part, (long long)a.vocab);
    const int hi = (int)min((long long)lo + part, (long long)a.vocab);
    bool residual = acc < n;
    // the integers of columns j .. j + 3
    auto steps = [&](int j, unsigned long long (&v)[4]) {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.vector && j + 4 <= hi) {
            const float4 x = *reinterpret_cast<const float4 *>(p + j);
            s[0] = x.x; s[1] = x.y; s[2] = x.z; s[3] = x.w;
            if (residual && q) {
                const float4 y = *reinterpret_cast<const float4 *>(q + j);
                w[0] = y.x; w[1] = y.y; w[2] = y.z; w[3] = y.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < hi) {
                    s[k] = p[j + k];
                    if (residual && q) w[k] = q[j + k];
                }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (residual && j + k == sure) w[k] = 1.f;
            v[k] = fixed40(__fsub_rn(s[k], w[k]));
        }
    };
    unsigned long long total = 0, before = 0, own = 0;      // of the row, before this warp, of this warp
    for (int tries = 0; tries < 2; ++tries) {
        own = 0;
#pragma unroll 4
        for (int j = lo + 4 * lane; j < hi; j += 128) {
            unsigned long long v[4];
            steps(j, v);
            own += v[0] + v[1] + v[2] + v[3];
        }
        own = warp_sum(own);
        __syncthreads();
        if (lane == 0) sums[warp] = own;
        __syncthreads();
        const unsigned long long w = lane < kWarps ? sums[lane] : 0ull;
        before = warp_sum(lane < warp ? w : 0ull);
        total = warp_sum(w);
        if (a.cluster > 1) {
            if (tries == 0) cluster_wait();                 // the peers run: their shared memory may be written
            if (threadIdx.x < a.cluster) {
                const uint32_t to = map_shared_rank(smem_u32(&peer[tries][rank]), threadIdx.x);
                st_shared_cluster_s32(to, (int)(uint32_t)total);
                st_shared_cluster_s32(to + 4, (int)(uint32_t)(total >> 32));
            }
            cluster_sync();
            const unsigned long long c = lane < a.cluster ? peer[tries][lane] : 0ull;
            before += warp_sum(lane < rank ? c : 0ull);
            total = warp_sum(c);
        }
        if (total || !residual) break;
        residual = false;                                   // the residual is empty: the target itself
    }
    int32_t *out = a.tokens + o0 + r;
    if (rank == 0) {
        if (threadIdx.x == 0) a.n_accepted[r] = acc;
        for (int i = threadIdx.x; i <= n; i += kThreads)
            if (i != acc || total == 0) out[i] = i < acc ? a.drafts[o0 + i] : -1;
    }
    const unsigned long long U = us >= 16777215.f ? 16777215ull : us > 0.f ? (unsigned long long)us : 0ull;
    const unsigned long long goal = (total >> 24) * U + (((total & 0xffffffull) * U) >> 24);
    // the lowest column whose running sum passes the goal, in the one warp that holds it
    if (before > goal || before + own <= goal) return;
    for (int j0 = lo; j0 < hi; j0 += 128) {
        unsigned long long v[4];
        const int j = j0 + 4 * lane;
        steps(j, v);
        const unsigned long long mine = v[0] + v[1] + v[2] + v[3];
        unsigned long long inc = mine;
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long w = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += w;
        }
        const unsigned long long b = before + inc - mine;
        if (b <= goal && b + mine > goal) {
            unsigned long long run = b;
            int k = 0;
            for (; k < 3 && run + v[k] <= goal; ++k) run += v[k];
            out[acc] = j + k;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        if (before > goal) return;
    }
}

// ------------------------------------------------------------------ host side

template <class K, class A>
hq_status launch(K kern, long long rows, int cluster, size_t smem, cudaStream_t stream, const char *what, const A &args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cluster));
    cfg.blockDim = dim3((unsigned)kThreads);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "%s launch: %s", what, cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

template <class T>
hq_status softmax_rows(const SoftmaxArgs &a, long long rows, cudaStream_t stream) {
    if (a.part > kPartCols) return launch(softmax_kernel<T, false>, rows, a.cluster, 0, stream, "softmax", a);
    static std::atomic<bool> done[64];
    int d = 0;
    cudaGetDevice(&d);
    if (d < 0 || d >= 64 || !done[d].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(softmax_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPartCols * 4);
        if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        if (d >= 0 && d < 64) done[d].store(true, std::memory_order_release);
    }
    return launch(softmax_kernel<T, true>, rows, a.cluster, (size_t)a.part * 4, stream, "softmax", a);
}

}  // namespace

hq_status launch_softmax(const void *logits, const float *temperature, float *p, int64_t n_rows, int64_t vocab,
                         int dtype, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    SoftmaxArgs a = {logits, temperature, p, (int)vocab, 1, 0, 0};
    // a part of at least one pass of the block; as many parts as the cluster allows
    while (a.cluster < kMaxCluster && vocab > (int64_t)a.cluster * 8 * kThreads) a.cluster *= 2;
    a.part = (int)(((vocab + 7 + a.cluster - 1) / a.cluster + 7) / 8 * 8);     // 7: the head of an unaligned row
    a.vector = ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(p)) & 15) == 0;
    switch (dtype) {
        case HQ_DT_F32: return softmax_rows<float>(a, n_rows, stream);
        case HQ_DT_F16: return softmax_rows<__half>(a, n_rows, stream);
        default: return softmax_rows<__nv_bfloat16>(a, n_rows, stream);
    }
}

hq_status launch_verify(const float *p, const float *q, const int32_t *drafts, const int32_t *off,
                        const float *u_accept, const float *u_sample, int32_t *n_accepted, int32_t *tokens,
                        int64_t n_req, int64_t n_drafts, int64_t vocab, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    int cluster = 1;
    while (cluster < kMaxCluster && vocab > (int64_t)cluster * 4 * kThreads) cluster *= 2;
    const int vector = vocab % 4 == 0 && ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    VerifyArgs a{p, q, drafts, off, u_accept, u_sample, n_accepted, tokens, (int)n_req, (int)n_drafts, (int)vocab,
                 cluster, vector, dev->fault};
    return launch(verify_kernel, n_req, cluster, 0, stream, "verify", a);
}

}  // namespace hq
