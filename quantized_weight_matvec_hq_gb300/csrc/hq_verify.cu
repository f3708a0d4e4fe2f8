// hq_verify.cu -- probabilities of logits (one temperature per row) and the
// verification of drafted tokens against them.
#include <cuda_bf16.h>

#include "hq_device.cuh"
#include "hq_internal.h"

namespace hq {
namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// ------------------------------------------------------------------ softmax

template <class T>
__global__ void __launch_bounds__(kThreads) softmax_kernel(const T *__restrict__ logits,
                                                           const float *__restrict__ temperature, float *p,
                                                           long long vocab) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float red[32];
    __shared__ int redi[32];
    const long long row = blockIdx.x;
    const T *l = logits + row * vocab;
    float *o = p + row * vocab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float t = temperature ? temperature[row] : 1.f;
    float m = -INFINITY;
    int at = 0x7fffffff;
    for (long long j = threadIdx.x; j < vocab; j += kThreads) {
        const float v = to_float(l[j]);
        if (v > m) { m = v; at = (int)j; }
    }
    for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, d);
        const int oa = __shfl_xor_sync(0xffffffffu, at, d);
        if (om > m || (om == m && oa < at)) { m = om; at = oa; }
    }
    if (lane == 0) { red[warp] = m; redi[warp] = at; }
    __syncthreads();
    m = red[lane];
    at = redi[lane];
    for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, d);
        const int oa = __shfl_xor_sync(0xffffffffu, at, d);
        if (om > m || (om == m && oa < at)) { m = om; at = oa; }
    }
    if (!(t > 0.f)) {
        __syncthreads();
        for (long long j = threadIdx.x; j < vocab; j += kThreads) o[j] = j == at ? 1.f : 0.f;
        return;
    }
    if (m == -INFINITY) m = 0.f;
    float s = 0.f;
    for (long long j = threadIdx.x; j < vocab; j += kThreads) s += expf((to_float(l[j]) - m) / t);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    __syncthreads();
    if (lane == 0) red[warp] = s;
    __syncthreads();
    s = red[lane];
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    for (long long j = threadIdx.x; j < vocab; j += kThreads) {
        const float e = expf((to_float(l[j]) - m) / t);
        o[j] = s == 0.f ? 0.f : e / s;
    }
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
    long long n_req, n_drafts;
    int vocab;
    uint32_t *fault;
};

__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = red[lane];
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ unsigned long long red[32];
    const long long r = blockIdx.x;
    const long long o0 = a.off[r], o1 = a.off[r + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.n_drafts || (r == 0 && o0 != 0) || (r == a.n_req - 1 && o1 != a.n_drafts)) {
        if (threadIdx.x == 0) atomicOr(a.fault, kFaultDraft);
        return;
    }
    const int n = (int)(o1 - o0);
    int acc = 0;
    for (; acc < n; ++acc) {
        const int d = a.drafts[o0 + acc];
        if (d < 0 || d >= a.vocab) {
            if (threadIdx.x == 0) atomicOr(a.fault, kFaultDraft);
            break;
        }
        const float qd = a.q ? a.q[(o0 + acc) * a.vocab + d] : 1.f;
        if (!(__fmul_rn(a.u_accept[o0 + acc], qd) < a.p[(o0 + r + acc) * a.vocab + d])) break;
    }
    const float *p = a.p + (o0 + r + acc) * a.vocab;
    const float *q = acc < n && a.q ? a.q + (o0 + acc) * a.vocab : nullptr;
    const int sure = acc < n && !a.q ? a.drafts[o0 + acc] : -1;
    bool residual = acc < n;
    auto step = [&](int j) -> unsigned long long {
        float s = p[j];
        if (residual) {
            if (q) s = __fsub_rn(s, q[j]);
            else if (j == sure) s = __fsub_rn(s, 1.f);
        }
        return fixed40(s);
    };
    unsigned long long total = 0;
    for (int tries = 0; tries < 2; ++tries) {
        unsigned long long s = 0;
        for (int j = threadIdx.x; j < a.vocab; j += kThreads) s += step(j);
        total = block_sum(s, red);
        if (total || !residual) break;
        residual = false;
    }
    if (threadIdx.x == 0) a.n_accepted[r] = acc;
    int32_t *out = a.tokens + o0 + r;
    for (int i = threadIdx.x; i <= n; i += kThreads)
        if (i != acc || total == 0) out[i] = i < acc ? a.drafts[o0 + i] : -1;
    if (total == 0) return;
    const float us = a.u_sample[r] * 16777216.f;
    const unsigned long long U = us >= 16777215.f ? 16777215ull : us > 0.f ? (unsigned long long)us : 0ull;
    const unsigned long long goal = (total >> 24) * U + (((total & 0xffffffull) * U) >> 24);
    // the lowest j whose running sum passes the goal: segments of kThreads values in order
    unsigned long long before = 0;
    for (int base = 0; base < a.vocab; base += kThreads) {
        const int j = base + threadIdx.x;
        const unsigned long long v = j < a.vocab ? step(j) : 0ull;
        const unsigned long long all = block_sum(v, red);
        if (before + all > goal) {
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            unsigned long long inc = v;
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned long long w = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += w;
            }
            __syncthreads();
            if (lane == 31) red[warp] = inc;
            __syncthreads();
            unsigned long long b = before;
            for (int w = 0; w < warp; ++w) b += red[w];
            if (b + inc > goal && b + inc - v <= goal) out[acc] = j;
            return;
        }
        before += all;
    }
}

template <class K, class... A>
hq_status launch(K kern, dim3 grid, int threads, cudaStream_t stream, const char *what, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "%s launch: %s", what, cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

}  // namespace

hq_status launch_softmax(const void *logits, const float *temperature, float *p, int64_t n_rows, int64_t vocab,
                         int dtype, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    const dim3 grid((unsigned)n_rows);
    switch (dtype) {
        case HQ_DT_F32: return launch(softmax_kernel<float>, grid, kThreads, stream, "softmax",
                                      (const float *)logits, temperature, p, (long long)vocab);
        case HQ_DT_F16: return launch(softmax_kernel<__half>, grid, kThreads, stream, "softmax",
                                      (const __half *)logits, temperature, p, (long long)vocab);
        default: return launch(softmax_kernel<__nv_bfloat16>, grid, kThreads, stream, "softmax",
                               (const __nv_bfloat16 *)logits, temperature, p, (long long)vocab);
    }
}

hq_status launch_verify(const float *p, const float *q, const int32_t *drafts, const int32_t *off,
                        const float *u_accept, const float *u_sample, int32_t *n_accepted, int32_t *tokens,
                        int64_t n_req, int64_t n_drafts, int64_t vocab, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    VerifyArgs a{p, q, drafts, off, u_accept, u_sample, n_accepted, tokens, (long long)n_req, (long long)n_drafts,
                 (int)vocab, dev->fault};
    return launch(verify_kernel, dim3((unsigned)n_req), kThreads, stream, "verify", a);
}

}  // namespace hq
