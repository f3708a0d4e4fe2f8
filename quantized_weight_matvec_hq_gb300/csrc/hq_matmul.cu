// hq_matmul.cu -- products of many tokens with quantized weights: grouped by
// expert, or shared with an adapter per request.
#include <cuda_bf16.h>

#include "hq_device.cuh"
#include "hq_internal.h"

namespace hq {
namespace {

__device__ __forceinline__ float load_elem(const void *x, long long i, int dtype) {
    if (dtype == HQ_DT_F32) return static_cast<const float *>(x)[i];
    if (dtype == HQ_DT_F16) return __half2float(static_cast<const __half *>(x)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
}

__device__ __forceinline__ void store_elem(void *y, long long i, int dtype, float v) {
    if (dtype == HQ_DT_F32) static_cast<float *>(y)[i] = v;
    else if (dtype == HQ_DT_F16) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

struct KArgs {
    MatmulArgs a;
    uint32_t *fault;
};

// sum_j w[row][j] x[xi][j]: one warp, a block of 32 columns at a time
__device__ float dot(const MatmulArgs &a, long long row, long long xi) {
    const int lane = threadIdx.x & 31;
    const int bytes = a.fmt == 8 ? 34 : 18;
    const uint8_t *w = static_cast<const uint8_t *>(a.W) + row * (a.cols / 32) * bytes;
    float s = 0.f;
    for (long long b = 0; b < a.cols / 32; ++b, w += bytes) {
        const float d = __half2float(*reinterpret_cast<const __half *>(w));
        const int q = a.fmt == 8 ? (int)reinterpret_cast<const int8_t *>(w)[2 + lane]
                                 : (int)((w[2 + (lane & 15)] >> (lane & 16 ? 4 : 0)) & 15) - 8;
        s = fmaf(d * (float)q, load_elem(a.x, xi * a.cols + 32 * b + lane, a.dtype), s);
    }
    return warp_sum(s);
}

// The plain form: one warp per output.
__global__ void __launch_bounds__(256) matmul_plain_kernel(KArgs k) {
    const MatmulArgs &a = k.a;
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long out_rows = a.epilogue == HQ_MOE_EPI_SWIGLU ? a.rows / 2 : a.rows;
    const long long slots = a.n_tokens * (a.epilogue == HQ_MOE_EPI_COMBINE ? 1 : a.n_active);
    for (long long o = blockIdx.x * 8ll + (threadIdx.x >> 5); o < out_rows * slots; o += gridDim.x * 8ll) {
        const long long slot = o / out_rows, i = o % out_rows;
        float y = 0.f;
        if (a.moe) {
            const int n = a.epilogue == HQ_MOE_EPI_COMBINE ? a.n_active : 1;
            for (int j = 0; j < n; ++j) {
                const long long s = slot * n + j;
                const int e = a.idx[s];
                float v;
                if (e < 0 || e >= a.n_mats) {
                    atomicOr(k.fault, kFaultExpertId);
                    v = __int_as_float(0x7fc00000);
                } else {
                    const long long xi = a.x_per_slot ? s : s / a.n_active;
                    if (a.epilogue == HQ_MOE_EPI_SWIGLU) {
                        const float g = dot(a, e * a.rows + 2 * i, xi), u = dot(a, e * a.rows + 2 * i + 1, xi);
                        v = g / (1.f + expf(-g)) * u;
                    } else {
                        v = dot(a, e * a.rows + i, xi);
                    }
                }
                y = a.epilogue == HQ_MOE_EPI_COMBINE ? fmaf(a.router_w[s], v, y) : v;
            }
        } else {
            y = dot(a, i, slot);
            const int ad = a.n_adapters ? a.idx[slot] : -1;
            if (ad < -1 || ad >= a.n_adapters) {
                atomicOr(k.fault, kFaultAdapterId);
                y = __int_as_float(0x7fc00000);
            } else if (ad >= 0) {
                float t = 0.f;
                for (int r = 0; r < a.rank; ++r) {
                    float u = 0.f;
                    for (long long j = lane; j < a.cols; j += 32)
                        u = fmaf(__uint_as_float((uint32_t)a.A[(ad * (long long)a.rank + r) * a.cols + j] << 16),
                                 load_elem(a.x, slot * a.cols + j, a.dtype), u);
                    u = warp_sum(u);
                    t = fmaf(__uint_as_float((uint32_t)a.B[(ad * a.rows + i) * a.rank + r] << 16), u, t);
                }
                y = fmaf(a.scales[ad], t, y);
            }
        }
        if (lane == 0) store_elem(a.y, o, a.dtype, y);
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

}  // namespace

int64_t matmul_workspace(const MatmulArgs &) { return 0; }

hq_status launch_matmul(const MatmulArgs &a, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    KArgs k{a, dev->fault};
    matmul_plain_kernel<<<(unsigned)(dev->num_sms * 8), 256, 0, stream>>>(k);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "matmul launch: %s", cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

hq_status launch_weight_exponents(int fmt, const void *W, int32_t *w_exp, int64_t n_mats, int64_t rows, int64_t cols,
                                  cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    weight_exponents_kernel<<<(unsigned)n_mats, 1024, 0, stream>>>(fmt == HQ_FMT_Q8_0 ? 34 : 18, (const uint8_t *)W,
                                                                   w_exp, rows * (cols / 32));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "exponents launch: %s", cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

}  // namespace hq
