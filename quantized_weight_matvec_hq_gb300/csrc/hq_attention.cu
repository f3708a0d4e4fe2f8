// hq_attention.cu -- attention of a batch's tokens over the quantized key/value
// cache.
//
// The plain kernel: a warp takes one query row and goes through the positions it sees one after another, its lanes the elements
// of the head (lane e has element e of every block of 32), with the running maximum and sum of the softmax.
#include <type_traits>

#include "hq_cache.cuh"

namespace hq {
namespace {

constexpr int kThreads = 256;

struct AttnArgs {
    CacheView c;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    int n_heads, causal;
    float scale;
    long long window;
};

template <class T, int BITS, int D>
__global__ void __launch_bounds__(kThreads) attention_plain_kernel(AttnArgs a) {
    using L = CellLayout<BITS, D>;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < a.c.n_req; r += kThreads)
            if (request_of(a.c, r).bad) atomicOr(a.c.fault, kFaultCache);
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long t = row / a.n_heads;
    const int h = (int)(row % a.n_heads), kvh = h / (a.n_heads / a.c.n_kv_heads);
    if (t >= a.c.n_tokens) return;
    int r = -1;
    for (int i = 0; i < a.c.n_req; ++i)
        if (a.c.offsets[i] <= t && t < a.c.offsets[i + 1]) r = i;
    if (r < 0) return;
    const Request rq = request_of(a.c, r);
    if (rq.n == 0) return;
    const int at = rq.length - rq.n + (int)(t - rq.first);
    const int hi = a.causal ? at + 1 : rq.length;
    const int lo = a.window > 0 && a.window <= at ? at + 1 - (int)a.window : 0;
    constexpr int NB = L::NB;
    float q[NB], o[NB], m = -INFINITY, s = 0.f;
    const T *qp = static_cast<const T *>(a.q) + t * a.q_stride + (long long)h * D;
#pragma unroll
    for (int b = 0; b < NB; ++b) { q[b] = (float)qp[32 * b + lane] * a.scale; o[b] = 0.f; }
    const int kc = lane / 8, ki = lane % 8, vj = lane / 8, vg = lane % 8;
    const uint8_t *cells = nullptr;
    for (int p = lo; p < hi; ++p) {
        if (p == lo || (p & ((1 << a.c.page_shift) - 1)) == 0) cells = page_cells(a.c, r, p, kvh);
        const uint8_t *cell = cells ? cell_of<L>(a.c, const_cast<uint8_t *>(cells), p) : nullptr;
        const int pos = p & (kCell - 1);
        float k[NB], v[NB], z = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (!cell) { k[b] = v[b] = __uint_as_float(0x7fffffffu); }
            else {
                uint32_t kq, vq;
                if (BITS == 8) {
                    kq = cell[L::k_word(pos, kc, 2 * b + ki / 4) + ki % 4] ;
                    vq = cell[L::v_word(pos / 2, vg, 2 * b + vj / 2) + 2 * (pos & 1) + vj % 2];
                } else {
                    kq = (cell[L::k_word(pos, kc, b) + (ki & 1) * 2 + ki / 4] >> (4 * (ki / 2 % 2))) & 15u;
                    vq = (cell[L::v_word(pos / 2, vg, b) + 2 * (pos & 1) + vj / 2] >> (4 * (vj % 2))) & 15u;
                }
                constexpr float kMid = BITS == 8 ? 128.f : 8.f;
                k[b] = ((float)kq - kMid) * __half2float(*reinterpret_cast<const __half *>(cell + L::k_scale(pos, b)));
                v[b] = ((float)vq - kMid) * __half2float(*reinterpret_cast<const __half *>(cell + L::v_scale(pos, b)));
            }
            z += q[b] * k[b];
        }
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        const float m1 = fmaxf(m, z), f = m == -INFINITY ? 0.f : expf(m - m1), w = expf(z - m1);
        s = s * f + w;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[b] = o[b] * f + w * v[b];
        m = m1;
    }
    T *out = static_cast<T *>(a.out) + t * a.out_stride + (long long)h * D;
#pragma unroll
    for (int b = 0; b < NB; ++b) out[32 * b + lane] = to_elem<T>(hi > lo ? __fdiv_rn(o[b], s) : 0.f);
}

template <class T, int BITS, int D>
hq_status launch(const AttnArgs &a, cudaStream_t stream) {
    const long long rows = a.c.n_tokens * a.n_heads;
    attention_plain_kernel<T, BITS, D><<<(unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(HQ_ERR_LAUNCH, "attention launch: %s", cudaGetErrorString(e));
    note_launch();
    return HQ_OK;
}

template <class T, int BITS>
hq_status launch_dim(int dim, const AttnArgs &a, cudaStream_t stream) {
    if (dim == 64) return launch<T, BITS, 64>(a, stream);
    if (dim == 128) return launch<T, BITS, 128>(a, stream);
    return launch<T, BITS, 256>(a, stream);
}

template <class T>
hq_status launch_bits(const AttentionArgs &x, const AttnArgs &a, cudaStream_t stream) {
    return x.cache.fmt == HQ_FMT_Q8_0 ? launch_dim<T, 8>(x.cache.head_dim, a, stream) : launch_dim<T, 4>(x.cache.head_dim, a, stream);
}

}  // namespace

int64_t attention_workspace(const AttentionArgs &) { return 0; }

hq_status launch_attention(const AttentionArgs &x, cudaStream_t stream) {
    DeviceInfo *dev = nullptr;
    hq_status st = device_info(&dev);
    if (st != HQ_OK) return st;
    AttnArgs a = {cache_view(x.cache, dev->fault), x.q, x.out, x.q_stride, x.out_stride, x.n_heads, x.causal, x.scale, x.window};
    switch (x.cache.dtype) {
        case HQ_DT_F32: return launch_bits<float>(x, a, stream);
        case HQ_DT_F16: return launch_bits<__half>(x, a, stream);
        default: return launch_bits<__nv_bfloat16>(x, a, stream);
    }
}

}  // namespace hq
