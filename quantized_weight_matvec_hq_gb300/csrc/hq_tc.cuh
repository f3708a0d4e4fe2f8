// hq_tc.cuh -- sm_103a tensor-core primitives: tcgen05 allocation, products
// with one operand in TMEM and one in shared memory, TMEM loads and stores.
// Inline PTX only.
#pragma once

#include "hq_device.cuh"

namespace hq {

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Bounded wait on phase `parity` of an mbarrier, small in code: the thread sleeps in hardware for up to 20 us a
// try, and gives up after limit_cycles SM cycles, or as soon as another wait of the block has.
// `abort` is the block's; the fault word gets the time-out.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *fault,
                                        uint32_t limit_cycles = (uint32_t)kWaitTimeoutCycles) {
    uint32_t t0 = 0;                                        // (the clock is not read by a wait that the first sleep ends)
#pragma unroll 1
    while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
        if (*abort) return false;
        const uint32_t now = (uint32_t)clock();             // its low 32 bits: the limit is below 2^32, and a sleep far shorter
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_cycles) {
            note_timeout(fault, (blockIdx.x & 0x7fffffu) << 9);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// The same on a path that counts every cycle, unless `known`: the thread goes on after a time-out as well (`*abort` is then
// set, no later wait of the block takes longer than its question, and the caller looks at the end of an item).
// A result that the caller tests costs more than the question: of two waits that are
// over, in one thread of a warp, 460 cycles with it and 200 without.  Its limit is a number of sleeps, each of which
// takes 32.8 us if nothing ends it (65536 cycles at 2 GHz; measured over 1 to 1000 of them): with a clock in the loop the
// f32 products took 141 us for 133 (131 tokens).
__device__ __forceinline__ void tc_wait_go(bool known, uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *fault,
                                           uint32_t limit_sleeps = (uint32_t)(kWaitTimeoutCycles >> 16)) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 a, n;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "@p bra D%=;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra D%=;\n\t"
        "mov.u32 n, %7;\n"
        "W%=:\n\t"
        "ld.volatile.shared.u32 a, [%3];\n\t"
        "setp.ne.u32 p, a, 0;\n\t"
        "@p bra D%=;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "@p bra D%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 p, n, 0;\n\t"
        "@p bra W%=;\n\t"
        "st.volatile.shared.u32 [%3], 1;\n\t"
        "atom.global.cas.b32 a, [%4], 0, %5;\n\t"
        "setp.ne.u32 p, a, 0;\n\t"
        "@p red.global.or.b32 [%4], %6;\n"
        "D%=:\n\t}"
        ::"r"((uint32_t)known), "r"(bar), "r"(parity), "r"(smem_u32(const_cast<int *>(abort))), "l"(fault),
          "r"(((blockIdx.x & 0x7fffffu) << 9) | kFaultWaitTimeout), "r"(kFaultWaitTimeout), "r"(limit_sleeps) : "memory");
}

// Whether phase `parity` of an mbarrier is complete.
__device__ __forceinline__ bool tc_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// D[128][N] (+)= A[128][16] B[N][16]^T: 16-bit floats, A in TMEM (8 columns of pairs), B in shared memory, fp32 in TMEM.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// Arrives on `bar` once every product this thread has issued so far is done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory descriptor of a K-major tile of 128-byte rows (64 16-bit
// elements) in the 128-byte swizzle: rows of 8 repeat every 1024 bytes.
__device__ __forceinline__ uint64_t tc_desc_sw128(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// fp32 sums of f16 (or bf16) products, both operands K-major, M = 128.
__device__ __forceinline__ uint32_t tc_idesc(int n, bool bf16) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// This warp's 32 lanes x 8 columns.  The values may be used only after
// tmem_wait_ld() has taken them.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 ::"r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                   "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                   "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(addr) : "memory");
}

// Waits for this warp's loads.  The loaded values pass through the statement,
// so that no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(float (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                 :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                   "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(addr) : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// 3-D tiled tensor load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy) : "memory");
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

}  // namespace hq
