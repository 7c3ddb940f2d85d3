// What the kernels around tcgen05.mma share: bounded waits of whole warps, the
// matrix descriptor of 8-bit operands, commits, meetings of a cluster, and
// accumulator reads.
#pragma once

#include "cluster.cuh"
#include "common.cuh"

namespace mr {

// Set when a bounded wait of this translation unit's kernels ran out (read by
// the host).
static __device__ int g_ex_timeout;

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The whole warp waits for the phase of this parity, at most limit_ns; a wait
// that runs out sets the device's flag and *abort, which ends every other
// wait of the CTA.
static __device__ __noinline__ bool ex_wait_slow(uint32_t bar, unsigned parity, unsigned long long limit_ns,
                                          volatile int* abort) {
    const unsigned long long t0 = global_ns();
    for (int i = 1;; ++i) {
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        if ((i & 15) != 0) continue;
        const bool late = global_ns() - t0 >= limit_ns;
        if (__any_sync(kFull, late)) {
            *abort = 1;
            atomicExch(&g_ex_timeout, 1);
        }
        if (__any_sync(kFull, *abort != 0)) return false;
    }
}
__device__ __forceinline__ bool ex_wait(uint32_t bar, unsigned parity, unsigned long long limit_ns,
                                        volatile int* abort) {
    return __all_sync(kFull, mbar_try_wait(bar, parity)) || ex_wait_slow(bar, parity, limit_ns, abort);
}
// The same where nothing of another CTA's memory is used after the wait (the
// arrivals are this CTA's copies, or products and accumulator reads, whose
// order tcgen05's own fences keep): acquired at the scope of the CTA.  No call:
// the caller may hold more registers than a call leaves.
__device__ __forceinline__ bool mbar_test_cta(uint32_t bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool ex_wait_cta(uint32_t bar, unsigned parity, unsigned long long limit_ns,
                                            volatile int* abort) {
    auto done = [&] { return __all_sync(kFull, mbar_test_cta(bar, parity)); };
    if (done()) return true;
    const unsigned long long t0 = global_ns();
    for (int i = 1;; ++i) {
        if (done()) return true;
        if ((i & 15) != 0) continue;
        if (__any_sync(kFull, global_ns() - t0 >= limit_ns)) {
            *abort = 1;
            atomicExch(&g_ex_timeout, 1);
        }
        if (__any_sync(kFull, *abort != 0)) return false;
    }
}
// The phase's state now, as a lane sees it, without waiting for it.  (Nothing that
// the phase publishes may be read before the answer has been looked at.)
__device__ __forceinline__ bool mbar_peek_cta(uint32_t bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool ex_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Shared-memory matrix descriptors without their address field (address >> 4
// in the low 14 bits).  Codes: K-major rows of 128 bytes in the 128-byte
// swizzle (8-row groups 1024 bytes apart); a k-step starts 32 bytes further.
constexpr unsigned long long kExDescCodes =
    (1ull << 16) | ((unsigned long long)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
__device__ __forceinline__ unsigned long long ex_desc(unsigned long long kind, uint32_t addr) {
    return kind | (unsigned long long)((addr >> 4) & 0x3FFFu);
}
// An arrival (PAIR: in both CTAs, at the same place) when the products issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void ex_commit(uint32_t bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"((unsigned short)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
// All threads of the cluster meet.  _meet: called from branches that a warp's
// lanes may have left at different times.
__device__ __forceinline__ void ex_cluster_meet() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void ex_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 accumulator columns of this warp's 32 lanes: the read is under way until
// ex_ld_wait; ex_ld_tie keeps later uses of a read's registers behind it.
__device__ __forceinline__ void ex_ld16_async(uint32_t (&v)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void ex_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void ex_ld_tie(uint32_t (&v)[16]) {
    asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}
__device__ __forceinline__ void ex_ld16(uint32_t (&v)[16], uint32_t addr) {
    ex_ld16_async(v, addr);
    ex_ld_wait();
    ex_ld_tie(v);
}
// Barrier id of threads threads (whole warps); true when ok holds in all of them.
__device__ __forceinline__ bool ex_sync(int id, int threads, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
        "barrier.cta.red.and.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// What one lane of a warp issues (lead: 1 in that lane, 0 in the others) is
// predicated in the instruction: in a branch of one lane the operands, which
// these instructions take from uniform registers, are moved there one by one
// (50 cycles a product).
__device__ __forceinline__ void ex_expect(uint32_t lead, uint32_t bar, unsigned bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void ex_load_2d(uint32_t lead, uint32_t dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
            "r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(bar), "r"(lead)
        : "memory");
}

// The same tile into L2 alone, by the calling lane.  Nothing is read by the kernel: it may
// come before the wait for the kernel launched before, whatever that one writes.
__device__ __forceinline__ void ex_prefetch_2d(const void* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<unsigned long long>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

}  // namespace mr
