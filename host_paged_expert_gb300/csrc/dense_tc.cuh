// PTX wrappers for the dense operators' tensor-core kernels, beyond those of
// tc_sm100.cuh: CTA pairs (cta_group::2), operands whose rows are contiguous
// along M or N, 8-bit operands, clusters.
#pragma once

#include "tc_sm100.cuh"

namespace pe {
namespace tc {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// Without waiting for this thread's memory accesses: where only the meeting
// counts (barriers already made visible by fence_barrier_init, or nobody
// leaves yet).
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Arrive on an mbarrier of any CTA of the cluster after reads of TMEM: what it
// orders are tcgen05 operations, by their fences, so it is relaxed.  (A
// release at cluster scope waits for all of the warp's memory accesses, which
// took a third of the 8-bit kernel's time.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The same after writes to this CTA's shared memory that the barrier's CTA is
// to see done, and a wait that sees them.
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// A warp waits for a barrier phase without sleeping in between, `limit` polls
// at most.  Its lanes poll one address by one instruction, so that they pass or
// give up together (a vote on it, after each wait, took 0.03 us a K block).
__device__ __forceinline__ bool mbar_spin(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    atomicOr(err, (uint32_t)PE_DEVERR_TIMEOUT);
    return false;
}

// The same where another CTA's writes are waited for.
__device__ __forceinline__ bool mbar_spin_cluster(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i)
        if (mbar_try_wait_cluster(bar, parity)) return true;
    atomicOr(err, (uint32_t)PE_DEVERR_TIMEOUT);
    return false;
}

// Polls of a wait before a block ends for what is on its way into it, some
// milliseconds.
constexpr uint32_t kLeavePolls = 1u << 16;
// After a wait gave up: about a millisecond for copies that no barrier here
// tells of.
__device__ __forceinline__ void settle() {
    const long long t0 = clock64();
    for (int i = 0; i < 1 << 16 && clock64() - t0 < 2000000; ++i) __nanosleep(256);
}

// One lane of a converged warp.  The loops that feed the tensor core are run
// by whole warps with warp-uniform values, and only the issue is left to this
// lane: descriptors then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Loads a box into this CTA's shared memory; the bytes count on `bar`, a
// shared::cluster address (of either CTA of the pair).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Stores a box from this CTA's shared memory; what lies past the map's extents
// is left out.  One thread's stores are waited for in groups: until all but N
// of them have been read from shared memory, or all are done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void tma_store_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Waits for this thread's loads from TMEM and hands their registers on: named
// here, no use of them can be moved ahead of the wait (an instruction that the
// compiler does not know to write them).
template <int N, int... M>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N], uint32_t (&... more)[M]) {
    if constexpr (sizeof...(more) > 0) tmem_ld_wait(more...);
    else tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// One MMA over a CTA pair (PAIR) or one CTA; FP8: E4M3 operands, 32 deep,
// else 16-bit operands, 16 deep.
template <bool PAIR, bool FP8>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
#define PE_MMA(G, KIND)                                                                                     \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                           \
                 "tcgen05.mma.cta_group::" G ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),      \
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)                                      \
                 : "memory")
    if (PAIR && FP8) PE_MMA("2", "f8f6f4");
    else if (PAIR) PE_MMA("2", "f16");
    else if (FP8) PE_MMA("1", "f8f6f4");
    else PE_MMA("1", "f16");
#undef PE_MMA
}

// Arrive on `bar` of both CTAs of the pair once the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// The same, on this CTA's `bar` alone.
__device__ __forceinline__ void mma_commit_pair_here(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Shared-memory descriptor of an operand tile written by TMA with 128-byte
// swizzling.
//   K-major: rows of 128 bytes along K, 1024-byte groups of 8 rows.  A step
//   along K inside the row adds its bytes to the address.
//   MN-major: boxes of 64 elements along M or N by 64 along K (8192 bytes,
//   one 128-byte row per k); the leading offset steps to the next box of 64,
//   the stride offset to the next 8 k.  A step of 16 k adds 2048 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool mn) {
    uint64_t d = smem_desc_sw128(saddr);
    if (mn) d = (d & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(8192 >> 4) << 16);
    return d;
}

// Instruction descriptor: fp32 accumulators, A and B of one type.
//   fmt: kind::f16: 0 fp16, 1 bf16; kind::f8f6f4: 0 E4M3.
__host__ __device__ constexpr uint32_t idesc(int fmt, int a_mn, int b_mn, int M, int N) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Two fp32 fused multiply-adds in one instruction: the low and the high half
// of 64-bit registers.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, uint32_t& lo, uint32_t& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <int R>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

}  // namespace tc
}  // namespace pe
