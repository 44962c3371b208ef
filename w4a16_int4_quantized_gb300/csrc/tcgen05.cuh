// tcgen05.cuh -- wrappers of the 5th-generation tensor-core instructions
// (sm_103a): TMEM allocation and access, shared-memory and instruction
// descriptors, the MMA kinds in use, and the bounded wait of a pipeline role.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace w4 {

W4_DEV void tmem_alloc(uint32_t *dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
W4_DEV void tmem_dealloc(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
W4_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
W4_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, K-major operand, 128-byte swizzle:
// 8-row atoms of 1024 bytes (stride byte offset 1024), start address >> 4.
W4_DEV uint64_t smem_desc_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;             // leading byte offset (unused for swizzled K-major)
    d |= (uint64_t)(1024 >> 4) << 32;   // stride byte offset: next 8-row atom
    d |= (uint64_t)1 << 46;             // descriptor version
    d |= (uint64_t)2 << 61;             // 128-byte swizzle
    return d;
}

// Operand whose M or N axis is contiguous (16-bit values, 128-byte swizzle):
// atoms of 64 values by 8 steps of K, 1024 bytes; along K the next atom follows
// at once, along M or N it is `next` bytes on.
W4_DEV uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t next) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(next >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Unswizzled rows of 16 bytes, 8 to a core matrix of 128 bytes (scale factors for tcgen05.cp).
W4_DEV uint64_t smem_desc_rows16(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(128 >> 4) << 16;
    d |= (uint64_t)(128 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

// Instruction descriptor of kind::f16: f32 accumulator, A/B f16 (0) or bf16 (1),
// both K-major, N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t ab_fmt, uint32_t M, uint32_t N) {
    return (1u << 4) | (ab_fmt << 7) | (ab_fmt << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// kind::mxf4, both operands e2m1 (1) with e8m0 scales (bit 23): sf_id is the
// first of the two scale bytes (0 or 2 of a 32-bit column) that A and B use.
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N, uint32_t sf_id) {
    return (sf_id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24) | (sf_id << 29);
}

W4_DEV void umma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The calls with `lead` are made by a whole converged warp, with the same
// arguments but for lead, which is 1 in one lane: that lane issues.  The
// operands are then uniform to the compiler and stay in uniform registers; in
// a branch of one lane each has to be moved there first (the tree attention with
// two row tiles: 368 us so, 283 by whole warps; the 4-bit GEMM 40.8 and 37.3).
W4_DEV uint32_t elect_lead() {
    uint32_t lead;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(lead));
    return lead;
}

W4_DEV void umma_f16_lead(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                          uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

// The same with A in TMEM (two 16-bit values to a column).
W4_DEV void umma_f16_ts_lead(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                             uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(tmem_d), "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

// 64 columns of 4-bit operands, a scale for 32: A, B descriptors, scales in TMEM.
W4_DEV void umma_mxf4_lead(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t tmem_sfa,
                           uint32_t tmem_sfb, uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(tmem_sfa), "r"(tmem_sfb), "r"(accumulate), "r"(lead)
        : "memory");
}

// 32 rows of 16 bytes from shared memory into 4 TMEM columns of all four lane quadrants.
W4_DEV void tmem_cp_sf_lead(uint32_t taddr, uint64_t sdesc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}"
        ::"r"(taddr), "l"(sdesc), "r"(lead)
        : "memory");
}

W4_DEV void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

W4_DEV void umma_commit_lead(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(lead)
        : "memory");
}

// A descriptor whose operand starts `bytes` further on (the address field does not overflow: 18 bits).
W4_DEV uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

#define W4_R8(v, i)                                                                                               \
    "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]),    \
        "=r"(v[i + 7])

// Reads and writes of TMEM are the whole warp's; lanes that went different ways before one
// (rows without a token, masks) come together in it.
// 32 consecutive columns of the warp's 32 TMEM lanes, complete on return.
W4_DEV void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : W4_R8(v, 0), W4_R8(v, 8), W4_R8(v, 16), W4_R8(v, 24)
        : "r"(taddr)
        : "memory");
}

// 64 columns.
W4_DEV void tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : W4_R8(v, 0), W4_R8(v, 8), W4_R8(v, 16), W4_R8(v, 24), W4_R8(v, 32), W4_R8(v, 40), W4_R8(v, 48), W4_R8(v, 56)
        : "r"(taddr)
        : "memory");
}
#undef W4_R8

// 32 consecutive columns of the warp's 32 TMEM lanes, written on return.
W4_DEV void tmem_st32(uint32_t taddr, const uint32_t *v) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n\t"
        "tcgen05.wait::st.sync.aligned;"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),
        "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),
        "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
        : "memory");
}

// The part of a wait that found its barrier not ready: tries on (each try
// suspends the thread for a while in hardware) until the phase completes,
// another role of the CTA aborts, or about a second has gone.  Out of line: the
// many waits of a pipeline keep their code, and their ready case, short.
static __device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, int *abort, uint32_t *status) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int *>(abort)) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, kStatusPipeTimeout);
            *reinterpret_cast<volatile int *>(abort) = 1;
            return false;
        }
    }
}

// Bounded wait that also ends as soon as another role of the CTA has aborted.
W4_DEV bool wait_or_abort(uint64_t *bar, uint32_t parity, int *abort, uint32_t *status) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, status);
}

// The same for a converged warp: true in all its lanes, or false in all.
W4_DEV bool wait_warp(uint64_t *bar, uint32_t parity, int *abort, uint32_t *status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_slow(bar, parity, abort, status)) != 0;
}

// After an abort: the copies and products that the CTA began and nobody waits for any more
// are through (or an eighth of a second has gone for each) before it gives up its shared
// memory and TMEM.
constexpr uint64_t kDrainLimitNs = kWaitLimitNs / 8;

// Fills of stage s after `begun` fills of a ring in order.
W4_HD constexpr int ring_fills(int s, int stages, int begun) { return (begun + stages - 1 - s) / stages; }
static_assert(ring_fills(0, 4, 0) == 0 && ring_fills(3, 4, 0) == 0 && ring_fills(0, 4, 1) == 1 &&
                  ring_fills(1, 4, 1) == 0 && ring_fills(3, 4, 8) == 2 && ring_fills(0, 4, 9) == 3 &&
                  ring_fills(1, 4, 9) == 2 && ring_fills(0, 1, 5) == 5,
              "a stage is filled once a round, in order");

// By one lane.  Out of line, as wait_slow is.
static __device__ __noinline__ void drain_ring(uint64_t *full, int stages, int begun) {
#pragma unroll 1
    for (int s = 0; s < stages; ++s) {
        const int n = ring_fills(s, stages, begun);
        if (n > 0) mbar_wait_bounded(&full[s], (uint32_t)(n - 1) & 1u, kDrainLimitNs);
    }
}

// By the converged warp that issued the products (the lane that issued them is elected again).
static __device__ __noinline__ void drain_products(uint64_t *bar) {
    umma_commit_lead(bar, elect_lead());
    mbar_wait_bounded(bar, 0, kDrainLimitNs);
}

}  // namespace w4
