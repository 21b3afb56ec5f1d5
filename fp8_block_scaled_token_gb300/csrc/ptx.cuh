// ptx.cuh -- hand-written PTX wrappers for sm_103a: mbarrier, TMA tensor
// loads, tcgen05 (tensor memory allocation, MMA, commit, loads), programmatic
// dependent launch, and the bounded waits every pipeline stage uses.
//
// Written from the public PTX ISA descriptions of each instruction.  Nothing
// here multicasts: every CTA fetches its own tiles.
#pragma once

#include <cstdint>
#include <cuda.h>

namespace fp8bs {

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// Make barrier initialisation visible to the async proxy (TMA, tensor core).
__device__ __forceinline__ void fence_mbar_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Order this thread's generic-proxy shared-memory writes before later
// async-proxy accesses (TMA, tcgen05.mma operand reads).
__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Stores a box of a 2-D tensor from shared memory (completion tracked by this
// thread's bulk async-groups); elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *smem_src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit_group()
{
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Every bulk group this thread committed has finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Every bulk group this thread committed has completed (writes included).
__device__ __forceinline__ void bulk_wait_all()
{
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// d0 = fma(a0, b0, d0), d1 = fma(a1, b1, d1) as one packed instruction
// (fma.rn.f32x2: each lane one fp32 fused multiply-add, round to nearest,
// the same result as two fmaf).
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%0, %1};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rc;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// d0 += a0, d1 += a1 as one packed instruction (add.rn.f32x2, the same
// result as two fp32 additions).
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1)
{
    asm("{\n\t.reg .b64 ra, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rc, {%0, %1};\n\t"
        "add.rn.f32x2 rc, rc, ra;\n\t"
        "mov.b64 {%0, %1}, rc;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// d0 = a0 * b, d1 = a1 * b as one packed instruction (mul.rn.f32x2, the same
// result as two fp32 multiplications).
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b)
{
    asm("{\n\t.reg .b64 ra, rb;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %4};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\t"
        "mov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b));
}

// Orders this thread's view of global memory (generic proxy) before its later
// bulk copies from global memory (async proxy).
__device__ __forceinline__ void fence_proxy_async_global()
{
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// True once the phase with parity `parity` has completed.  While the phase
// is open the thread may be suspended for up to 2 us (it wakes when the phase
// completes): spinning waiters would otherwise take issue slots from the
// warps doing the work, including those of the other CTA sharing the SM
// (measured on GB300: vocab layer 208.5 -> 198.2 us, MLP down 22.5 -> 22.0 us).
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same without suspending: whether the phase has completed by now.
__device__ __forceinline__ bool mbar_peek(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// commit of every MMA so far, by the lane whose `lead` is set
__device__ __forceinline__ void mma_commit_by(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// Device-side failure codes written to the status word.
enum : uint32_t {
    kErrTimeoutProducer = 1u << 0,
    kErrTimeoutMma = 1u << 1,
    kErrTimeoutEpilogue = 1u << 2,
    kErrTimeoutQuant = 1u << 3,
    kErrTimeoutDrain = 1u << 4,
    kErrBounds = 1u << 5, // FP8BS_DEBUG builds: an index or coordinate left its buffer
};

// Device-side bounds checks of the FP8BS_DEBUG build (the stand-in for a
// memory checker): a failed check records kErrBounds in the status word,
// raises the CTA's abort flag and returns false, and the caller skips the
// access.  Nothing traps.  In the normal build every check is the constant
// true and compiles away.
#ifdef FP8BS_DEBUG
__device__ __forceinline__ bool debug_check(bool ok, unsigned *status, volatile int *abort_flag)
{
    if (!ok) {
        *abort_flag = 1;
        atomicOr(status, static_cast<unsigned>(kErrBounds));
    }
    return ok;
}
#define FP8BS_CHECK(cond) ::fp8bs::debug_check((cond), p.status, abort_flag)
#else
#define FP8BS_CHECK(cond) true
#endif

// Bounded wait.  Returns false when the wait gave up: either another role of
// this CTA already raised `abort_flag`, or `timeout_ns` elapsed (then this
// call raises the flag and records `code` in the global status word).
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                          unsigned *status, uint32_t code, uint64_t timeout_ns)
{
    if (mbar_test(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_test(bar, parity))
            return true;
        if ((i & 63u) == 0u) {
            if (*abort_flag)
                return false;
            if (globaltimer_ns() - t0 > timeout_ns) {
                *abort_flag = 1;
                atomicOr(status, code);
                return false;
            }
        }
    }
}

// The same with the polling out of line, for loops whose instructions have to
// stay close together: warps of different roles share what a scheduler has
// fetched.
static __device__ __noinline__ bool mbar_wait_poll(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned *status,
                                            uint32_t code, uint64_t timeout_ns)
{
    return mbar_wait(bar, parity, abort_flag, status, code, timeout_ns);
}
__device__ __forceinline__ bool mbar_wait_far(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                              unsigned *status, uint32_t code, uint64_t timeout_ns)
{
    return mbar_test(bar, parity) || mbar_wait_poll(bar, parity, abort_flag, status, code, timeout_ns);
}

// --------------------------------------------------------------------- TMA
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_first()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

__device__ __forceinline__ uint64_t l2_policy_evict_last()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// 2-D tiled bulk tensor load global -> this CTA's shared memory; completion
// is counted in bytes on `bar`.  x is the innermost (contiguous) coordinate.
__device__ __forceinline__ void tma_load_2d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// 1-D bulk copy global -> this CTA's shared memory, completion counted in
// bytes on `bar`.  Both addresses 16-byte aligned, `bytes` a multiple of 16.
__device__ __forceinline__ void bulk_load_1d(void *smem_dst, const void *gsrc, uint32_t bytes, uint64_t *bar,
                                             uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(smem_dst)),
                 "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
                 : "memory");
}

// Fetch the 128-byte line holding `p` into this SM's L1 (no result).
__device__ __forceinline__ void prefetch_l1(const void *p)
{
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// ------------------------------------------------------- global atomics
// Device-scope add with acquire-release semantics: releases every write
// that happens-before it (including other threads' writes ordered by a
// preceding CTA barrier) and acquires the writes released by earlier adds.
__device__ __forceinline__ unsigned atomic_add_acq_rel_gpu(unsigned *p, unsigned v)
{
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// Publishes a word with everything that happens-before it, and the read that
// takes both up.
__device__ __forceinline__ void store_release_gpu(unsigned *p, unsigned v)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned load_acquire_gpu(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// ----------------------------------------------- programmatic dependent launch
__device__ __forceinline__ void grid_dependency_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// --------------------------------------------------------------- tcgen05
// Allocate `ncols` (power of two, >= 32) tensor-memory columns; the address
// is written to shared memory.  Whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t *smem_result, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(smem_result)),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_fence_before_sync()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after_sync()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, one CTA.  kind::f8f6f4 (E4M3 operands).
__device__ __forceinline__ void mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Same, kind::f16 (both operands bf16 here).
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on `bar` when every tcgen05 operation this thread issued so
// far has completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// 16 consecutive 32-bit columns of this warp's 32 TMEM lanes (lane i of the
// warp reads TMEM lane base+i), followed by the wait for their arrival.  One
// asm statement so no use of the registers can be scheduled before the wait.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 32 consecutive columns, same contract as tmem_load16 (one wait for all).
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// The load of tmem_load16 / tmem_load32 without its wait, and the wait on its
// own: a caller may promote one chunk while the next is in flight.  The wait
// names the destination registers as read and written, so no use of them can
// be scheduled before it, and none may come between the two.
__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Store 32 consecutive columns of this warp's 32 TMEM lanes and wait until
// they are written.
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 64 consecutive columns, same contract as tmem_load16 (one wait for all).
__device__ __forceinline__ void tmem_load64(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// Shared-memory matrix descriptor for a K-major operand stored in the
// 128-byte swizzle layout that a TMA load with SWIZZLE_128B produces: rows of
// 128 bytes, 8-row (1024-byte) swizzle atoms stacked contiguously.
//   bits  0-13 start address >> 4
//   bits 16-29 leading-dimension byte offset >> 4 (not used by swizzled
//              K-major layouts; set to 1)
//   bits 32-45 stride-dimension byte offset >> 4 (1024 B between 8-row groups)
//   bits 46-47 descriptor version (1 for tcgen05)
//   bits 49-51 base offset (0: atoms are 1024-byte aligned)
//   bits 61-63 swizzle mode (2 = 128-byte swizzle)
// Advancing along K inside the 128-byte row adds (bytes >> 4) to the start
// address; the hardware applies the swizzle to the final address.
__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// The same in two words: the upper one is the same for every tile.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) { return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16); }

// Instruction descriptor (kind::f16 / kind::f8f6f4 layout):
//   bits 4-5  D format (1 = fp32)
//   bits 7-9  A format, bits 10-12 B format (f8f6f4: 0 = E4M3; f16: 1 = BF16)
//   bit 15/16 A/B major (0 = K-major)
//   bits 17-22 N >> 3, bits 24-28 M >> 4
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int m, int n)
{
    return (1u << 4) | (0u << 7) | (0u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__host__ __device__ constexpr uint32_t idesc_bf16_f32(int m, int n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// ------------------------------------------ block-scaled (MX) tensor-core path
// Scale factors of the MX MMA live in tensor memory.  They are staged in
// shared memory as 512-byte atoms covering 128 rows (weight rows, or tokens)
// x 4 consecutive 32-wide K blocks: the byte of row r and K block j sits at
//     16 * (r % 32) + 4 * (r / 32) + j,
// i.e. 32 lines of 16 bytes, line r%32 holding rows r%32, +32, +64, +96.
// tcgen05.cp .32x128b.warpx4 copies the 32 lines into 32 lanes x 4 columns
// of every one of the four 32-lane sub-partitions, so the sub-partition that
// computes rows 32q..32q+31 finds row 32q + i's four bytes in its lane i,
// column q; byte j of that column is K block j, picked per MMA by the scale
// factor id of the instruction descriptor.

// Descriptor of one such atom: no swizzle, 16-byte lines, 8-line core
// matrices 128 bytes apart (same bit layout as sw128_kmajor_desc).
__device__ __forceinline__ uint64_t sf_atom_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128u >> 4) << 16; // leading byte offset (one core matrix wide: unused)
    d |= static_cast<uint64_t>(128u >> 4) << 32; // stride byte offset between 8-line core matrices
    d |= static_cast<uint64_t>(1u) << 46;        // tcgen05 descriptor version
    return d;                                   // bits 61-63 = 0: no swizzle
}

// Copy one scale-factor atom (smem) to tensor memory columns taddr..+3 of
// all 128 lanes (see above).  Asynchronous; ordered before later tcgen05.mma
// of the same thread, and tracked by tcgen05.commit like them.
__device__ __forceinline__ void tmem_cp_sf_atom(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// D[tmem] (+)= (A . sfA) * (B . sfB)^T with E4M3 operands and one UE8M0
// scale per 32 K per row (kind::mxf8f6f4, scale vector 1X).
__device__ __forceinline__ void mma_mxf8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

// Instruction descriptor of the block-scaled kinds:
//   bits 4-5  scale factor id of B (byte of the 32-bit column), bits 7-9 /
//   10-12 A / B format (0 = E4M3), bits 15/16 A/B major (0 = K-major),
//   bits 17-22 N >> 3, bit 23 scale format (1 = UE8M0), bits 27-28 M >> 7,
//   bits 29-30 scale factor id of A.  D is fp32.
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int m, int n, uint32_t a_sf_id, uint32_t b_sf_id)
{
    return (b_sf_id << 4) | (0u << 7) | (0u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 7) << 27) | (a_sf_id << 29);
}

// ------------------------------------------------------- 4-bit operands
// E2M1 operands, two to a byte (the lower K in the lower four bits): a
// 128-byte K-major row holds 256 values, four MMAs of 64.  The scale factors
// use the atoms above, read four blocks of K to an atom:
//   scale_vec::4X (one UE4M3 factor per 16 K): an atom covers 64 K, one MMA;
//     its four bytes per row are the MMA's four factors (scale factor id 0);
//   scale_vec::2X (one UE8M0 factor per 32 K): an atom covers 128 K, two
//     MMAs, which take the byte pairs 0-1 and 2-3 (scale factor ids 0, 2).
//
// One unit's four MMAs and the commit of its stage, by the lane whose `lead` is
// set, as one predicated sequence: the whole warp runs it, so there is no
// divergent branch and every operand stays in uniform registers.  a_lo, b_lo:
// desc_lo of the stage's tiles; accumulate: whether the first MMA adds to D.
#define FP8BS_FP4_MMA(kind, sfa, sfb, idesc, pred)                                                                     \
    "@e tcgen05.mma.cta_group::1.kind::" kind " [%0], a, b, " idesc ", [" sfa "], [" sfb "], " pred ";\n\t"
#define FP8BS_FP4_NEXT_K                                                                                               \
    "add.u32 al, al, 2;\n\tadd.u32 bl, bl, 2;\n\tmov.b64 a, {al, %3};\n\tmov.b64 b, {bl, %3};\n\t"
#define FP8BS_FP4_BEGIN                                                                                                \
    "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 al, bl, fa, fb;\n\t"                                   \
    "setp.ne.b32 e, %7, 0;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"                                    \
    "mov.b32 al, %1;\n\tmov.b32 bl, %2;\n\tmov.b32 fa, %4;\n\tmov.b32 fb, %5;\n\t"                                \
    "mov.b64 a, {al, %3};\n\tmov.b64 b, {bl, %3};\n\t"
#define FP8BS_FP4_NEXT_SF "add.u32 fa, fa, 4;\n\tadd.u32 fb, fb, 4;\n\t"
#define FP8BS_FP4_END "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%8];\n\t}"

__device__ __forceinline__ void mma_nvf4_unit(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                              uint32_t accumulate, uint32_t stage_free)
{
    asm volatile(FP8BS_FP4_BEGIN
                 FP8BS_FP4_MMA("mxf4nvf4.block_scale.scale_vec::4X", "fa", "fb", "%9", "p") FP8BS_FP4_NEXT_K FP8BS_FP4_NEXT_SF
                 FP8BS_FP4_MMA("mxf4nvf4.block_scale.scale_vec::4X", "fa", "fb", "%9", "t") FP8BS_FP4_NEXT_K FP8BS_FP4_NEXT_SF
                 FP8BS_FP4_MMA("mxf4nvf4.block_scale.scale_vec::4X", "fa", "fb", "%9", "t") FP8BS_FP4_NEXT_K FP8BS_FP4_NEXT_SF
                 FP8BS_FP4_MMA("mxf4nvf4.block_scale.scale_vec::4X", "fa", "fb", "%9", "t") FP8BS_FP4_END ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(lead),
                 "r"(stage_free), "r"(idesc)
                 : "memory");
}

// idesc, idesc2: scale factor ids 0 and 2 (bytes 0-1 and 2-3 of the atoms' columns).
__device__ __forceinline__ void mma_mxf4_unit(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t idesc, uint32_t idesc2, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                              uint32_t accumulate, uint32_t stage_free)
{
    asm volatile(FP8BS_FP4_BEGIN
                 FP8BS_FP4_MMA("mxf4.block_scale.scale_vec::2X", "fa", "fb", "%9", "p") FP8BS_FP4_NEXT_K
                 FP8BS_FP4_MMA("mxf4.block_scale.scale_vec::2X", "fa", "fb", "%10", "t") FP8BS_FP4_NEXT_K FP8BS_FP4_NEXT_SF
                 FP8BS_FP4_MMA("mxf4.block_scale.scale_vec::2X", "fa", "fb", "%9", "t") FP8BS_FP4_NEXT_K
                 FP8BS_FP4_MMA("mxf4.block_scale.scale_vec::2X", "fa", "fb", "%10", "t") FP8BS_FP4_END ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate), "r"(lead),
                 "r"(stage_free), "r"(idesc), "r"(idesc2)
                 : "memory");
}
#undef FP8BS_FP4_MMA
#undef FP8BS_FP4_NEXT_K
#undef FP8BS_FP4_BEGIN
#undef FP8BS_FP4_NEXT_SF
#undef FP8BS_FP4_END

// Instruction descriptor of kind::mxf4 / kind::mxf4nvf4: as idesc_mx_e4m3,
// with A and B format 1 (E2M1), scale format 0 = UE4M3, 1 = UE8M0, and bit 31
// = 0 (64 K per dense MMA).
__host__ __device__ constexpr uint32_t idesc_fp4(int m, int n, uint32_t ue8m0, uint32_t sf_id)
{
    return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (ue8m0 << 23) |
           (static_cast<uint32_t>(m >> 7) << 27) | (sf_id << 29);
}

// Named barrier over `nthreads` threads (ids 1..15; 0 is __syncthreads).
__device__ __forceinline__ void named_bar_sync(uint32_t id, uint32_t nthreads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}


} // namespace fp8bs
