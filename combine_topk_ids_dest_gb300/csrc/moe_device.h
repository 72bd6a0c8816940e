// moe_device.h -- device helpers of the MoE operators: mbarriers with bounded
// waits, TMA copies, tcgen05 matrix instructions and tensor-memory access.
//
// Every wait has a limit (kWaitCycles of the SM's clock, about 2 s; the
// nanosecond timer takes longer to read than most waits last). A wait that
// runs out sets the block's abort flag; every other wait of the block sees the
// flag and gives up too, the roles leave their loops and the block ends
// through its normal exit, which drains its copies and frees its tensor memory.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace moe {

constexpr long long kWaitCycles = 4000000000LL;

static __device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// True in one lane of a converged warp, the same one each time. The compiler
// knows what elect.sync does: tcgen05 and TMA instructions under it are issued
// with uniform registers at 36 to 55 cycles an MMA, against 190 under a test
// of the lane's number.
static __device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// Programmatic dependent launch: lets the next kernel of the stream start as
// SMs come free; and waits for the kernel before this one to be complete and
// its writes to be visible. Both do nothing without the launch attribute.
static __device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
static __device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- mbarriers ----------------------------------------------------------------

static __device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

static __device__ __forceinline__ void mbar_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

static __device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

static __device__ __forceinline__ void mbar_arrive(uint32_t bar, uint32_t count = 1)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

static __device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Which wait gave up first in a block (the abort flag's value).
enum WaitSite { kWaitEmptyA = 1, kWaitEmptyB, kWaitEmptyD, kWaitFullA, kWaitFullB, kWaitFullD, kWaitDone, kWaitOther };

static __device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    const long long t0 = clock64();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try(bar, parity))
                return true;
        if (abort && *abort)
            return false;
        if (clock64() - t0 > kWaitCycles) {
            if (abort)
                *abort = site;
            return false;
        }
    }
}

// True once the barrier's phase of this parity has completed; false when the
// wait ran out or the block is aborting. abort may be NULL (only the limit).
static __device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    if (mbar_try(bar, parity))
        return true;
    return mbar_wait_slow(bar, parity, abort, site);
}

// mbar_wait by a whole converged warp, with one answer for all lanes (which
// lets the compiler keep what follows in uniform registers).
static __device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    return __all_sync(~0u, mbar_wait(bar, parity, abort, site));
}

// Whether the phases of both of two barriers have completed; this lane's view.
static __device__ __forceinline__ uint32_t mbar_peek2(uint32_t bar1, uint32_t parity1, uint32_t bar2, uint32_t parity2)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
                 "and.pred p, p, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar1), "r"(parity1), "r"(bar2), "r"(parity2)
                 : "memory");
    return ok;
}

// Waits for both of two barriers, by a whole converged warp. ready: what
// mbar_peek2 said of them at some time before, whose answer is at hand by now:
// then it is one vote and one branch (a branch costs some 25 cycles, a test
// that has to be waited for some 100).
static __device__ __forceinline__ bool mbar_wait2_warp(uint32_t ready, uint32_t bar1, uint32_t parity1, uint32_t bar2,
                                                       uint32_t parity2, volatile int *abort, int site1, int site2)
{
    if (__all_sync(~0u, ready))
        return true;
    return __all_sync(~0u, mbar_wait(bar1, parity1, abort, site1) && mbar_wait(bar2, parity2, abort, site2));
}

// mbar_arrive on two barriers where `me` is true, without a branch.
static __device__ __forceinline__ void mbar_arrive2_if(bool me, uint32_t bar1, uint32_t bar2)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
                 "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t"
                 "@p mbarrier.arrive.shared::cta.b64 _, [%2];\n\t}" ::"r"(uint32_t(me)),
                 "r"(bar1), "r"(bar2)
                 : "memory");
}

// ---- TMA ------------------------------------------------------------------------

static __device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

static __device__ __forceinline__ uint64_t policy_evict_first()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

static __device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(m), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

// Into this block's memory; bar may be the other block's of a pair.
static __device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(m), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

static __device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

static __device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y,
                                                   int z, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
                 "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
                 : "memory");
}

// Four rows r0..r3 of a two-dimensional map (box one row high), to 4 consecutive tile rows.
static __device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int r0,
                                                   int r1, int r2, int r3)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(m), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// Untiled copy: addresses 16-byte aligned, bytes a multiple of 16.
static __device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                                 uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar), "l"(policy)
                 : "memory");
}

// Orders this thread's ordinary accesses with TMA accesses to the same memory.
static __device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ---- tcgen05 --------------------------------------------------------------------

// PAIR: for matrix instructions of two neighbouring blocks (cta_group::2); both
// blocks call it, and all tcgen05 instructions of a kernel are of one kind.
template <bool PAIR = false> static __device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols)
{
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <bool PAIR = false> static __device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

static __device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
static __device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on the barrier when every earlier tcgen05.mma of this thread has completed.
static __device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The same for the instructions of a pair, on the barrier at this offset of both blocks.
static __device__ __forceinline__ void tc_commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}

static __device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The address of this offset in the cluster's first block.
static __device__ __forceinline__ uint32_t in_first_block(uint32_t at)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(at));
    return r;
}

// Instruction descriptor of kind::f16: fp32 accumulators, A and B both bf16
// (bf16 != 0) or both fp16, both K-major.
static __host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int bf16)
{
    return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

// Shared-memory descriptor of a K-major tile in 128-byte rows, 128-byte
// swizzle, 8-row blocks 1024 bytes apart. addr: of the tile's row 0 (1024-byte
// aligned) plus the byte offset along K.
static __device__ __forceinline__ uint64_t desc_sw128(uint32_t addr)
{
    return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t(1) << 16) | (uint64_t(64) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}

// D[tmem] (+)= A[smem] B[smem]^T
static __device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
                 : "memory");
}

// The same by a pair of blocks, issued in the first: 256 rows of A, 128 in each block's memory, and half of B's rows
// in each (at the same offsets); a block's tensor memory gets the sums of its rows with all of B.
static __device__ __forceinline__ void mma_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
                 : "memory");
}

// 8 consecutive columns of this warp's 32 lanes (lane = row).
static __device__ __forceinline__ void tmem_ld8(uint32_t addr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

static __device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- warp-level MMA -------------------------------------------------------------

// c[16 x 8] = (ADD ? c : 0) + a[16 x 16] b[16 x 8], bf16 or fp16 fragments
template <bool BF16, bool ADD>
static __device__ __forceinline__ void mma_16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    const float z = 0.0f;
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %11, %12, %13};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(ADD ? c[0] : z),
                       "f"(ADD ? c[1] : z), "f"(ADD ? c[2] : z), "f"(ADD ? c[3] : z));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%10, %11, %12, %13};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(ADD ? c[0] : z),
                       "f"(ADD ? c[1] : z), "f"(ADD ? c[2] : z), "f"(ADD ? c[3] : z));
}

// ---- global flags -----------------------------------------------------------------

static __device__ __forceinline__ int ld_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Adds n with release/acquire order and returns the old value. After a block
// barrier it publishes what every thread of the barrier wrote.
static __device__ __forceinline__ int add_acq_rel(int *p, int n)
{
    int v;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(v) : "l"(p), "r"(n) : "memory");
    return v;
}

// Waits until *p has reached `target`.
static __device__ __forceinline__ bool wait_count(const int *p, int target, volatile int *abort, int site)
{
    if (ld_acquire(p) >= target)
        return true;
    const long long t0 = clock64();
    while (ld_acquire(p) < target) {
        if (*abort)
            return false;
        if (clock64() - t0 > kWaitCycles) {
            *abort = site;
            return false;
        }
    }
    return true;
}

static __device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// True in all `threads` threads of the barrier if `v` is true in all of them.
static __device__ __forceinline__ bool named_all(int id, int threads, bool v)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "bar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"(uint32_t(v))
                 : "memory");
    return r != 0;
}

}  // namespace moe
