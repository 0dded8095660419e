// Tensor-core products (tcgen05), tensor memory and the waits of the attention kernels that use them.
#pragma once

#include "attention.cuh"

namespace sv {

constexpr int kTcRows = 128;           // M of the products
constexpr int kTcSpinLimit = 1 << 20;  // polls before a wait gives up

// One item's share of a CTA, as the copying warp tells it to the other roles.
struct Segment {
    int32_t t0, t1;            // tiles [t0, t1); none: the CTA is done
    int32_t sink_tiles, first_tile, low, high, sink;   // as in Item
    int32_t len, r0, rows, head;
    int32_t whole, slot;       // the whole item, or the slot of its part
    int64_t row0;              // the block's first packed row
    __device__ __forceinline__ int start(int t) const { return (t < sink_tiles ? t : first_tile + t - sink_tiles) * kTile; }
};
constexpr int kSegments = 4;   // told ahead
__device__ __forceinline__ Segment segment_of(const AttnParams& p, const Walk& w, int cta) {
    return {w.t0, w.t1, w.it.sink_tiles, w.it.first_tile, w.it.low, w.it.high, w.it.sink, w.len, w.it.r0, w.it.r1 - w.it.r0, w.h,
            w.whole(), w.slot(cta), first_row(p.a.cu_drafts, w.b, p.a.kmax)};
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One look at the phase, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase; false when the wait (or another one of the CTA) gave up.  The whole warp decides: a loop that each lane
// leaves for itself costs twice as much when the phase is already there (heads of 64: 61 us against 57 for 64 streams).
__device__ __forceinline__ bool warp_wait_for(uint64_t* bar, unsigned parity, int* abort) {
    for (int n = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++n) {
        if ((n & 15) == 0) {
            if (n > kTcSpinLimit) *reinterpret_cast<volatile int*>(abort) = 1;
            if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(abort) != 0)) return false;
        }
    }
    return true;
}

// Shared-memory matrix descriptors, 128-byte swizzle, strides in units of 16 bytes.  K-major (Q, K): 8 rows of 128
// bytes are an atom of 1,024 bytes, the next 8 rows begin `group` further on.  MN-major (V, whose rows are the
// product's K): the same atoms, and `panel` from one 64-column panel to the next.  The low word holds the
// address, so that stepping through an operand is one 32-bit addition.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t panel) { return (addr & 0x3ffff) >> 4 | panel << 16; }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t group) {
    const uint32_t hi = group | 1u << 14 | 2u << 29;
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
// kind::f16: float32 accumulator, bf16 operands, M = 128; `mn` = the B operand is MN-major
constexpr uint32_t mma_desc(int n, bool mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kTcRows >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define SV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define SV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SV_W8(r, 0),
        SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24), "r"(addr)
        : "memory");
}
// ... eight, four columns
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::SV_W8(r, 0), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(a), "r"(b), "r"(c), "r"(d), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t addr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
#undef SV_R8
#undef SV_W8

// Registers of a warpgroup, all of whose warps ask together; what all ask for is at most what the CTA was launched with.
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 bytes in one store
__device__ __forceinline__ void store32(void* to, const uint32_t* x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ bool all_test(uint64_t* bar, unsigned parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)); }
__device__ __forceinline__ bool elected() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
// A warp of products gave up: what it issued has to end before the CTA's memory is given back.
__device__ __forceinline__ void drain(uint64_t* bar) {
    if (elected()) mma_commit(bar);
    __syncwarp();
    for (int n = 0; n < kTcSpinLimit / 64 && !all_test(bar, 0); ++n) {}
}

}  // namespace sv
