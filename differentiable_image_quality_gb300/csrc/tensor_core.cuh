// Fifth-generation tensor cores (tcgen05) as the attention kernels use them: one
// CTA, 16-bit operands in shared memory or tensor memory, float32 accumulators
// in tensor memory, 128 rows of 128 lanes.
//
// Operand tiles lie in shared memory as the tensor-copy unit writes them with
// 128-byte swizzle: slabs of 64 columns (128 bytes a row), rows one behind the
// other.  Such a slab serves both as an operand whose summed index runs along
// its rows' bytes (K-major) and as one whose summed index counts its rows
// (MN-major); only the descriptor differs.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "dtypes.cuh"

namespace gbssim {
namespace tc {

constexpr int kSlabCols = 64;        // 16-bit columns of a slab
constexpr int kRowBytes = 128;       // of a slab
constexpr int kTileRows = 128;
constexpr int kSlabBytes = kTileRows * kRowBytes;

// ---------------------------------------------------------------- descriptors

// Shared-memory matrix descriptor: start address, the two byte offsets between the
// 8-row groups of the swizzle's pattern, 128-byte swizzle.  Only the low word
// depends on the address, and steps add to it: one thread issues all products, 64
// cycles apart at full rate, so what it spends on each counts (descriptors formed
// anew for each product: half that rate).
struct Desc {
    unsigned lo, hi;
};

__device__ __forceinline__ Desc make_desc(unsigned smem, unsigned leading, unsigned stride)
{
    return {(smem & 0x3ffffu) >> 4 | (leading >> 4) << 16, (stride >> 4) | 1u << 14 | 2u << 29};
}
__device__ __forceinline__ Desc advance(Desc d, unsigned bytes) { return {d.lo + (bytes >> 4), d.hi}; }

// Summed index along the rows' bytes: 8 rows are 1024 bytes.  Step i of 16 elements.
__device__ __forceinline__ Desc desc_k(unsigned slab) { return make_desc(slab, 16, 1024); }
__device__ __forceinline__ constexpr unsigned step_k(int i) { return (i / 4) * kSlabBytes + (i % 4) * 32; }

// Summed index counts the rows: slabs of 64 columns lie kSlabBytes apart.  Step i of 16
// rows.
__device__ __forceinline__ Desc desc_mn(unsigned slab) { return make_desc(slab, kSlabBytes, 1024); }
__device__ __forceinline__ constexpr unsigned step_mn(int i) { return i * 16 * kRowBytes; }

// Instruction descriptor: float32 accumulator, both operands of type T, M = 128 rows,
// n columns; b_mn: the second operand's summed index counts its rows.
template <typename T>
__device__ __forceinline__ unsigned instr_desc(int n, bool b_mn)
{
    constexpr unsigned type = sizeof(T) == 2 && std::is_same<T, bf16>::value ? 1u : 0u;
    return 1u << 4 | type << 7 | type << 10 | (b_mn ? 1u << 16 : 0u) | unsigned(n >> 3) << 17 |
           unsigned(kTileRows >> 4) << 24;
}

// ----------------------------------------------------------------- instructions

// The products are issued by a whole warp that goes one way, with a predicate that one
// lane has (`leader`): the compiler then keeps descriptors in the warp's uniform
// registers, where these instructions want them.  One lane in a branch of its own had
// to move them there for each product and issued one in 75 cycles beside busy warps,
// where the tensor cores take 64.

// 1 in one lane of the warp, 0 in the others.
__device__ __forceinline__ unsigned elect_leader()
{
    unsigned r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r;
}

// D (+)= A B, A and B in shared memory.
__device__ __forceinline__ void mma(unsigned d, Desc a, Desc b, unsigned idesc, bool add, unsigned leader)
{
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n setp.ne.u32 q, %7, 0;\n"
        " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d), "r"(a.lo), "r"(a.hi),
        "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(unsigned(add)), "r"(leader)
        : "memory");
}

// The same with A in tensor memory (two 16-bit elements a column).
__device__ __forceinline__ void mma_ta(unsigned d, unsigned a, Desc b, unsigned idesc, bool add, unsigned leader)
{
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.u32 p, %5, 0;\n setp.ne.u32 q, %6, 0;\n"
        " mov.b64 b, {%2, %3};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d), "r"(a), "r"(b.lo),
        "r"(b.hi), "r"(idesc), "r"(unsigned(add)), "r"(leader)
        : "memory");
}

// D = A B^T of two tiles of 128 rows, their columns summed over in `steps` of 16, at most
// MOST.
template <int MOST>
__device__ __forceinline__ void product_k(unsigned d, Desc a, Desc b, int steps, unsigned idesc, unsigned leader)
{
#pragma unroll
    for (int i = 0; i < MOST; ++i)
        if (i == 0 || i < steps) mma(d, advance(a, step_k(i)), advance(b, step_k(i)), idesc, i > 0, leader);
}

// D (+)= A B: A [128, 64] in tensor memory, B's 64 rows summed over.
__device__ __forceinline__ void product_half(unsigned d, unsigned a, Desc b, unsigned idesc, bool add,
                                             unsigned leader)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) mma_ta(d, a + i * 8, advance(b, step_mn(i)), idesc, i > 0 || add, leader);
}

// D (+)= A B: A [128, 128] in tensor memory, its quarters of 32 columns (16 of tensor
// memory) 32 columns of tensor memory apart, B's 128 rows summed over.
__device__ __forceinline__ void product_parts(unsigned d, unsigned a, Desc b, unsigned idesc, bool add,
                                              unsigned leader)
{
#pragma unroll
    for (int i = 0; i < kTileRows / 16; ++i)
        mma_ta(d, a + (i / 2) * 32 + (i % 2) * 8, advance(b, step_mn(i)), idesc, i > 0 || add, leader);
}

// Arrives on the barrier (by its shared-memory address) when all products issued by the
// leader so far are done.
__device__ __forceinline__ void commit(unsigned bar, unsigned leader)
{
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(leader)
        : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// All 512 columns, by one warp; the address arrives in shared memory.  Waits while
// another block of the SM holds them: that block frees them when it ends.
__device__ __forceinline__ void alloc_all(unsigned *smem_out)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     smem_u32(smem_out))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void free_all(unsigned base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(base) : "memory");
}

// A warp's 32 lanes (its quarter of the 128) of 32 or 16 neighbouring columns: one
// lane a thread.  wait_ld() before the values are used.
__device__ __forceinline__ void ld32(unsigned addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void ld16(unsigned addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void st16(unsigned addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// Writes of this thread to shared memory become visible to the tensor cores and the
// copy unit.
__device__ __forceinline__ void fence_proxy()
{
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

// A warpgroup's registers per thread, given up or taken from what others of the block
// gave up (of those that it was launched with).
template <int N>
__device__ __forceinline__ void release_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// 2^x by the hardware instruction (relative error about 2^-22).
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace tc
}  // namespace gbssim
