// sdm_tensor.cuh -- the fifth-generation tensor core's instructions (tcgen05) as the operators use them: bfloat16 operands in
// shared memory, float32 accumulators in tensor memory, one thread that issues.
//
// Computed operands lie in cores of 8 x 8 elements, 128 contiguous bytes: 8 rows of 16 bytes. A matrix whose rows run along the summed
// dimension (K) has cores of 8 rows x 8 summands; one whose rows run along M or N has cores of 8 summands x 8 columns. A
// descriptor names the first core and the distances between cores along K and along M or N; no swizzle. The same bytes serve
// ldmatrix and stmatrix without bank conflicts, and either reading of a matrix (itself or its transpose) needs no copy. Rows that a
// tensor map brings are swizzled. Measured on a GB300: 128 x N x 16 takes 34 cycles for N of 32, 42 for 64, 65 for 128, 130 for
// 256, whatever the layout and the direction.
#pragma once

#include <cstdint>

namespace sdm {
namespace tensor {

// One thread of a whole warp, always the same. Products and copies that it names in a branch that whole warps take are issued back to
// back (four products: 76 cycles, 265 from a thread chosen by its number).
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
// A matrix operand at shared address `a`: bytes between cores along K and along M or N (the descriptor's leading and stride
// distances; 0b001 in bits 46..48 is its version).
__device__ __forceinline__ uint64_t operand(uint32_t a, uint32_t along_k, uint32_t along_mn) {
    return static_cast<uint64_t>((a & 0x3FFFF) >> 4) | static_cast<uint64_t>((along_k & 0x3FFFF) >> 4) << 16 |
           static_cast<uint64_t>((along_mn & 0x3FFFF) >> 4) << 32 | uint64_t(1) << 46;
}
// The same of rows of 128 bytes whose units of 16 lie swizzled by the row's number in its eight (as a tensor map's boxes of 64
// columns arrive): along M or N in tiles `next` bytes apart where rows run along M or N, eight rows 1024 bytes.
__device__ __forceinline__ uint64_t swizzled(uint32_t a, uint32_t next) { return operand(a, next, 1024) | uint64_t(2) << 61; }
// The instruction's shape: M x N, bfloat16 operands, float32 sums; ta / tb: the operand's rows run along M / N.
__host__ __device__ constexpr uint32_t shape(int M, int N, bool ta, bool tb) {
    return 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(ta) << 15 | static_cast<uint32_t>(tb) << 16 |
           static_cast<uint32_t>(N >> 3) << 17 | static_cast<uint32_t>(M >> 4) << 24;
}
// D (+)= A B over 16 summands: by one thread.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
        "r"(shape), "r"(static_cast<uint32_t>(add)) : "memory");
}
// The barrier gets one arrival when the products issued so far are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Columns of tensor memory: by one whole warp. The address lands in shared memory.
template <int COLS>
__device__ __forceinline__ void allocate(uint32_t at) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(at), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void release(uint32_t d) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(d), "n"(COLS) : "memory");
}
// 32 columns of this warp's 32 rows (rows 32 (warp % 4) ..): lane l holds row l. What fetch32 names is there once arrived has
// named it too.
__device__ __forceinline__ void fetch32(uint32_t d, float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(d));
}
__device__ __forceinline__ void arrived(float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                   "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
    asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                      "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void load32(uint32_t d, float (&v)[32]) {
    fetch32(d, v);
    arrived(v);
}
// 16 columns
__device__ __forceinline__ void fetch16(uint32_t d, float (&v)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(d));
}
__device__ __forceinline__ void arrived(float (&v)[16]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                   "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}
// 32 columns as 16 pairs of neighbours.
__device__ __forceinline__ void load32(uint32_t d, uint64_t (&v)[16]) {
    float x[32];
    load32(d, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "f"(x[2 * i]), "f"(x[2 * i + 1]));
}

__device__ __forceinline__ void barrier_init(uint32_t bar, int arrivals) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(arrivals) : "memory");
}
__device__ __forceinline__ void barrier_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// An arrival that also announces bytes of copies to come.
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Contiguous bytes (a multiple of 16) from global to shared memory; and a box of a tensor map, from a column that is a multiple of 8 on.
__device__ __forceinline__ void copy_bulk(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t to, const void* map, int col, int row, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(to),
                 "l"(map), "r"(col), "r"(row), "r"(bar)
                 : "memory");
}
// Waits for the phase to end, for a second or so at most; false where it has not.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t phase, int tries = 1 << 18) {
    for (int i = 0; i < tries; ++i) {   // a try takes 7800 cycles
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}"
            : "=r"(done) : "r"(bar), "r"(phase) : "memory");
        if (done) return true;
    }
    return false;
}

// After a wait that ran out: waits, a tenth of a second each at most, for what the barriers still expect, before memory is given back.
__device__ __forceinline__ void drain(uint32_t bars, int n) {
    for (int x = 0; x < n; ++x) {
        barrier_wait(bars + 8 * x, 0, 1 << 15);
        barrier_wait(bars + 8 * x, 1, 1 << 15);
    }
}

}  // namespace tensor
}  // namespace sdm
