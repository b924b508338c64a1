// sdm_operators.cuh -- what the kernels of the operators around the memory share (sdm_glr.cu, sdm_rope.cu, sdm_logprob.cu, sdm_gdr.cu,
// sdm_gdr_bwd.cu, sdm_norm.cu, sdm_embed.cu): their launches, plain loads, pairs of float32 and the parts of a cluster. The memory's own kernels include none of it, so
// that captured figures of theirs stay tied to their sources alone.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <initializer_list>
#include <utility>

#include "sdm_checks.cuh"
#include "sdm_internal.cuh"
#include "sdm_rows.cuh"

namespace sdm {

// The first instruction of a kernel that is launched as a programmatic dependent: waits for the kernel before. It does not
// let the kernel behind start while it runs: the waiting blocks cost more than the launch they hide (8 x 131072 token
// log probabilities 10.2 us with, 7.9 without; a short rotation 14.6 and 13.7; long kernels equal).
__device__ __forceinline__ void start_dependent() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch of clusters of `cluster` blocks (a multiple of them) with `smem` bytes of dynamic shared memory, as a programmatic
// dependent.
template <typename... Params, typename... Args>
cudaError_t launch_cluster_smem(void (*kernel)(Params...), dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t stream,
                                Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... Params, typename... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, int cluster, cudaStream_t stream,
                           Args&&... args) {
    return launch_cluster_smem(kernel, grid, block, cluster, 0, stream, std::forward<Args>(args)...);
}

namespace checks {

// Whether every pointer (NULL among them) lies on a multiple of n bytes.
inline bool aligned_all(unsigned n, std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) % n != 0) return false;
    return true;
}

}  // namespace checks

namespace rows {

// A lane's 4 columns through plain loads: the kernels may start before the kernel before has written what they read, and
// start_dependent makes those writes visible to plain loads, while the read-only path (Raw4::ld) asks for data that nothing
// writes while the kernel runs.
__device__ __forceinline__ void ld_plain(Raw4<float>& r, const float* p) { r.v = *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void ld_plain(Raw4<__nv_bfloat16>& r, const __nv_bfloat16* p) { r.v = *reinterpret_cast<const uint2*>(p); }

// One element: float32 as it is, bfloat16 rounded to nearest even.
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two float32 in one 64-bit register pair: one instruction multiplies, adds or multiply-adds both (each rounded as the
// scalar instruction rounds it).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t o;
    asm("mov.b64 %0, {%1, %2};" : "=l"(o) : "f"(a), "f"(b));
    return o;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t o;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(o) : "l"(a), "l"(b), "l"(c));
    return o;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t o;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(a), "l"(b));
    return o;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t o;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(a), "l"(b));
    return o;
}

// Four columns as two pairs of float32.
struct Quad {
    uint64_t lo, hi;
};
__device__ __forceinline__ Quad quad(const float (&v)[4]) { return {pack2(v[0], v[1]), pack2(v[2], v[3])}; }
__device__ __forceinline__ Quad quad(float v) { return {pack2(v, v), pack2(v, v)}; }
__device__ __forceinline__ void floats(const Quad& q, float (&v)[4]) {
    unpack2(q.lo, v[0], v[1]);
    unpack2(q.hi, v[2], v[3]);
}
__device__ __forceinline__ Quad fma4(const Quad& a, const Quad& b, const Quad& c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ Quad mul4(const Quad& a, const Quad& b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Quad add4(const Quad& a, const Quad& b) { return {add2(a.lo, b.lo), add2(a.hi, b.hi)}; }
template <typename T>
__device__ __forceinline__ Quad quad(const Raw4<T>& r) {
    float v[4];
    r.get(v);
    return quad(v);
}
__device__ __forceinline__ Raw4<float> load4(const float* p) {
    Raw4<float> r;
    ld_plain(r, p);
    return r;
}
__device__ __forceinline__ Quad quad_at(const float* p) {   // 16 bytes of shared memory
    float v[4];
    get4(p, v);
    return quad(v);
}
template <typename T>
__device__ __forceinline__ void st4(T* p, const Quad& q) {
    float v[4];
    floats(q, v);
    st4(p, v);
}

// The blocks of a cluster: this one's rank, the barrier in its two halves (release / acquire of every thread's accesses;
// relaxed: the arrival alone), and the address of another block's copy of a shared variable.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t remote_address(const void* p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
    return a;
}

}  // namespace rows
}  // namespace sdm
