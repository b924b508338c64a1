// sdm_gdr.cuh -- what the kernels of the gated delta rule share (sdm_gdr.cu, sdm_gdr_bwd.cu): their arguments, how rows are cut
// into blocks of 64, tiles of bfloat16 in shared memory, and the tensor cores' fragments.
//
// Mathematics. With gam the running sum of g over a block's rows, D_ij = e^(gam_i - gam_j), G = D o K K^T strictly below the
// diagonal, A = D o Q K^T up to it, and T = (I + diag(beta) G)^-1, a block that starts from the state S gives
//   R = V - e^gam o K S,   U = T (beta o R),   y = scale (e^gam o Q S + A U),   S' = e^gam_last S + K^T (e^(gam_last - gam) o U),
// which is the rule row by row with the rows' writes u_t = beta_t (v_t - e^g_t S_{t-1}^T k_t) solved for together.
//
// Numbers. The tensor cores multiply bfloat16 and add in float32. A float32 operand is a sum of bfloat16 terms, its value
// rounded, the rest rounded, and so on: two terms hold 16 bits of mantissa and a bit (2^-17 off at most), three hold all 24.
// Of two such operands' product the terms (i, j) with i + j below the number of terms are taken. bfloat16 rows are exact
// operands of one term, and what is computed from them has two: states, writes and the solution of the triangular system
// keep 17 bits through a product and 24 where they are added (measured: states 4e-6 off 64 bits after 4096 rows, where the rows'
// answers are rounded to 2e-3; a third term would bring 3e-7 for 1.4 times the products). float32 rows are cut into three
// terms once, ahead of everything, and so are what is computed from them; their products are added a step of 16 summands at a time
// (measured: all outputs 1.0e-7 to 2.5e-7 off 64 bits, 7e-7 to 4e-6 with one run of additions in the tensor core, for 1.16 times the time).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"
#include "sdm_tensor.cuh"

namespace sdm {
namespace gdr {

using namespace rows;

constexpr int kC = SDM_GDR_CHUNK;   // rows of a block
constexpr int kMaxD = 128;          // channels of a head at most
constexpr int kVecs = 5;
constexpr int kTerms = 3;           // of float32 rows, and of what is computed from them

// A write strength below 2^-80 counts as 2^-80, so that the error v - e^g S^T k behind a write, which the strength's gradient
// takes, can be had from the write. What a row of strength 0 writes is then 2^-80 of that error, which no other value feels.
__device__ __forceinline__ float strength(float beta) { return fabsf(beta) < 0x1p-80f ? copysignf(0x1p-80f, beta) : beta; }

// Rows as the tensor cores take them: planes of bfloat16 (one, or the three terms of float32 rows).
struct Planes {
    const __nv_bfloat16* p;
    int64_t ld;      // elements between rows
    int64_t plane;   // elements between planes
};

struct Args {
    Planes q, k, v, dy;
    const void* g;
    const void* beta;
    const int64_t* offsets;   // nullable: equal lengths
    const float* h0;          // nullable
    const float* dhT;         // nullable
    float* hT;                // nullable
    float* dh0;               // nullable
    __nv_bfloat16* states;    // nullable in the forward: [blocks][Hv] (float32 rows: [dv / 16] tiles)
    __nv_bfloat16* writes;    // behind the states: U, [blocks][Hv]
    void* y;
    void* dq;
    void* dk_out;
    void* dv_out;
    void* dg;
    void* dbeta;
    __nv_bfloat16* tri;       // behind the writes, or workspace: [blocks][Hv]: of bfloat16 rows two terms of [T; scale A T], [128][64] in cores of 8 rows; of
                              // float32 rows six planes [64][64], T's terms and A's
    float* vec;               // as `tri`: [blocks][Hv][kVecs][64]: e^gam, beta, e^(gam_last - gam), gam as a sum of two floats
    __nv_bfloat16* dstates;   // workspace of the backward: the gradients of the states behind the blocks, as `states`
    __nv_bfloat16* du;        // workspace of the backward: the gradients of the writes (dv before beta), as `writes`
    float* part;              // workspace of the backward: gradients of shared queries and keys
    uint32_t* status;         // nullable
    int64_t rows, len;        // len: rows of every sequence where offsets is null
    int64_t g_ld, b_ld, y_ld, dq_ld, dk_ld, dv_ld, dg_ld, db_ld;
    int P, Hk, Hv, dk, dv, g_bf16;
    float scale;
};

// Tensor maps of bfloat16 rows [rows][heads x d] for boxes of 64 rows x 64 columns.
struct Maps {
    CUtensorMap k, q, v;   // v: V of the walk, dY from the end
    int boxes;             // whether they serve: heads of 64 or 128 columns, rows apart from one another
};

// Segments of every sequence that are walked side by side (columns of bfloat16 rows' states): n of them, and what they need.
struct Segments {
    int n;
    float* start;   // [P][Hv][n][dk][dv]: the states before them (n = 1: h0, nullable)
    float* move;    // [P][Hv][n - 1][dk][dk]: what they make of a state that they start from, beside what they write
    int32_t* ends;  // [P][Hv]: segments that start from a state of finite values; the last of them walks on to the sequence's end
};

// The rows [b, b + n) of sequence p. Offsets that are not ascending within [0, rows] are cut to it and reported.
__device__ __forceinline__ void sequence(const Args& a, int p, int64_t& b, int64_t& n) {
    if (a.offsets == nullptr) {
        b = p * a.len;
        n = a.len;
        return;
    }
    const int64_t lo = a.offsets[p], hi = a.offsets[p + 1];
    b = min(max(lo, int64_t(0)), a.rows);
    n = max(min(hi, a.rows) - b, int64_t(0));
    if ((lo < 0 || hi > a.rows || lo > hi) && a.status != nullptr && threadIdx.x == 0) atomicOr(a.status, SDM_DEV_BAD_OFFSET);
}

// Sequence p's blocks have the numbers from b / 64 + p on; numbers between two sequences' name nothing.
__device__ __forceinline__ int64_t first_block(int64_t b, int p) { return b / kC + p; }

// The rows [b, b + n) of block number `id`, n <= 0 where it names nothing. Warp-wide.
__device__ __forceinline__ void block_rows(const Args& a, int64_t id, int64_t& b, int& n) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.P;   // the last sequence whose first number is at most id is in [lo, hi): 32 probes a round
    if (a.offsets == nullptr) {
        // len / 64 + 1 numbers a sequence or one less: b / 64 + p with b = p len
        while (hi - lo > 1) {
            const int w = (hi - lo + 31) / 32, q = lo + (lane + 1) * w;
            const bool le = q < hi && first_block(q * a.len, q) <= id;
            const int c = __popc(__ballot_sync(kFull, le));
            lo += c * w;
            hi = min(hi, lo + w);
        }
    } else {
        while (hi - lo > 1) {
            const int w = (hi - lo + 31) / 32, q = lo + (lane + 1) * w;
            const bool le = q < hi && first_block(min(max(a.offsets[q], int64_t(0)), a.rows), q) <= id;
            const int c = __popc(__ballot_sync(kFull, le));
            lo += c * w;
            hi = min(hi, lo + w);
        }
    }
    int64_t b0, len;
    sequence(a, lo, b0, len);
    const int64_t j = id - first_block(b0, lo);
    b = b0 + j * kC;
    n = j < 0 ? 0 : static_cast<int>(min(len - j * kC, int64_t(kC)));
}

// The sequence that a launch's rank-th one walks: the longest first where their number allows a look by one warp. Warp-wide.
__device__ __forceinline__ int by_length(const Args& a, int rank) {
    if (a.offsets == nullptr || a.P > 32 || a.P == 1) return rank;
    const int lane = threadIdx.x & 31;
    const int64_t mine = lane < a.P ? a.offsets[lane + 1] - a.offsets[lane] : -1;
    int before = 0;
    for (int q = 0; q < a.P; ++q) {
        const int64_t other = __shfl_sync(kFull, mine, q);
        before += other > mine || (other == mine && q < lane);
    }
    return __ffs(__ballot_sync(kFull, before == rank && lane < a.P)) - 1;
}

__device__ __forceinline__ float gate_at(const void* p, int64_t i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// e^x of a difference of decays' sums. Beside bfloat16 rows by the hardware's exponential: 2 + 1.2 |x| units of 2^-23, and what e^x
// loses in digits it has lost in size.
template <int XT>
__device__ __forceinline__ float decay(float x) {
    return XT == 1 ? __expf(x) : expf(x);
}

// ---- tiles in shared memory: rows of W bfloat16 in units of 16 bytes, which the row's number permutes so that eight rows'
// units of one column lie in different banks ------------------------------------------------------------
template <int W>
__device__ __forceinline__ uint32_t tile_at(int r, int u) {
    constexpr int U = W / 8;
    static_assert(U == 2 || U == 4 || U % 8 == 0, "tile width");
    const int s = U >= 8 ? (r & 7) : U == 4 ? ((r >> 1) & 3) : ((r >> 2) & 1);
    return static_cast<uint32_t>(r * (W * 2) + ((u ^ s) << 4));
}
__device__ __forceinline__ uint32_t smem_of(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {   // zeros where it is not
    const int n = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile of 64 rows x W columns of `planes` planes from rows [b, b + n) and columns [c0, c0 + cols) of x; the rest zeros.
template <int W, int THREADS>
__device__ __forceinline__ void load_rows(uint32_t dst, const Planes& x, int planes, int64_t b, int n, int c0, int cols, int tid) {
    constexpr int U = W / 8;
    for (int pl = 0; pl < planes; ++pl) {
        const __nv_bfloat16* const src = x.p + pl * x.plane + b * x.ld + c0;
#pragma unroll
        for (int i = tid; i < kC * U; i += THREADS) {
            const int r = i / U, u = i % U;
            const bool there = r < n && u * 8 < cols;
            copy16(dst + pl * (kC * W * 2) + tile_at<W>(r, u), there ? src + r * x.ld + u * 8 : x.p, there);
        }
    }
}
// A 64 x 64 plane's blocks of 16 up to the diagonal, as the workspace holds them
template <int THREADS>
__device__ __forceinline__ void load_tri(uint32_t dst, const __nv_bfloat16* src, int tid) {
#pragma unroll
    for (int i = tid; i < kC * 8; i += THREADS) {
        const int r = i >> 3, u = i & 7;
        if (u <= (r >> 4) * 2 + 1) copy16(dst + tile_at<kC>(r, u), src + r * kC + u * 8, true);
    }
}

// Rows as boxes bring them: 128 bytes, a unit of 16 swizzled by the row
__device__ __forceinline__ uint32_t swizzled_at(int r, int u) { return static_cast<uint32_t>(r * 128 + ((u ^ (r & 7)) << 4)); }
// [T; scale A T]: units of 8 columns, of each 128 rows of 16 bytes
__device__ __forceinline__ uint32_t stacked_at(int r, int u) { return static_cast<uint32_t>(u * 2048 + (r >> 3) * 128 + (r & 7) * 16); }

// ---- fragments ------------------------------------------------------------------------------------------
// (loads of fragments keep their place among barriers and stores by being volatile; the products are free to move)
__device__ __forceinline__ void ldsm4(uint32_t (&f)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&f)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(a));
}
__device__ __forceinline__ void stsm4(uint32_t a, const uint32_t (&f)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(f[0]), "r"(f[1]), "r"(f[2]),
                 "r"(f[3]) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, const uint32_t (&f)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(f[0]), "r"(f[1]),
                 "r"(f[2]), "r"(f[3]) : "memory");
}
__device__ __forceinline__ void st_word(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t transposed(uint32_t f) {
    uint32_t o;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(f));
    return o;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two float32 as bfloat16 (the first in the low half), and as a sum of N such (an infinity's rests are NaN)
__device__ __forceinline__ uint32_t round2(float x, float y) {
    uint32_t o;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(y), "f"(x));
    return o;
}
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = round2(x, y);
        if (i + 1 < N) {
            x -= __uint_as_float(t[i] << 16);
            y -= __uint_as_float(t[i] & 0xFFFF0000u);
        }
    }
}
// The places that a lane's address of ldsm4 / ldsm4t names in a tile, for fragments
//   B of n x k from a tile [n][k] (not transposed): n 0..15, k 0..15 -> {b0, b1} of n 0..7, {b0, b1} of n 8..15
//   B from a tile [k][n] (transposed): the same order
//   A of m x k from a tile [m][k] (not transposed), and from a tile [k][m] (transposed)
struct Lane {
    int rB, uB;     // B, not transposed: row, unit
    int rBt, uBt;   // B, transposed
    int rA, uA;     // A, not transposed
    int rAt, uAt;   // A, transposed (also an accumulator's own transpose)
    __device__ __forceinline__ explicit Lane(int lane) {
        const int m = lane >> 3, r = lane & 7;
        rB = (m >> 1) * 8 + r; uB = m & 1;
        rBt = (m & 1) * 8 + r; uBt = m >> 1;
        rA = (m & 1) * 8 + r; uA = m >> 1;
        rAt = (m >> 1) * 8 + r; uAt = m & 1;
    }
};
// An operand A of 16 columns k from the accumulators of two neighbouring tiles of 8, in N terms
template <int N>
__device__ __forceinline__ void terms_of(const float (&c0)[4], const float (&c1)[4], uint32_t (&f)[N][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float(&c)[4] = i < 2 ? c0 : c1;
        uint32_t t[N];
        split2<N>(c[2 * (i & 1)], c[2 * (i & 1) + 1], t);
#pragma unroll
        for (int n = 0; n < N; ++n) f[n][i] = t[n];
    }
}
// What a step of 16 summands adds to a sum. The tensor core cuts off what lies below the last place at every addition: of three terms a
// step's products are added by themselves, the small ones first, and then to the sum with a rounding.
template <int N, typename F>
__device__ __forceinline__ void add_step(float (&acc)[4], F f) {
    if constexpr (N == 3) {
        float t[4] = {};
        f(t);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += t[e];
    } else {
        f(acc);
    }
}
// acc += A B for an operand A of NA terms and tiles of 16 columns of B, np0 .. np1 - 1, of NB planes (`plane` bytes apart), whose
// fragments `at(np)` names; terms (i, j) with i + j < N. The same accumulator comes round after the others.
template <int NA, int NB, int N, bool TRANS, int NP, typename At, int M>
__device__ __forceinline__ void products(float (&acc)[M][4], const uint32_t (&a)[NA][4], int plane, At at, int np0 = 0, int np1 = NP) {
    constexpr int G = NP < 4 ? NP : 4;   // tiles whose fragments are held together
#pragma unroll
    for (int g0 = 0; g0 < NP; g0 += G) {
        float t[2 * G][4] = {};   // of three terms: the step's own sums
#pragma unroll
        for (int x = 0; x < (NB < N ? NB : N); ++x) {
            const int j = N == 3 ? NB - 1 - x : x;
            uint32_t f[G][4];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (g0 + g < np0 || g0 + g >= np1) continue;
                if (TRANS) ldsm4t(f[g], at(g0 + g) + j * plane);
                else ldsm4(f[g], at(g0 + g) + j * plane);
            }
#pragma unroll
            for (int y = 0; y < NA; ++y) {
                const int i = N == 3 ? NA - 1 - y : y;
                if (i + j >= N) continue;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    if (g0 + g < np0 || g0 + g >= np1) continue;
                    mma(N == 3 ? t[2 * g] : acc[2 * (g0 + g)], a[i], f[g][0], f[g][1]);
                    mma(N == 3 ? t[2 * g + 1] : acc[2 * (g0 + g) + 1], a[i], f[g][2], f[g][3]);
                }
            }
        }
        if constexpr (N == 3) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (g0 + g < np0 || g0 + g >= np1) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[2 * (g0 + g)][e] += t[2 * g][e];
                    acc[2 * (g0 + g) + 1][e] += t[2 * g + 1][e];
                }
            }
        }
    }
}

// Float32 rows' saved tiles lie in cores of 8 rows of 16 bytes: states [16 value columns][dk], writes and their gradients [64
// rows][16 value columns]; row r, unit u of 8 columns. bfloat16 rows' are whole: per term units of 8 value columns, of dk or 64
// rows of 16 bytes.
__device__ __forceinline__ uint32_t state_at(int r, int u) { return static_cast<uint32_t>(u * 256 + (r >> 3) * 128 + (r & 7) * 16); }
__device__ __forceinline__ uint32_t rows_at(int r, int u) { return static_cast<uint32_t>(u * 1024 + (r >> 3) * 128 + (r & 7) * 16); }

// A whole tile in shared memory leaves for contiguous global memory by itself; the writes before were the block's own.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, int bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- the walks of bfloat16 rows, forwards and from the end ---------------------------------------------------------------------
template <int DKP, int BV>
struct WalkTc {
    static constexpr int kKQ = 2 * kC * DKP * 2, kV = kC * (BV < 64 ? 64 : BV) * 2, kT = 2 * 16384, kS = BV * DKP * 2, kR = kC * BV * 2;
    // [K; Q] twice (a tile of 128 rows for 64 columns), V or dY (64 rows for 64 columns), [T; scale A T], the state's terms, R's and
    // U's (or their gradients')
    static constexpr int KQ = 0, V = 2 * kKQ, T = V + kV, S = T + kT, R = S + 2 * kS, end = R + 2 * kR;
    // K^T and T^T are read as operands of 128 columns from their tiles' starts (what lies beyond their own is not used)
    static constexpr int bytes = end > kKQ + 32768 ? end : kKQ + 32768;
    static constexpr int threads = BV * 4;
    // Two terms of a computed operand lie side by side, so one product takes both, with sums side by side, where that is faster:
    // 42 cycles for 2 x 32 columns and 65 for 2 x 64, not 2 x 34 and 2 x 42; 130 for 2 x 128 columns as for 2 products.
    static constexpr int terms = BV <= 64 ? 1 : 2, N = BV <= 64 ? 2 * BV : BV;   // products for two terms, and the columns of each
    static constexpr int cols = 2 * N;
    // 32 columns of a row of the sums
    __device__ static __forceinline__ void sums(uint32_t d, uint64_t (&v)[16]) {
        if constexpr (terms == 1) {
            float x[32], y[32];
            tensor::fetch32(d, x);
            tensor::fetch32(d + BV, y);
            tensor::arrived(x);
            tensor::arrived(y);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = add2(pack2(x[2 * i], x[2 * i + 1]), pack2(y[2 * i], y[2 * i + 1]));
        } else {
            tensor::load32(d, v);
        }
    }
};

// Two float32 as two terms of bfloat16, the rests subtracted together
__device__ __forceinline__ void terms2(uint64_t v, uint32_t& hi, uint32_t& lo) {
    float x, y;
    unpack2(v, x, y);
    hi = round2(x, y);
    float s, t;
    unpack2(fma2(pack2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)), pack2(-1.f, -1.f), v), s, t);
    lo = round2(s, t);
}
// 32 values (16 pairs) as two terms: units of 8 columns, 16 bytes each, `pitch` bytes apart
__device__ __forceinline__ void put_terms(unsigned char* hi, unsigned char* lo, int pitch, const uint64_t (&v)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) terms2(v[4 * q + e], h[e], l[e]);
        *reinterpret_cast<uint4*>(hi + q * pitch) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + q * pitch) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}
// Two bfloat16 as a pair of float32
__device__ __forceinline__ uint64_t widen2(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

// The copies of a walk's blocks. Whole blocks arrive by themselves (one thread names them);
// a sequence's last rows, and heads of other sizes, are copied by all threads, with zeros where there is nothing.
template <int DKP, int BV>
struct WalkLoads {
    using W = WalkTc<DKP, BV>;
    const Args& a;
    const Maps& m;
    const Planes& v;
    int64_t b, len, id0;
    uint32_t base, vecs, bar;   // bar: of [K; Q]'s two stages, and of V and T
    int h, kh, c0, cols, tid, warp;
    bool empty;                 // V is zero
    __device__ __forceinline__ int rows_of(int64_t j) const { return static_cast<int>(min(len - j * kC, int64_t(kC))); }
    __device__ __forceinline__ bool boxed(int64_t j) const { return m.boxes && rows_of(j) == kC; }
    __device__ __forceinline__ int first() const { return BV < 64 ? c0 >> 3 & 4 : 0; }   // the block's first unit of its box
    __device__ __forceinline__ void kq(int64_t j) const {
        const int s = static_cast<int>(j & 1);
        const uint32_t to = base + W::KQ + s * W::kKQ, full = bar + 8 * s;
        const bool box = boxed(j);
        if (warp == 1 && tensor::elect()) {
            tensor::barrier_expect(full, kVecs * kC * 4 + (box ? W::kKQ : 0));
            if (box) {
                const int row = static_cast<int>(b + j * kC);
#pragma unroll
                for (int x = 0; x < DKP / 64; ++x) {
                    tensor::copy_box(to + x * 16384, &m.k, kh * DKP + x * 64, row, full);
                    tensor::copy_box(to + x * 16384 + 8192, &m.q, kh * DKP + x * 64, row, full);
                }
            }
            tensor::copy_bulk(vecs + s * (kVecs * kC * 4), a.vec + ((id0 + j) * a.Hv + h) * kVecs * kC, kVecs * kC * 4, full);
        }
        if (!box) {
            const int n = rows_of(j);
            for (int i = tid; i < 2 * kC * (DKP / 8); i += W::threads) {
                const int r = i / (DKP / 8), u = i % (DKP / 8), t = r & 63;
                const Planes x = r < kC ? a.k : a.q;
                const bool there = t < n && u * 8 < a.dk;
                copy16(to + (u >> 3) * 16384 + swizzled_at(r, u & 7), there ? x.p + (b + j * kC + t) * x.ld + kh * a.dk + u * 8 : x.p, there);
            }
            copies_commit();
        }
    }
    __device__ __forceinline__ void vt(int64_t j) const {
        const uint32_t full = bar + 16;
        const bool box = boxed(j) && !empty;
        if (warp == 1 && tensor::elect()) {
            tensor::barrier_expect(full, W::kT + (box ? W::kV : 0));
            tensor::copy_bulk(base + W::T, a.tri + ((id0 + j) * a.Hv + h) * (W::kT / 2), W::kT, full);
            if (box) {
#pragma unroll
                for (int x = 0; x < W::kV / 8192; ++x)
                    tensor::copy_box(base + W::V + x * 8192, &m.v, h * a.dv + (c0 & ~63) + x * 64, static_cast<int>(b + j * kC), full);
            }
        }
        if (!box && !empty) {
            const int n = rows_of(j);
            for (int i = tid; i < kC * (BV / 8); i += W::threads) {
                const int r = i / (BV / 8), u = i % (BV / 8);
                const bool there = r < n && u * 8 < cols;
                copy16(base + W::V + (u >> 3) * 8192 + swizzled_at(r, first() + (u & 7)), there ? v.p + (b + j * kC + r) * v.ld + h * a.dv + c0 + u * 8 : v.p, there);
            }
            copies_commit();
        }
    }
};

// ---- host side, in sdm_gdr.cu ---------------------------------------------------------------------------
inline int padded(int d) { return d <= 64 ? 64 : 128; }
inline int64_t blocks_of(const sdm_gdr_shape* s) { return s->rows / kC + s->P; }

// Value columns of a block of a walk of bfloat16 rows, of `heads` walks of dv (and dk, for a segment's move) columns. A block of rows
// took 1.8 us with 32, 2.1 with 64 and 3.6 with 128 columns (keys of 64) on an SM of its own, and the rule takes the SMs to hold one
// block each: the fewest rounds of the grid times that (`time`, in 0.36 us a block of rows). With keys of 64 two blocks of 32 columns, or
// of 64 in segments' first walk, do fit an SM, which the rule leaves out: it then counts rounds that run side by side. 12 prompts of 16 heads of 128 took 294 us with 64 and 402 with 128, 8 of 4096 rows 380 with 64 and 349 with 128,
// one of 8 heads 952 with 32 and 1143 with 64.
inline int columns(int64_t heads, int dv, int dk = 0, int64_t* time = nullptr) {
    int best = 32;
    int64_t least = INT64_MAX;
    for (const auto& [bv, cost] : {std::pair{128, 10}, {64, 6}, {32, 5}}) {
        if (bv > 32 && dv <= bv / 2) continue;
        const int64_t grid = heads * ((dv + bv - 1) / bv + (dk + bv - 1) / bv), t = (grid + 151) / 152 * cost;
        if (t < least) best = bv, least = t;
    }
    if (time != nullptr) *time = least;
    return best;
}
inline sdm_status check_array(const void* p, int64_t ld, int64_t n, int elem, int align, bool out) {
    if (p == nullptr) return SDM_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(p) % align != 0 || (ld * elem) % align != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? n : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

// The workspace's parts in bytes from its start
struct Layout {
    int64_t tri, vec, q, k, v, start, move, ends, dy, dstates, du, part, bytes;
};
inline int terms(const sdm_gdr_shape* s) { return s->x_dtype == SDM_F32 ? 3 : 2; }   // of what is computed
sdm_status check_shape(const sdm_gdr_shape* s);
Layout layout(const sdm_gdr_shape* s, bool backward);
// The saved states, writes, triangles and gates: the parts of one array
void set_states(const sdm_gdr_shape* s, void* states, Args* a);
// The checks of what both directions take, and the arguments that follow from it
sdm_status check_inputs(const sdm_gdr_shape* s, const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                        const void* g, int64_t g_ld, const void* beta, int64_t b_ld, const int64_t* offsets, void* ws,
                        size_t ws_bytes, bool backward, uint32_t* status, Args* a);
cudaError_t launch_split(const void* x, int64_t ld, int64_t rows, int cols, __nv_bfloat16* out, cudaStream_t cs);
// q, k and v as planes (float32 rows are cut first)
cudaError_t launch_planes(const sdm_gdr_shape* s, const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                          void* ws, bool backward, Args* a, cudaStream_t cs);
cudaError_t launch_prepare(const Args& a, const sdm_gdr_shape* s, cudaStream_t cs);
// The maps of a walk over bv value columns a block
cudaError_t make_maps(Maps* m, const Args& a, const Planes& v, int bv);

}  // namespace gdr
}  // namespace sdm
