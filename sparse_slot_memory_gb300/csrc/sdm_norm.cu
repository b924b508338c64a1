// sdm_norm.cu -- the norms behind and before a block, fused with its gate, the residual's scale and its sum, and their backward:
// sdm_block_norm / sdm_block_norm_backward (include/sdm.h).
//
// Mathematics. Of a row: m = o rsqrt(mean o^2 + eps) w_post by groups of columns, n = m act(z), r = x + scale cs n rounded to
// the rows' type, y = r rsqrt(mean r^2 + eps) w_pre of r as it is stored. Backward, with p and q the two rsqrt, u = dy w_pre:
//   dR = dr + q (u - r q^2 mean(u r)) = dx,   dn = scale cs dR,   dz = dn m act'(z),   v = dn act(z) w_post,
//   do = p (v - o p^2 mean(v o)),   dw_pre += dy r q,   dw_post += dn act(z) o p,   dcs += scale dR n.
// Everything between the loads and the stores is float32; each output is rounded once.
//
// Layout. A group's columns lie on `lanes` threads (a power of two), U units of 4 columns each, a row's groups on neighbouring
// threads, so a row is read once and stays in registers through both norms; sums go through shuffles and, beyond a warp, one
// barrier. Blocks walk the rows, of the backward as many as reside, of the forward 2048 threads an SM, of which registers let a quarter
// (float32) to three eighths reside, so that its last blocks come late. The weights' gradients grow in shared memory, where every place has one thread, to
// a row of partial sums for each block, which a second kernel adds in order. The floor is HBM. Measured: 16384 x 4096 bf16 with every
// part, both directions, 454 us of 198 (the backward issues in 57 % of the cycles, 60 instructions an element, among them 8-byte loads and
// stores, weights read for every row and sums in shared memory, at 25 % of the warps, which its rows' registers leave; 3.1 TB/s under the
// profiler); 16001 x 16 heads of 120, 171 us of 54 (instructions too: of a head's 32 places of 4 columns 2 are idle). float32 rows' backward
// with four places a thread and a gate spills 100 to 116 bytes, with eight places both directions spill up to 204.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

constexpr int kNormThreads = 512;
constexpr int kMaxCols = 16384;
constexpr int kPartBlocks = 304;   // blocks of the backward at most (two for each of 152 SMs): a row of partial sums each

struct NormArgs {
    const void* o;
    const void* z;          // gate: nullable
    const void* x;          // forward, residual: nullable
    const void* rin;        // backward: r
    const void* dr;         // nullable: zeros
    const void* dy;
    const float* w_post;    // nullable: ones
    const float* w_pre;     // nullable: ones
    const float* cs;        // nullable: ones
    void* r;
    void* y;
    void* d_o;
    void* dz;
    void* dx;               // nullable
    float* part;            // backward: [3][blocks][D]: dw_post (of its rows the first G columns), dw_pre, dcs
    int64_t o_ld, z_ld, x_ld, r_ld, dr_ld, dy_ld, y_ld, do_ld, dz_ld, dx_ld;
    int64_t rows;
    int D, G, groups, post, pre;
    int lanes;              // threads of a group
    int row_threads;        // threads of a row: a power of two up to a warp, else whole warps
    int rows_block;         // rows of a block
    int want;               // backward: 1 dw_post, 2 dw_pre, 4 dcs
    float eps, scale;
};

// Sums of NR values over a row's threads and of NG over a group's. Beyond a warp they meet in shared memory, a warp's sum a lane;
// two buffers take turns, so that one barrier a call suffices.
struct Sums {
    float (*red)[3][kNormThreads / 32];
    int turn, lane, warp, row_warp, row_warps, group_warp, group_warps, row_width, group_width;
    __device__ __forceinline__ Sums(const NormArgs& a, float (*shared)[3][kNormThreads / 32]) : red(shared), turn(0) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        row_width = min(a.row_threads, 32);
        group_width = min(a.lanes, 32);
        row_warps = (a.row_threads + 31) / 32;
        group_warps = (a.lanes + 31) / 32;
        row_warp = warp / row_warps * row_warps;
        // a group of several warps starts at a multiple of its threads within its row
        group_warp = row_warp + (warp - row_warp) / group_warps * group_warps;
    }
    template <int N>
    __device__ __forceinline__ static void across(float (&v)[N], int width) {
        if (width == 32) {
#pragma unroll
            for (int m = 16; m > 0; m /= 2)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], m);
        } else {
            for (int m = width / 2; m > 0; m /= 2)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], m);
        }
    }
    template <int N>
    __device__ __forceinline__ void meet(float (&v)[N], int first, int warps, int at) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane < warps ? red[turn][at + i][first + lane] : 0.f;
#pragma unroll
        for (int m = kNormThreads / 64; m > 0; m /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], m);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(kFull, v[i], 0);
    }
    template <int N>
    __device__ __forceinline__ void row(float (&v)[N]) {
        across(v, row_width);
        if (row_warps == 1) return;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][i][warp] = v[i];
        }
        __syncthreads();
        meet(v, row_warp, row_warps, 0);
        turn ^= 1;
    }
    __device__ __forceinline__ void group(float& x) {
        float v[1] = {x};
        across(v, group_width);
        if (group_warps > 1) {
            if (lane == 0) red[turn][2][warp] = v[0];
            __syncthreads();
            meet(v, group_warp, group_warps, 2);
            turn ^= 1;
        }
        x = v[0];
    }
    __device__ __forceinline__ void row_and_group(float (&r)[2], float& x) {
        float v[1] = {x};
        across(r, row_width);
        across(v, group_width);
        if (row_warps > 1) {
            if (lane == 0) {
                red[turn][0][warp] = r[0];
                red[turn][1][warp] = r[1];
                red[turn][2][warp] = v[0];
            }
            __syncthreads();
            meet(r, row_warp, row_warps, 0);
            if (group_warps > 1) meet(v, group_warp, group_warps, 2);
            turn ^= 1;
        }
        x = v[0];
    }
};

// act and its slope: GATE 1 sigmoid, 2 z sigmoid(z); at infinite z their limits, NaN stays. bfloat16 rows take the hardware's
// exponential and reciprocal, off by 2^-21 (|z| + 1) at most where the rows are 2^-8 apart, and cut z off at -88 and, in the
// slope, at 88. Both instructions give 0 for what is below 2^-126, so that gates and slopes are at their limits there, and what they
// lose on the way is below 2^-126 of a sigmoid and 2^-119 of z sigmoid(z). float32 rows take expf and a rounded division.
__device__ __forceinline__ float max_nan(float a, float b) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
    return o;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float o;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
    return o;
}
template <typename T, int GATE>
__device__ __forceinline__ void gate_of(float z, float& act, float& slope) {
    float sg, rest, zc = z;   // sigmoid, 1 - sigmoid
    if (sizeof(T) == 2) {
        z = max_nan(z, -88.f);
        zc = min_nan(z, 88.f);
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(zc * -1.44269504088896341f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(sg) : "f"(1.f + e));
        rest = e * sg;
    } else {
        const float t = expf(-fabsf(z)), s = 1.f / (1.f + t);
        sg = z >= 0.f ? s : t * s;
        rest = z >= 0.f ? t * s : s;
        if (t == 0.f) {
            z = sg == 0.f ? 0.f : z;
            zc = 0.f;
        }
    }
    if (GATE == 1) {
        act = sg;
        slope = sg * rest;
    } else {
        act = z * sg;
        slope = fmaf(zc * sg, rest, sg);
    }
}
template <typename T, int GATE>
__device__ __forceinline__ void gates_of(const Raw4<T>& z, Quad& act, Quad& slope) {
    float v[4], a[4], s[4];
    z.get(v);
#pragma unroll
    for (int e = 0; e < 4; ++e) gate_of<T, GATE>(v[e], a[e], s[e]);
    act = quad(a);
    slope = quad(s);
}

// Four values in the rows' type, as they are stored
__device__ __forceinline__ Raw4<float> rounded(const Quad& q, float) {
    float v[4];
    floats(q, v);
    Raw4<float> r;
    r.v = make_float4(v[0], v[1], v[2], v[3]);
    return r;
}
__device__ __forceinline__ Raw4<__nv_bfloat16> rounded(const Quad& q, __nv_bfloat16) {
    float v[4];
    floats(q, v);
    Raw4<__nv_bfloat16> r;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    r.v.x = *reinterpret_cast<const uint32_t*>(&lo);
    r.v.y = *reinterpret_cast<const uint32_t*>(&hi);
    return r;
}
__device__ __forceinline__ void put(float* p, const Raw4<float>& r) { *reinterpret_cast<float4*>(p) = r.v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, const Raw4<__nv_bfloat16>& r) { *reinterpret_cast<uint2*>(p) = r.v; }
__device__ __forceinline__ float sum_of(const Quad& q) {
    float v[4];
    floats(q, v);
    return (v[0] + v[1]) + (v[2] + v[3]);
}

// A thread's units: U places of 4 columns, `lanes` units apart within its group.
template <int U>
struct Columns {
    int c[U];
    int w[U];   // its place in the group
    bool on[U];
    int row;    // its row within the block's
    __device__ __forceinline__ explicit Columns(const NormArgs& a) {
        row = threadIdx.x / a.row_threads;
        const int t = threadIdx.x - row * a.row_threads, group = t / a.lanes, sub = t - group * a.lanes;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = sub + i * a.lanes;
            on[i] = group < a.groups && u * 4 < a.G && row < a.rows_block;
            w[i] = on[i] ? u * 4 : 0;
            c[i] = on[i] ? group * a.G + u * 4 : 0;
        }
    }
};

__device__ __forceinline__ Quad weights(const float* w, int c) { return w == nullptr ? quad(1.f) : quad(load4(w + c)); }
template <typename T>
__device__ __forceinline__ void take(Raw4<T>& r, const void* p, int64_t row, int64_t ld, int c, bool on) {
    r.zero();
    if (on) ld_plain(r, static_cast<const T*>(p) + row * ld + c);
}

// MAXT: threads of a block at most
template <typename T, int U, int GATE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? (sizeof(T) == 2 ? 3 : 2) : 1) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float red[2][3][kNormThreads / 32];
    start_dependent();
    const Columns<U> col(a);
    Sums sums(a, red);
    const int64_t stride = gridDim.x * int64_t(a.rows_block);
    Raw4<T> o[U], z[U], x[U];
    auto take_row = [&](int64_t row, int i) {
        const bool on = row < a.rows && col.on[i];
        take(o[i], a.o, row, a.o_ld, col.c[i], on);
        take(z[i], a.z, row, a.z_ld, col.c[i], on && GATE != 0);
        take(x[i], a.x, row, a.x_ld, col.c[i], on && a.x != nullptr);
    };
#pragma unroll
    for (int i = 0; i < U; ++i) take_row(blockIdx.x * int64_t(a.rows_block) + col.row, i);
    for (int64_t base = blockIdx.x * int64_t(a.rows_block); base < a.rows; base += stride) {
        const int64_t row = base + col.row;
        const bool here = row < a.rows;
        float p = 1.f;
        if (a.post) {
            Quad sq = quad(0.f);
#pragma unroll
            for (int i = 0; i < U; ++i) sq = fma4(quad(o[i]), quad(o[i]), sq);
            float s = sum_of(sq);
            sums.group(s);
            p = rsqrtf(s / a.G + a.eps);
        }
        Raw4<T> r[U];
        Quad sq = quad(0.f);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            Quad n = quad(o[i]);
            if (a.post) n = mul4(mul4(n, quad(p)), weights(a.w_post, col.w[i]));
            if constexpr (GATE != 0) {
                Quad act, slope;
                gates_of<T, GATE>(z[i], act, slope);
                n = mul4(n, act);
            }
            Quad k = quad(a.scale);
            if (a.cs != nullptr) k = mul4(k, weights(a.cs, col.c[i]));
            r[i] = rounded(fma4(k, n, quad(x[i])), T{});   // as it is stored
            if (here && col.on[i]) put(static_cast<T*>(a.r) + row * a.r_ld + col.c[i], r[i]);
            else r[i].zero();
            sq = fma4(quad(r[i]), quad(r[i]), sq);
        }
        // the next row comes while this one's second norm goes on
#pragma unroll
        for (int i = 0; i < U; ++i) take_row(row + stride, i);
        if (!a.pre) continue;
        float s[1] = {sum_of(sq)};
        sums.row(s);
        const float q = rsqrtf(s[0] / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!here || !col.on[i]) continue;
            put(static_cast<T*>(a.y) + row * a.y_ld + col.c[i],
                rounded(mul4(mul4(quad(r[i]), quad(q)), weights(a.w_pre, col.c[i])), T{}));
        }
    }
}

// With U of 8 a thread cannot hold five rows' places: they are read again (from the L2) where they are used.
template <typename T, int U, int GATE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool kAgain = U == 8;
    __shared__ float red[2][3][kNormThreads / 32];
    extern __shared__ __align__(16) float grown[];   // [rows of the block][kinds wanted][D]
    start_dependent();
    const Columns<U> col(a);
    Sums sums(a, red);
    const int kinds = __popc(a.want);
    float* const mine = grown + static_cast<int64_t>(min(col.row, a.rows_block - 1)) * kinds * a.D;
    float* const dpost = mine;
    float* const dpre = mine + __popc(a.want & 1) * a.D;
    float* const dcs = mine + __popc(a.want & 3) * a.D;
    auto grow = [&](float* p, const Quad& v) { st4(p, add4(quad_at(p), v)); };
    for (int i = threadIdx.x; i < a.rows_block * kinds * a.D; i += blockDim.x) grown[i] = 0.f;
    __syncthreads();
    const int64_t stride = gridDim.x * int64_t(a.rows_block);
    Raw4<T> o[U], z[U], r[U], g[U], dy[U], next[U];
    auto take_r = [&](int64_t row, int i) {
        const bool on = row < a.rows && col.on[i] && a.pre;
        take(r[i], a.rin, row, a.r_ld, col.c[i], on);
        take(dy[i], a.dy, row, a.dy_ld, col.c[i], on);
    };
    auto take_g = [&](int64_t row, int i) {
        const bool on = row < a.rows && col.on[i];
        take(z[i], a.z, row, a.z_ld, col.c[i], on && GATE != 0);
        take(g[i], a.dr, row, a.dr_ld, col.c[i], on && a.dr != nullptr);
    };
    auto take_o = [&](Raw4<T>& to, int64_t row, int i) { take(to, a.o, row, a.o_ld, col.c[i], row < a.rows && col.on[i]); };
    if (!kAgain) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t row = blockIdx.x * int64_t(a.rows_block) + col.row;
            take_r(row, i);
            take_o(next[i], row, i);
            take_g(row, i);
        }
    }
    for (int64_t base = blockIdx.x * int64_t(a.rows_block); base < a.rows; base += stride) {
        const int64_t row = base + col.row;
        const bool here = row < a.rows;
        if (!kAgain) {
#pragma unroll
            for (int i = 0; i < U; ++i) o[i] = next[i];
        }
        Quad rr = quad(0.f), ur = quad(0.f), oo = quad(0.f);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (kAgain) {
                take_r(row, i);
                take_o(o[i], row, i);
            }
            if (a.pre) {
                const Quad rv = quad(r[i]);
                rr = fma4(rv, rv, rr);
                ur = fma4(mul4(quad(dy[i]), weights(a.w_pre, col.c[i])), rv, ur);
            }
            if (a.post) oo = fma4(quad(o[i]), quad(o[i]), oo);
        }
        float s[2] = {sum_of(rr), sum_of(ur)}, so = sum_of(oo);
        if (a.pre && a.post) sums.row_and_group(s, so);
        else if (a.pre) sums.row(s);
        else if (a.post) sums.group(so);
        const float q = rsqrtf(s[0] / a.D + a.eps), p = a.post ? rsqrtf(so / a.G + a.eps) : 1.f;
        const Quad back = quad(-q * q * (s[1] / a.D)), q4 = quad(q), p4 = quad(p), scale = quad(a.scale);
        Quad v[U], vo = quad(0.f);   // dn act(z) w_post, and its product with o
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (kAgain) {
                take_r(row, i);
                take_o(o[i], row, i);
                take_g(row, i);
            }
            const bool on = here && col.on[i];
            Quad d = quad(g[i]);
            if (a.pre) {
                const Quad rv = quad(r[i]), dv = quad(dy[i]);
                d = fma4(q4, fma4(rv, back, mul4(dv, weights(a.w_pre, col.c[i]))), d);
                if (on && (a.want & 2)) grow(dpre + col.c[i], mul4(dv, mul4(rv, q4)));
            }
            if (a.dx != nullptr && on) put(static_cast<T*>(a.dx) + row * a.dx_ld + col.c[i], rounded(d, T{}));
            const Quad ov = quad(o[i]), h = mul4(ov, p4);
            const Quad w = a.post ? weights(a.w_post, col.w[i]) : quad(1.f);
            const Quad m = a.post ? mul4(h, w) : ov;
            d = mul4(scale, d);
            Quad act = quad(1.f), slope;
            if constexpr (GATE != 0) gates_of<T, GATE>(z[i], act, slope);
            if (on && (a.want & 4)) grow(dcs + col.c[i], mul4(d, GATE != 0 ? mul4(m, act) : m));
            if (a.cs != nullptr) d = mul4(d, weights(a.cs, col.c[i]));
            if constexpr (GATE != 0) {
                if (on) put(static_cast<T*>(a.dz) + row * a.dz_ld + col.c[i], rounded(mul4(mul4(d, m), slope), T{}));
                d = mul4(d, act);
            }
            v[i] = d;
            if (a.post) {
                if (on && (a.want & 1)) grow(dpost + col.c[i], mul4(d, h));
                v[i] = mul4(d, w);
                vo = fma4(v[i], ov, vo);
            }
        }
        if (!kAgain) {   // the next row comes while this one's second sum goes on
#pragma unroll
            for (int i = 0; i < U; ++i) {
                take_r(row + stride, i);
                take_o(next[i], row + stride, i);
                take_g(row + stride, i);
            }
        }
        Quad k = quad(0.f);
        if (a.post) {
            float sv = sum_of(vo);
            sums.group(sv);
            k = quad(-p * p * (sv / a.G));
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (kAgain) take_o(o[i], row, i);
            if (!here || !col.on[i]) continue;
            put(static_cast<T*>(a.d_o) + row * a.do_ld + col.c[i], rounded(a.post ? mul4(p4, fma4(quad(o[i]), k, v[i])) : v[i], T{}));
        }
    }
    if (kinds == 0) return;
    __syncthreads();
    // the block's rows in order, of dw_post for each group in order
    for (int kind = 0; kind < 3; ++kind) {
        if (!(a.want >> kind & 1)) continue;
        const float* const from = kind == 0 ? grown + (dpost - mine) : kind == 1 ? grown + (dpre - mine) : grown + (dcs - mine);
        const int n = kind == 0 ? a.G : a.D;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            float s = 0.f;
            for (int w = 0; w < a.rows_block; ++w)
                for (int c = i; c < a.D; c += n) s += from[w * kinds * a.D + c];
            a.part[(static_cast<int64_t>(kind) * gridDim.x + blockIdx.x) * a.D + i] = s;
        }
    }
}

// A kind's gradients: the blocks' rows in 32 shares, each in order, and those in order. Block y: the kind. What the shape does not have
// (asked for and not in `want`, so that no block wrote a row of it) is the sum of no rows: 0.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int blocks, int D, int G, int asked, int want, float* dw_post,
                                                       float* dw_pre, float* dcs) {
    __shared__ float s[32][33];
    start_dependent();
    const int kind = blockIdx.y, n = kind == 0 ? G : D;
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (!(asked >> kind & 1) || blockIdx.x * 32 >= n) return;
    if (!(want >> kind & 1)) blocks = 0;
    float sum = 0.f;
    if (c < n) {
        const float* const p = part + static_cast<int64_t>(kind) * blocks * D + c;
#pragma unroll 5
        for (int b = threadIdx.y; b < blocks; b += 32) sum += p[static_cast<int64_t>(b) * D];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y != 0 || c >= n) return;
    sum = 0.f;
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    (kind == 0 ? dw_post : kind == 1 ? dw_pre : dcs)[c] = sum;
}

// ---- host side ------------------------------------------------------------------------------------
using checks::aligned16;
using checks::aligned_all;

sdm_status check(const sdm_norm_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->dtype < 0 || s->dtype > 1) return SDM_ERR_DTYPE;
    if (s->rows < 0 || s->rows > (int64_t(1) << 40) || s->D < 1 || s->D > kMaxCols || s->group < 1 || s->group > s->D ||
        s->D % s->group != 0 || s->post < 0 || s->post > 1 || s->gate < 0 || s->gate > 2 || s->residual < 0 || s->residual > 1 ||
        s->pre < 0 || s->pre > 1 || !(s->eps >= 0.f) || !(s->scale == s->scale))
        return SDM_ERR_SHAPE;
    if (s->group % 4 != 0) return SDM_ERR_ALIGN;
    return SDM_OK;
}

sdm_status check_rows(const sdm_norm_shape* s, const void* p, int64_t ld, bool out) {
    if (p == nullptr) return SDM_ERR_ARG;
    const int e = s->dtype == SDM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(p) % (4 * e) != 0 || ld % 4 != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? s->D : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

int pow2(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// The threads of a group, U and the rows of a block: the U that leaves the fewest places idle, 4 where it makes no difference; 8 where a
// row's threads fit a block no other way, of which more than 256 are left.
// 0: a row's threads do not fit a block.
int geometry(const sdm_norm_shape* s, NormArgs* a) {
    memset(a, 0, sizeof(*a));
    a->rows = s->rows;
    a->D = s->D;
    a->G = s->post ? s->group : s->D;   // without the norm behind the block its groups do not matter
    a->groups = a->D / a->G;
    a->post = s->post;
    a->pre = s->pre;
    a->eps = s->eps;
    a->scale = s->scale;
    int best = 0, U = 0;
    for (int u : {4, 3, 2, 1, 8}) {
        const int lanes = pow2((a->G / 4 + u - 1) / u), threads = a->groups * lanes;
        if (threads > kNormThreads) continue;
        if (U != 0 && lanes * u >= best) continue;
        best = lanes * u;
        U = u;
        a->lanes = lanes;
    }
    if (U == 0) return 0;
    const int threads = a->groups * a->lanes;
    a->row_threads = threads <= 32 ? pow2(threads) : (threads + 31) / 32 * 32;
    a->rows_block = std::max(1, 256 / a->row_threads);
    return U;
}

int bwd_blocks(const NormArgs& a) {
    const int64_t n = (a.rows + a.rows_block - 1) / a.rows_block;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kPartBlocks, n)));
}

template <typename F>
cudaError_t by_type(const sdm_norm_shape* s, int U, F f) {
    auto gates = [&](auto t, auto u) {
        return s->gate == 0 ? f(t, u, std::integral_constant<int, 0>{})
               : s->gate == 1 ? f(t, u, std::integral_constant<int, 1>{}) : f(t, u, std::integral_constant<int, 2>{});
    };
    auto units = [&](auto t) {
        switch (U) {
            case 1: return gates(t, std::integral_constant<int, 1>{});
            case 2: return gates(t, std::integral_constant<int, 2>{});
            case 3: return gates(t, std::integral_constant<int, 3>{});
            case 4: return gates(t, std::integral_constant<int, 4>{});
            default: return gates(t, std::integral_constant<int, 8>{});
        }
    };
    return s->dtype == SDM_BF16 ? units(__nv_bfloat16{}) : units(0.f);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_block_norm_workspace_bytes(const sdm_norm_shape* shape) {
    NormArgs a;
    if (check(shape) != SDM_OK || geometry(shape, &a) == 0) return 0;
    return static_cast<size_t>(3) * bwd_blocks(a) * a.D * sizeof(float);
}

extern "C" sdm_status sdm_block_norm(const sdm_norm_shape* shape, const void* o, int64_t o_ld, const void* z, int64_t z_ld,
                                     const void* x, int64_t x_ld, const float* w_post, const float* w_pre,
                                     const float* channel_scale, void* r, int64_t r_ld, void* y, int64_t y_ld,
                                     sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    NormArgs a;
    const int U = geometry(shape, &a);
    if (U == 0) return SDM_ERR_SHAPE;
    if (shape->rows == 0) return SDM_OK;
    if ((st = check_rows(shape, o, o_ld, false)) != SDM_OK) return st;
    if (shape->gate && (st = check_rows(shape, z, z_ld, false)) != SDM_OK) return st;
    if (shape->residual && (st = check_rows(shape, x, x_ld, false)) != SDM_OK) return st;
    if ((st = check_rows(shape, r, r_ld, true)) != SDM_OK) return st;
    if (shape->pre && (st = check_rows(shape, y, y_ld, true)) != SDM_OK) return st;
    if (!aligned_all(16, {w_post, w_pre, channel_scale})) return SDM_ERR_ALIGN;
    a.o = o; a.o_ld = o_ld; a.z = z; a.z_ld = z_ld; a.x = shape->residual ? x : nullptr; a.x_ld = x_ld;
    a.w_post = w_post; a.w_pre = w_pre; a.cs = channel_scale; a.r = r; a.r_ld = r_ld; a.y = y; a.y_ld = y_ld;
    const int threads = (a.rows_block * a.row_threads + 31) / 32 * 32;
    const int64_t blocks = std::min<int64_t>((a.rows + a.rows_block - 1) / a.rows_block, 152 * (2048 / threads));
    const cudaError_t e = by_type(shape, U, [&](auto t, auto u, auto gate) {
        constexpr int N = decltype(u)::value, G = decltype(gate)::value;
        auto* const k = threads <= 256 ? norm_fwd_kernel<decltype(t), N, G, N == 8 ? kNormThreads : 256> : norm_fwd_kernel<decltype(t), N, G, kNormThreads>;
        return launch_dependent(k, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream), a);
    });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_block_norm_backward(const sdm_norm_shape* shape, const void* o, int64_t o_ld, const void* z, int64_t z_ld,
                                              const void* r, int64_t r_ld, const void* dr, int64_t dr_ld, const void* dy,
                                              int64_t dy_ld, const float* w_post, const float* w_pre,
                                              const float* channel_scale, void* d_o, int64_t do_ld, void* dz, int64_t dz_ld,
                                              void* dx, int64_t dx_ld, float* dw_post, float* dw_pre, float* d_channel_scale,
                                              void* ws, size_t ws_bytes, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    NormArgs a;
    const int U = geometry(shape, &a);
    if (U == 0) return SDM_ERR_SHAPE;
    if (shape->rows > 0) {
        if ((st = check_rows(shape, o, o_ld, false)) != SDM_OK) return st;
        if (shape->gate && (st = check_rows(shape, z, z_ld, false)) != SDM_OK) return st;
        if (shape->pre && (st = check_rows(shape, r, r_ld, false)) != SDM_OK) return st;
        if (shape->pre && (st = check_rows(shape, dy, dy_ld, false)) != SDM_OK) return st;
        if (dr == nullptr && !shape->pre) return SDM_ERR_ARG;
        if (dr != nullptr && (st = check_rows(shape, dr, dr_ld, false)) != SDM_OK) return st;
        if ((st = check_rows(shape, d_o, do_ld, true)) != SDM_OK) return st;
        if (shape->gate && (st = check_rows(shape, dz, dz_ld, true)) != SDM_OK) return st;
        if (dx != nullptr && (st = check_rows(shape, dx, dx_ld, true)) != SDM_OK) return st;
    }
    if (!aligned_all(16, {w_post, w_pre, channel_scale}) || !aligned_all(4, {dw_post, dw_pre, d_channel_scale})) return SDM_ERR_ALIGN;
    const int asked = (dw_post != nullptr ? 1 : 0) | (dw_pre != nullptr ? 2 : 0) | (d_channel_scale != nullptr ? 4 : 0);
    a.want = asked & ((shape->post ? 1 : 0) | (shape->pre ? 2 : 0) | 4);
    const int blocks = bwd_blocks(a);
    if (a.want && (ws == nullptr || !aligned16(ws) || ws_bytes < static_cast<size_t>(3) * blocks * a.D * sizeof(float)))
        return SDM_ERR_WORKSPACE;
    a.o = o; a.o_ld = o_ld; a.z = z; a.z_ld = z_ld; a.rin = r; a.r_ld = r_ld; a.dr = dr; a.dr_ld = dr_ld; a.dy = dy; a.dy_ld = dy_ld;
    a.w_post = w_post; a.w_pre = w_pre; a.cs = channel_scale;
    a.d_o = d_o; a.do_ld = do_ld; a.dz = dz; a.dz_ld = dz_ld; a.dx = dx; a.dx_ld = dx_ld;
    a.part = static_cast<float*>(ws);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int threads = (a.rows_block * a.row_threads + 31) / 32 * 32;
    const int kinds = (a.want & 1) + (a.want >> 1 & 1) + (a.want >> 2 & 1);
    const int smem = a.rows_block * kinds * a.D * static_cast<int>(sizeof(float));
    cudaError_t e = cudaSuccess;
    if (shape->rows > 0)
        e = by_type(shape, U, [&](auto t, auto u, auto gate) {
            constexpr int N = decltype(u)::value, G = decltype(gate)::value;
            auto* const k = threads <= 256 ? norm_bwd_kernel<decltype(t), N, G, N == 8 ? kNormThreads : 256> : norm_bwd_kernel<decltype(t), N, G, kNormThreads>;
            if (smem > 47 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
                if (e != cudaSuccess) return e;
            }
            return launch_dependent(k, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, cs, a);
        });
    if (e == cudaSuccess && asked)
        e = launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((a.D + 31) / 32), 3), dim3(32, 32), 0, cs, static_cast<const float*>(ws),
                             shape->rows > 0 ? blocks : 0, a.D, shape->group, asked, a.want, dw_post, dw_pre, d_channel_scale);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
