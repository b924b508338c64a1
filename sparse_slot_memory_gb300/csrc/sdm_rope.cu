// sdm_rope.cu -- the norm of every query and key head with the position rotation in the same pass, its
// backward, and the table of the rotation: sdm_qk_norm_rope / sdm_qk_norm_rope_backward / sdm_rope_table
// (include/sdm.h).
//
// Mathematics. A head's row x [hd] with r = rsqrt(mean x^2 + eps): n = x r w, then every pair (a, b) of the
// first rot_dim columns turns by its angle: a' = a c - b s, b' = b c + a s. Backward: e = the gradient turned
// back; dw += e x r; with t = e w: dx = r (t - x r^2 mean(t x)). Everything between the load and the store is
// float32; each output is rounded once.
//
// Layout. A head's columns are taken in units of 8 that hold whole pairs: interleaved, columns 8u .. 8u + 7;
// half, columns 4u .. and rot_dim / 2 + 4u ..; behind rot_dim, 8 columns in a row. A unit's four pairs have the
// frequencies 4u .. 4u + 3 in either layout. A lane owns the same units of every head it meets, so a token's
// cosines and sines and the weights stay in registers over the heads of the token, up to four of which (two in float32)
// are on their way at once. Resident blocks walk the tokens; the weights' gradients stay in registers to the end.
//
// Bound by HBM: 4 bytes a bfloat16 element forward, 6 backward; the table's 512 bytes a token of 128 columns count
// little beside the heads. Measured on a GB300 (6.7 TB/s copy), 32768 tokens of 32 + 8 heads of 128 columns, bfloat16,
// slices of a fused projection: forward 112 us (6.0 TB/s), forward and backward 286 us (5.9 TB/s), 295 with half of the
// head turned; 32 tokens: 9.4 to 10 us a call, the host's time for it (the kernel 2.7 in a graph). 5003 tokens of 12 + 2 heads
// of 120, forward and backward: 30 to 36 us, 26 in a graph, three short kernels one after another.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

constexpr int kThreads = 256;
// Blocks of the forward on an SM: 80 registers hold four bfloat16 heads, 64 two float32 ones (4099 tokens of 32 float32
// heads of 64: 15.7 us with 3, 15.4 with 4; 32768 tokens of 40 bfloat16 heads of 128: 112 with 3, 115 with 4).
constexpr int fwd_blocks(bool bf16) { return bf16 ? 3 : 4; }
constexpr int kMaxHd = 1024;
constexpr int kMaxFreq = kMaxHd / 2;
constexpr int kPartBlocks = 304;   // blocks of the backward at most (two for each of 152 SMs): a row of weight gradients each

struct RopeArgs {
    const void* q;
    const void* k;
    const void* dqo;
    const void* dko;
    const int32_t* pos;
    const float* table;   // [max_pos, rot_dim]: cosines, then sines
    const float* wq;      // nullable: ones
    const float* wk;
    void* qo;
    void* ko;
    float* part;          // backward: [blocks][2][hd] weight gradients
    uint32_t* status;
    int64_t q_ld, k_ld, dqo_ld, dko_ld, qo_ld, ko_ld;
    int64_t tokens;
    int Hq, Hk, hd, rd, max_pos, interleaved, norm;
    float eps;
};

// A lane's place: `lanes` lanes hold a head, each `U` units of 8 columns (unit sub + i * lanes).
template <int U>
struct Place {
    int a[U], b[U];       // first columns of the unit's two halves of 4
    int f[U];             // its first frequency, or -1 behind rot_dim
    bool on[U];
    __device__ __forceinline__ void set(const RopeArgs& s, int sub, int lanes) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = sub + i * lanes;
            on[i] = u * 8 < s.hd;
            const int v = on[i] ? u : 0;
            const bool turned = v * 8 < s.rd;
            f[i] = turned ? 4 * v : -1;
            a[i] = turned && !s.interleaved ? 4 * v : 8 * v;
            b[i] = turned && !s.interleaved ? s.rd / 2 + 4 * v : 8 * v + 4;
        }
    }
};

// A unit's eight values as the first and the second ones of its four pairs. Behind rot_dim and in the half layout those
// are its two halves; in the interleaved one its even and odd columns.
struct Pairs {
    Quad a, b;
};
template <bool INTER>
__device__ __forceinline__ Pairs pairs(const float (&x)[4], const float (&y)[4]) {
    if (INTER) return {{pack2(x[0], x[2]), pack2(y[0], y[2])}, {pack2(x[1], x[3]), pack2(y[1], y[3])}};
    return {quad(x), quad(y)};
}
template <bool INTER, typename T>
__device__ __forceinline__ Pairs pairs(const Raw4<T>& x, const Raw4<T>& y) {
    float u[4], v[4];
    x.get(u);
    y.get(v);
    return pairs<INTER>(u, v);
}
template <bool INTER, typename T>
__device__ __forceinline__ void st_pairs(T* x, T* y, const Pairs& p) {
    float u[4], v[4];
    floats(p.a, u);
    floats(p.b, v);
    if (INTER) {
        const float s[4] = {u[0], v[0], u[1], v[1]}, t[4] = {u[2], v[2], u[3], v[3]};
        rows::st4(x, s);
        rows::st4(y, t);
    } else {
        rows::st4(x, u);
        rows::st4(y, v);
    }
}

// The cosines and sines of a unit's four pairs at a position
struct Turn {
    Quad c, s;
};
__device__ __forceinline__ Turn turn_of(const RopeArgs& s, int pos, int f) {
    if (f < 0) return {quad(1.f), quad(0.f)};
    const float* const t = s.table + static_cast<int64_t>(pos) * s.rd + f;
    return {quad(load4(t)), quad(load4(t + s.rd / 2))};
}
__device__ __forceinline__ Quad negative(const Quad& q) {
    return {q.lo ^ 0x8000000080000000ull, q.hi ^ 0x8000000080000000ull};
}
// The gradient's pairs turned back by the angle; those behind rot_dim (cosine 1, sine 0) stay as they are, whatever they
// hold: `all` says that there are none.
__device__ __forceinline__ Pairs turned_back(const Pairs& p, const Turn& t, bool all, bool on) {
    Pairs o = {fma4(p.a, t.c, mul4(p.b, t.s)), fma4(p.b, t.c, mul4(p.a, negative(t.s)))};
    if (!all && !on) o = p;
    return o;
}
// The forward's rotation with the weights in it: a' = a (wa c) - b (wb s), b' = b (wb c) + a (wa s)
struct Weighted {
    Quad ca, sb, cb, sa;
};
__device__ __forceinline__ Weighted weighted(const Turn& t, const Pairs& w) {
    return {mul4(w.a, t.c), negative(mul4(w.b, t.s)), mul4(w.b, t.c), mul4(w.a, t.s)};
}
__device__ __forceinline__ Pairs turned(const Pairs& p, const Weighted& t, bool all, bool on) {
    Pairs o = {fma4(p.a, t.ca, mul4(p.b, t.sb)), fma4(p.b, t.cb, mul4(p.a, t.sa))};
    if (!all && !on) o = {mul4(p.a, t.ca), mul4(p.b, t.cb)};
    return o;
}

template <bool INTER>
__device__ __forceinline__ Pairs weights(const float* w, int a, int b) {
    if (w == nullptr) return {quad(1.f), quad(1.f)};
    return pairs<INTER>(load4(w + a), load4(w + b));
}
__device__ __forceinline__ float sum4(const Quad& q) {
    float a, b;
    unpack2(add2(q.lo, q.hi), a, b);
    return a + b;
}
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) { return sum4(fma4(x.a, y.a, mul4(x.b, y.b))); }
__device__ __forceinline__ Pairs times(const Pairs& x, const Pairs& y) { return {mul4(x.a, y.a), mul4(x.b, y.b)}; }
__device__ __forceinline__ Pairs times(const Pairs& x, float f) {
    const Quad q = quad(f);
    return {mul4(x.a, q), mul4(x.b, q)};
}

// Each of the n values summed over the group's lanes, in every lane.
template <int n>
__device__ __forceinline__ void lanes_sum(float (&v)[n], int lanes) {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1)
        if (k < lanes) {
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(kFull, v[i], k);
        }
}

// Heads that a group of lanes takes together (their loads in flight at once, one set of cosines and sines for all).
template <typename T, int U>
constexpr int heads_at_once() {
    return U > 1 ? 1 : sizeof(T) == 2 ? 4 : 2;
}

// The token's position, or -1 for a padding token, which takes no row of the table.
__device__ __forceinline__ int position(const RopeArgs& s, int t) {
    const int pos = s.pos[t];
    if (pos < s.max_pos) return pos < 0 ? -1 : pos;
    if (s.status != nullptr) atomicOr(s.status, SDM_DEV_BAD_POSITION);
    return -1;
}

// A group's walk over units of up to HU heads of a token: unit u is token u / chunks, chunk u % chunks, and the
// next is a fixed number of units on, so that no step divides.
struct Walk {
    int u, t, ch, dt, dch, du;
    __device__ __forceinline__ Walk(int first, int step, int chunks) : u(first), t(first / chunks), ch(first % chunks), dt(step / chunks), dch(step % chunks), du(step) {}
    __device__ __forceinline__ void next(int chunks) {
        u += du;
        t += dt;
        ch += dch;
        if (ch >= chunks) {
            ch -= chunks;
            ++t;
        }
    }
};

// Groups of `lanes` lanes walk the tokens' heads, up to HU heads of one kind of one token at a time.
template <typename T, int U, bool INTER>
__global__ void __launch_bounds__(kThreads, U == 1 ? fwd_blocks(sizeof(T) == 2) : 1) rope_fwd_kernel(const RopeArgs s, int lanes) {
    constexpr int HU = heads_at_once<T, U>();
    start_dependent();
    const int per = kThreads / lanes, cq = (s.Hq + HU - 1) / HU, ct = cq + (s.Hk + HU - 1) / HU;
    const int units = static_cast<int>(s.tokens) * ct, sub = threadIdx.x % lanes;
    const float inv = 1.f / s.hd;
    const bool all = s.rd == s.hd;   // every column turns
    Place<U> pl;
    pl.set(s, sub, lanes);
    Walk at(blockIdx.x * per + threadIdx.x / lanes, gridDim.x * per, ct);
    int pos = at.u < units ? position(s, at.t) : -1;
    for (int u0 = blockIdx.x * per; u0 < units; u0 += gridDim.x * per) {   // block-uniform
        const bool live = at.u < units, isq = at.ch < cq && s.Hq > 0;
        const int t = live ? at.t : 0, h0 = live ? (isq ? at.ch : at.ch - cq) * HU : 0;
        const int n = live ? min(HU, (isq ? s.Hq : s.Hk) - h0) : 0;
        const T* const x = (isq ? static_cast<const T*>(s.q) + t * s.q_ld : static_cast<const T*>(s.k) + t * s.k_ld) + h0 * s.hd;
        T* const y = (isq ? static_cast<T*>(s.qo) + t * s.qo_ld : static_cast<T*>(s.ko) + t * s.ko_ld) + h0 * s.hd;
        const int p = pos;
        auto body = [&](auto full, auto whole) {   // full: HU heads of a real token; whole: every column turns
            constexpr bool FULL = decltype(full)::value, WHOLE = decltype(whole)::value;
            Raw4<T> ra[HU][U], rb[HU][U];
#pragma unroll
            for (int h = 0; h < HU; ++h)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (!FULL) {
                        ra[h][i].zero();
                        rb[h][i].zero();
                    }
                    if (FULL || (h < n && p >= 0)) {
                        ra[h][i].ld_cg(x + h * s.hd + pl.a[i]);
                        rb[h][i].ld_cg(x + h * s.hd + pl.b[i]);
                    }
                }
            Weighted wt[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (FULL || p >= 0)
                    wt[i] = weighted(turn_of(s, p, pl.f[i]), weights<INTER>(s.norm ? (isq ? s.wq : s.wk) : nullptr, pl.a[i], pl.b[i]));
                else   // a padding token, not read: zeros whatever the table and the weights hold
                    wt[i] = {quad(0.f), quad(0.f), quad(0.f), quad(0.f)};
            }
            at.next(ct);
            pos = at.u < units ? position(s, at.t) : -1;
            float ss[HU];
#pragma unroll
            for (int h = 0; h < HU; ++h) {
                ss[h] = 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const Pairs v = pairs<INTER>(ra[h][i], rb[h][i]);
                    const float d = dot(v, v);
                    if (pl.on[i]) ss[h] += d;
                }
            }
            if (s.norm) lanes_sum(ss, lanes);
#pragma unroll
            for (int h = 0; h < HU; ++h) {
                float r = s.norm ? rsqrtf(fmaf(ss[h], inv, s.eps)) : 1.f;
                if (!FULL && p < 0) r = 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const Pairs o = times(turned(pairs<INTER>(ra[h][i], rb[h][i]), wt[i], WHOLE, pl.f[i] >= 0), r);
                    if ((FULL || h < n) && pl.on[i]) st_pairs<INTER>(y + h * s.hd + pl.a[i], y + h * s.hd + pl.b[i], o);
                }
            }
        };
        if (!__all_sync(kFull, n == HU && p >= 0))
            body(std::false_type{}, std::false_type{});
        else if (all)
            body(std::true_type{}, std::true_type{});
        else
            body(std::true_type{}, std::false_type{});
    }
}

// Groups of lanes walk the tokens' heads, queries first, then keys; a lane's weight gradients stay in registers,
// are joined over the block in a fixed order and written as the block's row of `part`. mean(t x) does not depend on
// r, so both of a head's sums go over the lanes together.
template <typename T, int U, bool INTER>
__global__ void __launch_bounds__(kThreads, U == 1 ? 2 : 1) rope_bwd_kernel(const RopeArgs s, int lanes) {
    constexpr int HU = heads_at_once<T, U>();
    extern __shared__ float sm[];   // [groups][hd]
    start_dependent();
    const int per = kThreads / lanes, group = threadIdx.x / lanes, sub = threadIdx.x % lanes;
    const float inv = 1.f / s.hd;
    const bool all = s.rd == s.hd;   // every column turns
    Place<U> pl;
    pl.set(s, sub, lanes);
    for (int side = 0; side < 2; ++side) {
        const int H = side ? s.Hk : s.Hq, chunks = max(1, (H + HU - 1) / HU);
        const T* const X = static_cast<const T*>(side ? s.k : s.q);
        const T* const G = static_cast<const T*>(side ? s.dko : s.dqo);
        T* const Y = static_cast<T*>(side ? s.ko : s.qo);
        const int64_t x_ld = side ? s.k_ld : s.q_ld, g_ld = side ? s.dko_ld : s.dqo_ld, y_ld = side ? s.ko_ld : s.qo_ld;
        Pairs wt[U], dw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            wt[i] = weights<INTER>(s.norm ? (side ? s.wk : s.wq) : nullptr, pl.a[i], pl.b[i]);
            dw[i] = {quad(0.f), quad(0.f)};
        }
        const int units = H == 0 ? 0 : static_cast<int>(s.tokens) * chunks;
        Walk at(blockIdx.x * per + group, gridDim.x * per, chunks);
        int pos = at.u < units ? position(s, at.t) : -1;
        for (int u0 = blockIdx.x * per; u0 < units; u0 += gridDim.x * per) {   // block-uniform
            const bool live = at.u < units;
            const int t = live ? at.t : 0, h0 = live ? at.ch * HU : 0, n = live ? min(HU, H - h0) : 0;
            const T* const x = X + t * x_ld + h0 * s.hd;
            const T* const g = G + t * g_ld + h0 * s.hd;
            T* const y = Y + t * y_ld + h0 * s.hd;
            const int p = pos;
            auto body = [&](auto full, auto whole) {   // full: HU heads of a real token; whole: every column turns
                constexpr bool FULL = decltype(full)::value, WHOLE = decltype(whole)::value;
                Raw4<T> ra[HU][U], rb[HU][U], ga[HU][U], gb[HU][U];
#pragma unroll
                for (int h = 0; h < HU; ++h)
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        if (!FULL) {
                            ra[h][i].zero();
                            rb[h][i].zero();
                            ga[h][i].zero();
                            gb[h][i].zero();
                        }
                        if (FULL || (h < n && p >= 0)) {
                            ra[h][i].ld_cg(x + h * s.hd + pl.a[i]);
                            rb[h][i].ld_cg(x + h * s.hd + pl.b[i]);
                            ga[h][i].ld_cg(g + h * s.hd + pl.a[i]);
                            gb[h][i].ld_cg(g + h * s.hd + pl.b[i]);
                        }
                    }
                Turn turn[U];
#pragma unroll
                for (int i = 0; i < U; ++i) turn[i] = turn_of(s, p, FULL || p >= 0 ? pl.f[i] : -1);
                at.next(chunks);
                pos = at.u < units ? position(s, at.t) : -1;
                float sums[2 * HU];
#pragma unroll
                for (int h = 0; h < HU; ++h) {
                    sums[2 * h] = sums[2 * h + 1] = 0.f;
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const Pairs v = pairs<INTER>(ra[h][i], rb[h][i]);
                        const Pairs e = turned_back(pairs<INTER>(ga[h][i], gb[h][i]), turn[i], WHOLE, pl.f[i] >= 0);
                        const float vv = dot(v, v), ev = dot(times(e, wt[i]), v);
                        if (pl.on[i]) {
                            sums[2 * h] += vv;
                            sums[2 * h + 1] += ev;
                        }
                    }
                }
                if (s.norm) lanes_sum(sums, lanes);
#pragma unroll
                for (int h = 0; h < HU; ++h) {
                    // dx = r (t + k x); a padding token or a head past the last was not read and adds nothing
                    float r = 1.f, k = 0.f;
                    if (s.norm) {
                        r = rsqrtf(fmaf(sums[2 * h], inv, s.eps));
                        k = -sums[2 * h + 1] * inv * r * r;
                    }
                    if (!FULL && (p < 0 || h >= n)) r = k = 0.f;
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const Pairs v = pairs<INTER>(ra[h][i], rb[h][i]);
                        const Pairs e = times(turned_back(pairs<INTER>(ga[h][i], gb[h][i]), turn[i], WHOLE, pl.f[i] >= 0), r);
                        dw[i] = {fma4(e.a, v.a, dw[i].a), fma4(e.b, v.b, dw[i].b)};
                        Pairs d = e;
                        if (s.norm) {
                            const Quad kr = quad(k * r);
                            d = times(e, wt[i]);
                            d = {fma4(v.a, kr, d.a), fma4(v.b, kr, d.b)};
                        }
                        if (!FULL && p < 0) d = {quad(0.f), quad(0.f)};   // whatever the weights are
                        if ((FULL || h < n) && pl.on[i]) st_pairs<INTER>(y + h * s.hd + pl.a[i], y + h * s.hd + pl.b[i], d);
                    }
                }
            };
            if (!__all_sync(kFull, n == HU && p >= 0))
                body(std::false_type{}, std::false_type{});
            else if (all)
                body(std::true_type{}, std::true_type{});
            else
                body(std::true_type{}, std::false_type{});
        }
        if (s.part == nullptr) continue;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (pl.on[i]) st_pairs<INTER>(sm + group * s.hd + pl.a[i], sm + group * s.hd + pl.b[i], dw[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < s.hd; c += kThreads) {
            float v = 0.f;
            for (int k = 0; k < per; ++k) v += sm[k * s.hd + c];
            s.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * s.hd + c] = v;
        }
        __syncthreads();
    }
}

// The weight gradients: the blocks' rows summed in a fixed order. A block a column group of 32, its 32 rows of
// threads each a strided share of the partial rows.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int blocks, int hd, float* dwq, float* dwk) {
    __shared__ float sm[32][33];
    start_dependent();
    const int c = blockIdx.x * 32 + threadIdx.x;   // of 2 * hd columns
    float v = 0.f;
    if (c < 2 * hd)
        for (int k = threadIdx.y; k < blocks; k += 32) v += part[static_cast<int64_t>(k) * 2 * hd + c];
    sm[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = allsum(sm[threadIdx.x][threadIdx.y]);
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < 2 * hd) {
        float* const d = o < hd ? dwq : dwk;
        if (d != nullptr) d[o < hd ? o : o - hd] = v;
    }
}

struct TableArgs {
    uint64_t turns[kMaxFreq];   // a position's turn in units of 2^-64
    float* table;
    float scale;
    int n, max_pos;
};

// cos and sin of pos * f: the whole turns drop out of the 64-bit product exactly, whatever the position.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
    start_dependent();
    const int64_t i = blockIdx.x * int64_t(256) + threadIdx.x;
    if (i >= static_cast<int64_t>(a.n) * a.max_pos) return;
    const int64_t pos = i / a.n;
    const int f = static_cast<int>(i - pos * a.n);
    const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(pos) * a.turns[f]);   // [-1/2, 1/2) turns
    float s, c;
    sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);
    a.table[pos * 2 * a.n + f] = c * a.scale;
    a.table[pos * 2 * a.n + a.n + f] = s * a.scale;
}

// ---- host side ------------------------------------------------------------------------------------
using checks::aligned16;
using checks::aligned_all;

sdm_status check(const sdm_rope_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->dtype < 0 || s->dtype > 1) return SDM_ERR_DTYPE;
    if (s->tokens < 0 || s->tokens > (int64_t(1) << 31) || s->q_heads < 0 || s->k_heads < 0 || s->q_heads > 65536 ||
        s->k_heads > 65536 || s->q_heads + s->k_heads < 1 || s->hd < 1 || s->hd > kMaxHd || s->rot_dim < 0 ||
        s->rot_dim > s->hd || s->max_pos < 1 || s->layout < 0 || s->layout > 1 || s->norm < 0 || s->norm > 1 ||
        !(s->eps >= 0.f))
        return SDM_ERR_SHAPE;
    if (s->hd % 8 != 0 || s->rot_dim % 8 != 0) return SDM_ERR_ALIGN;
    if (s->tokens * (s->q_heads + s->k_heads) >= (int64_t(1) << 31) - (1 << 20)) return SDM_ERR_SHAPE;
    return SDM_OK;
}

sdm_status check_heads(const sdm_rope_shape* s, const void* p, int64_t ld, int heads, bool out) {
    if (heads == 0) return SDM_OK;
    if (p == nullptr) return SDM_ERR_ARG;
    const int e = s->dtype == SDM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(p) % (4 * e) != 0 || ld % 4 != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? static_cast<int64_t>(heads) * s->hd : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

void fill(const sdm_rope_shape* s, RopeArgs* a) {
    memset(a, 0, sizeof(*a));
    a->tokens = s->tokens;
    a->Hq = s->q_heads;
    a->Hk = s->k_heads;
    a->hd = s->hd;
    a->rd = s->rot_dim;
    a->max_pos = s->max_pos;
    a->interleaved = s->layout;
    a->norm = s->norm;
    a->eps = s->eps;
}

int head_lanes(int hd) {
    int lanes = 1;
    while (lanes < 32 && lanes * 8 < hd) lanes *= 2;
    return lanes;
}

int heads_together(const sdm_rope_shape* s) { return s->hd > 256 ? 1 : s->dtype == SDM_BF16 ? 4 : 2; }

int bwd_blocks(const sdm_rope_shape* s) {
    const int hu = heads_together(s);
    const int64_t units = s->tokens * ((std::max(s->q_heads, s->k_heads) + hu - 1) / hu), per = kThreads / head_lanes(s->hd);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kPartBlocks, (units + per - 1) / per)));
}

template <typename F>
cudaError_t by_type(const sdm_rope_shape* s, F f) {
    const int u = (s->hd / 8 + 31) / 32;
    auto units = [&](auto t, auto inter) {
        return u == 1 ? f(t, std::integral_constant<int, 1>{}, inter)
               : u == 2 ? f(t, std::integral_constant<int, 2>{}, inter) : f(t, std::integral_constant<int, 4>{}, inter);
    };
    auto with = [&](auto t) { return s->layout ? units(t, std::true_type{}) : units(t, std::false_type{}); };
    return s->dtype == SDM_BF16 ? with(__nv_bfloat16{}) : with(0.f);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_rope_workspace_bytes(const sdm_rope_shape* shape) {
    if (check(shape) != SDM_OK) return 0;
    return static_cast<size_t>(bwd_blocks(shape)) * 2 * shape->hd * sizeof(float);
}

extern "C" sdm_status sdm_rope_table(const sdm_rope_shape* shape, const double* inv_freq, float scale, float* table,
                                     sdm_stream_t stream) {
    const sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->rot_dim == 0) return SDM_OK;
    if (inv_freq == nullptr || table == nullptr) return SDM_ERR_ARG;
    if (!aligned16(table)) return SDM_ERR_ALIGN;
    TableArgs a;
    memset(&a, 0, sizeof(a));
    a.n = shape->rot_dim / 2;
    a.max_pos = shape->max_pos;
    a.scale = scale;
    a.table = table;
    for (int i = 0; i < a.n; ++i) {
        if (!std::isfinite(inv_freq[i])) return SDM_ERR_ARG;
        double turn = inv_freq[i] / 6.283185307179586476925;
        turn -= std::floor(turn);
        // two parts of 32 bits: a double holds either exactly
        const double hi = std::floor(std::ldexp(turn, 32));
        a.turns[i] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::ldexp(std::ldexp(turn, 32) - hi, 32));
    }
    const int64_t blocks = (static_cast<int64_t>(a.n) * a.max_pos + 255) / 256;
    if (blocks > 0x7FFFFFFF) return SDM_ERR_SHAPE;
    const cudaError_t e = launch_dependent(rope_table_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                           reinterpret_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_qk_norm_rope(const sdm_rope_shape* shape, const void* q, int64_t q_ld, const void* k,
                                       int64_t k_ld, const int32_t* positions, const float* table, const float* wq,
                                       const float* wk, void* q_out, int64_t qo_ld, void* k_out, int64_t ko_ld,
                                       uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->tokens == 0) return SDM_OK;
    if (positions == nullptr || (shape->rot_dim > 0 && table == nullptr)) return SDM_ERR_ARG;
    if ((st = check_heads(shape, q, q_ld, shape->q_heads, false)) != SDM_OK) return st;
    if ((st = check_heads(shape, k, k_ld, shape->k_heads, false)) != SDM_OK) return st;
    if ((st = check_heads(shape, q_out, qo_ld, shape->q_heads, true)) != SDM_OK) return st;
    if ((st = check_heads(shape, k_out, ko_ld, shape->k_heads, true)) != SDM_OK) return st;
    if (!aligned_all(16, {table, wq, wk}) || !aligned_all(4, {positions, status})) return SDM_ERR_ALIGN;
    RopeArgs a;
    fill(shape, &a);
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.pos = positions; a.table = table; a.wq = wq; a.wk = wk;
    a.qo = q_out; a.qo_ld = qo_ld; a.ko = k_out; a.ko_ld = ko_ld; a.status = status;
    const int lanes = head_lanes(shape->hd);
    const int hu = heads_together(shape);
    const int64_t units = shape->tokens * ((a.Hq + hu - 1) / hu + (a.Hk + hu - 1) / hu);
    const int64_t blocks = std::min<int64_t>((units * lanes + kThreads - 1) / kThreads, 152 * fwd_blocks(shape->dtype == SDM_BF16));
    const cudaError_t e = by_type(shape, [&](auto t, auto u, auto inter) {
        return launch_dependent(rope_fwd_kernel<decltype(t), decltype(u)::value, decltype(inter)::value>, dim3(static_cast<unsigned>(blocks)),
                                dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), a, lanes);
    });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_qk_norm_rope_backward(const sdm_rope_shape* shape, const void* dq_out, int64_t dqo_ld,
                                                const void* dk_out, int64_t dko_ld, const void* q, int64_t q_ld,
                                                const void* k, int64_t k_ld, const int32_t* positions,
                                                const float* table, const float* wq, const float* wk, void* dq,
                                                int64_t dq_ld, void* dk, int64_t dk_ld, float* dwq, float* dwk,
                                                void* ws, size_t ws_bytes, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->tokens > 0) {
        if (positions == nullptr || (shape->rot_dim > 0 && table == nullptr)) return SDM_ERR_ARG;
        if ((st = check_heads(shape, dq_out, dqo_ld, shape->q_heads, false)) != SDM_OK) return st;
        if ((st = check_heads(shape, dk_out, dko_ld, shape->k_heads, false)) != SDM_OK) return st;
        if ((st = check_heads(shape, q, q_ld, shape->q_heads, false)) != SDM_OK) return st;
        if ((st = check_heads(shape, k, k_ld, shape->k_heads, false)) != SDM_OK) return st;
        if ((st = check_heads(shape, dq, dq_ld, shape->q_heads, true)) != SDM_OK) return st;
        if ((st = check_heads(shape, dk, dk_ld, shape->k_heads, true)) != SDM_OK) return st;
    }
    if (!aligned_all(16, {table, wq, wk}) || !aligned_all(4, {positions, status, dwq, dwk})) return SDM_ERR_ALIGN;
    const bool sums = shape->norm && (dwq != nullptr || dwk != nullptr);
    if (sums && (ws == nullptr || !aligned16(ws) || ws_bytes < sdm_rope_workspace_bytes(shape))) return SDM_ERR_WORKSPACE;
    RopeArgs a;
    fill(shape, &a);
    a.dqo = dq_out; a.dqo_ld = dqo_ld; a.dko = dk_out; a.dko_ld = dko_ld;
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.pos = positions; a.table = table; a.wq = wq; a.wk = wk;
    a.qo = dq; a.qo_ld = dq_ld; a.ko = dk; a.ko_ld = dk_ld; a.status = status;
    a.part = sums ? static_cast<float*>(ws) : nullptr;
    const int lanes = head_lanes(shape->hd), blocks = bwd_blocks(shape);
    const size_t smem = static_cast<size_t>(kThreads / lanes) * shape->hd * sizeof(float);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = by_type(shape, [&](auto t, auto u, auto inter) {
        return launch_dependent(rope_bwd_kernel<decltype(t), decltype(u)::value, decltype(inter)::value>, dim3(static_cast<unsigned>(blocks)),
                                dim3(kThreads), smem, cs, a, lanes);
    });
    if (e == cudaSuccess && (dwq != nullptr || dwk != nullptr))   // without the norm the sum of no blocks' rows: 0
        e = launch_dependent(rope_dw_kernel, dim3(static_cast<unsigned>((2 * shape->hd + 31) / 32)), dim3(32, 32), 0, cs,
                             static_cast<const float*>(ws), sums ? blocks : 0, shape->hd, dwq, dwk);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
