// sdm_glr.cu -- the gated linear recurrence: forward, backward and the single-token step behind
// sdm_glr_forward / sdm_glr_backward / sdm_glr_step (include/sdm.h).
//
// Mathematics. h_t = a_t h_{t-1} + x_t with a_t = exp(g_t). A span of rows acts on the state as the pair
// (A, B): h_out = A h_in + B with A the product of its gates and B its result from a zero state; spans join as
// (A2 A1, A2 B1 + B2). The backward runs the same way from the end: with l_t the gradient of h_t and
// m_t = a_t l_t what flows to h_{t-1}, l_t = dy_t + m_{t+1}, dx_t = l_t, dg_t = m_t h_{t-1}. States, products
// and sums are float32.
//
// Layout. A block owns a tile of at most 128 channels (4 per lane; whole heads where gates are per head) of one
// sequence and walks it in steps of 64 rows: each of its 8 warps holds 8 consecutive rows in registers, forms their
// pair, the warps exchange pairs through shared memory and each then runs its rows again from its own starting state.
// The data are read once. Sequences long against the number of tiles are walked by clusters of 2, 4 or 8 blocks, whose
// pairs meet through each other's shared memory, one cluster barrier a step; and where even that leaves SMs idle they
// are cut into segments (`divide` has the rule): one kernel forms the segments' pairs, one chains them, and then every
// segment is walked on its own, the inputs read twice. The values between the three kernels lie in the first rows of
// the segments' own outputs, so no workspace is needed.
//
// The backward walks the steps from the end. It computes the states inside a step again from the saved state at its
// start, so it reads x instead of y: the same bytes, and no rounding of y in the gradients. A gate per head sums its
// channels' products over the lanes (and, for heads wider than a tile, over tiles in order in a second kernel).
//
// Bound by HBM in principle (6 bytes a bfloat16 element forward, 10 backward, 2 flops a byte); in fact by what the 16
// warps an SM that 128 registers allow wait for: the barriers of a step's exchange in the forward, loads and barriers in the
// backward (issue slots are used in 24 to 46 % of the cycles). One pass holds 8 rows, their gates and the next step's rows.
// Measured on a GB300 (6.7 TB/s copy): 8 x 8192 x 2048 with a gate per channel, bfloat16 rows and gates, forward 151 us
// (5.3 TB/s of its bytes), forward and backward 400 us (5.4 TB/s); with float32 gates 228 us (4.7 TB/s; 104 to 184 bytes of
// registers spilled a thread) and 533 us (5.5 TB/s); half the rows in float32 with float32 gates 123 us (6.5 TB/s) and
// 360 us (6.0 TB/s; the backward spills 152 to 204 bytes). 1 x 65537 x 512 float32 with gates per head, both, 178 us
// (671 MB of single reads: 3.8 TB/s; 940 MB moved); 24 ragged sequences, 30011 x 1920, forward 79 to 90 us by their lengths
// (2.6 to 2.9 TB/s). Heads that leave lanes of a tile idle, 8 x 4096 x 2040 to 2048 bfloat16, forward / both: 66 / 203 us at
// widths 64, 128 and 256, 127 / 325 at 96, 178 / 456 to 464 at 68 and 132. One token of 64 requests: 6.8 us a call (the
// kernel 1.6 in a graph), the host's time for it.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

constexpr int kTileCols = 128;   // channels of a tile
constexpr int kMaxCluster = 8;

// How a block divides its step of SDM_GLR_CHUNK rows: kRows rows to each of kWarps warps.
constexpr int kRows = 8, kWarps = SDM_GLR_CHUNK / kRows, kThreads = kWarps * 32;

struct GlrArgs {
    const void* x;
    const void* g;
    const void* dy;
    const int64_t* offsets;   // nullable: equal lengths
    const float* h0;          // nullable
    const float* dhT;         // nullable
    float* states;            // forward: nullable
    void* y;
    float* hT;                // nullable
    void* dx;
    void* dg;
    float* part;              // [tiles per head][rows][heads] gate gradients of a tile
    float* dh0;               // nullable
    uint32_t* status;         // nullable
    int64_t rows, len;        // len: rows of every sequence where offsets is null
    int64_t x_ld, g_ld, y_ld, dy_ld, dx_ld, dg_ld;
    int P, D, H, gw;
    int tiles, tile_cols, tiles_per_head;
    int cluster;              // blocks that walk a span together
    int64_t seg;              // rows of a segment (a multiple of SDM_GLR_CHUNK); 0: sequences are walked whole
};

// A tile's columns and this lane's place in it.
struct Tile {
    int col0, n;  // the tile's first channel and its channels
    int col;      // the lane's first channel
    bool on;      // whether the lane has channels
    bool full;    // whether every lane has
    int gate;     // the lane's gate (head)
    int seg;      // lanes from this one to the end of its head's part in the tile
    int sub;      // which of its head's tiles this is
    bool lead;    // the first lane of its head in the tile
};

template <bool PERCH>
__device__ __forceinline__ Tile tile_of(const GlrArgs& a, int tile, int lane) {
    Tile t;
    int c0, n;
    if (PERCH || a.tiles_per_head == 1) {
        c0 = tile * a.tile_cols;
        n = min(a.tile_cols, a.D - c0);
        t.sub = 0;
    } else {
        const int head = tile / a.tiles_per_head;
        t.sub = tile - head * a.tiles_per_head;
        c0 = head * a.gw + t.sub * a.tile_cols;
        n = min(a.tile_cols, (head + 1) * a.gw - c0);
    }
    t.col0 = c0;
    t.n = n;
    t.on = lane * 4 < n;
    t.full = n == kTileCols;
    t.col = c0 + (t.on ? lane * 4 : 0);
    if (PERCH) {
        t.gate = t.col;
        t.seg = 1;
        t.lead = false;
    } else {
        t.gate = t.col / a.gw;
        const int end = min(c0 + n, (t.gate + 1) * a.gw);
        t.seg = t.on ? (end - t.col) / 4 : 1;
        t.lead = t.on && (t.col == c0 || t.col % a.gw == 0);
    }
    return t;
}

// The rows [b, b + n) of sequence p. Offsets that are not ascending within [0, rows] are cut to it and reported.
__device__ __forceinline__ void sequence(const GlrArgs& a, int p, int64_t& b, int64_t& n) {
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

// A gate's exp is 2^(g log2 e): within 4 u + 1.25 |g| u (u = 2^-24; the product is rounded once, log2 e by 0.22 u), and
// exactly 0 and 1 at -inf and 0. The hardware's 2^t is low by 0.09 to 0.36 u on average for gates between 1 and 1/e, and a
// long memory adds that row by row. For float32 rows a fifth of u goes into the product's place, which leaves a mean within
// 0.16 u: 3000 rows with g about -0.05 (-0.0025) are within 1.3e-7 (4.6e-7) of 64 bits, without it 2.2e-7 (2.3e-6), float32
// rows one by one with expf 1.4e-7 (1.4e-6). bfloat16 rows are 2^-9 apart, and the registers for it would cost their training
// steps 1 to 3 %.
constexpr float kLog2e = 1.44269504088896341f, kCenter = 0.2f * 0x1p-24f * kLog2e;
__device__ __forceinline__ float exp2_gate(float t) {
    float o;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(t));
    return o;
}

// What a block (or cluster) walks: rows [b, b + n) of sequence p, segment k of `of`.
struct Part {
    int p, k, of;
    int64_t b, n;
    int64_t chunk;   // its first saved state
};

// Part number `id` of the launch. Without segments that is sequence id. With segments of L rows (the last of a sequence
// takes the rest, L to 2 L - 1 rows) sequence p's parts have the numbers from offsets[p] / L + p on; numbers between
// two sequences' name nothing (n < 0). Warp-wide; every block of a cluster finds the same.
__device__ __forceinline__ Part part_of(const GlrArgs& a, int id) {
    Part r;
    const int lane = threadIdx.x & 31;
    int64_t b, n;
    r.k = 0;
    r.of = 1;
    if (a.seg == 0) {
        r.p = id;
        if (a.offsets != nullptr && a.P <= 32 && a.P > 1) {
            // the longest sequences first: lane p counts those before sequence p
            const int64_t mine = lane < a.P ? a.offsets[lane + 1] - a.offsets[lane] : -1;
            int before = 0;
            for (int q = 0; q < a.P; ++q) {
                const int64_t other = __shfl_sync(kFull, mine, q);
                before += other > mine || (other == mine && q < lane);
            }
            r.p = __ffs(__ballot_sync(kFull, before == id && lane < a.P)) - 1;
        }
    } else if (a.offsets == nullptr) {
        r.of = static_cast<int>(max(a.len / a.seg, int64_t(1)));
        r.p = id / r.of;
        r.k = id - r.p * r.of;
    } else {
        // the last sequence whose first number is at most id: 32 probes a round
        int lo = 0, hi = a.P;   // in [lo, hi)
        while (hi - lo > 1) {
            const int w = (hi - lo + 31) / 32, q = lo + (lane + 1) * w;
            const bool le = q < hi && min(max(a.offsets[q], int64_t(0)), a.rows) / a.seg + q <= id;
            const int c = __popc(__ballot_sync(kFull, le));
            lo += c * w;
            hi = min(hi, lo + w);
        }
        r.p = lo;
    }
    if (r.p >= a.P) {
        r.n = -1;
        return r;
    }
    sequence(a, r.p, b, n);
    if (a.seg != 0) {
        if (a.offsets != nullptr) {
            r.of = static_cast<int>(max(n / a.seg, int64_t(1)));
            r.k = id - static_cast<int>(b / a.seg) - r.p;
        }
        if (r.k < 0 || r.k >= r.of) {
            r.n = -1;
            return r;
        }
    }
    r.chunk = b / SDM_GLR_CHUNK + r.p + r.k * (a.seg / SDM_GLR_CHUNK);
    r.b = b + r.k * a.seg;
    r.n = r.k + 1 < r.of ? a.seg : n - r.k * a.seg;
    return r;
}

// Between its passes a segmented walk keeps float32 values of a lane's columns in the first rows of the segment's own
// output, which the last pass overwrites: value i in the rows from i * 4 / sizeof(T) on.
template <typename T>
__device__ __forceinline__ void keep(T* row, int64_t ld, int i, const Quad& q) {
    if constexpr (sizeof(T) == 4) {
        st4(row + i * ld, q);
    } else {
        *reinterpret_cast<uint64_t*>(row + 2 * i * ld) = q.lo;
        *reinterpret_cast<uint64_t*>(row + (2 * i + 1) * ld) = q.hi;
    }
}
template <typename T>
__device__ __forceinline__ Quad kept(const T* row, int64_t ld, int i) {   // written by an earlier kernel
    if constexpr (sizeof(T) == 4) {
        float v[4];
        ld4cg(row + i * ld, v);
        return quad(v);
    } else {
        return {__ldcg(reinterpret_cast<const unsigned long long*>(row + 2 * i * ld)),
                __ldcg(reinterpret_cast<const unsigned long long*>(row + (2 * i + 1) * ld))};
    }
}

// The gates of one row as they lie in memory: the lane's four, or its head's one. CENTER: of float32 rows.
template <typename GT, bool PERCH, bool CENTER>
struct RawGate;
template <typename GT, bool CENTER>
struct RawGate<GT, true, CENTER> {
    Raw4<GT> v;
    __device__ __forceinline__ void zero() { v.zero(); }
    __device__ __forceinline__ Quad exps() const {
        float o[4];
        if constexpr (CENTER)
            floats(fma4(quad(v), quad(kLog2e), quad(kCenter)), o);
        else
            floats(mul4(quad(v), quad(kLog2e)), o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = exp2_gate(o[i]);
        return quad(o);
    }
};
template <typename GT, bool CENTER>
struct RawGate<GT, false, CENTER> {
    GT v;
    __device__ __forceinline__ void zero() { v = GT(0.f); }
    __device__ __forceinline__ Quad exps() const {
        return quad(exp2_gate(CENTER ? fmaf(widen(v), kLog2e, kCenter) : widen(v) * kLog2e));
    }
};

template <typename GT, bool CENTER>
__device__ __forceinline__ void ld_plain(RawGate<GT, true, CENTER>& r, const GT* p) { rows::ld_plain(r.v, p); }
template <typename GT, bool CENTER>
__device__ __forceinline__ void ld_plain(RawGate<GT, false, CENTER>& r, const GT* p) { r.v = *p; }

// kRows rows of a lane's columns; those from `live` on are zeros (the identity: gate 1, nothing added).
template <typename Row, typename T>
__device__ __forceinline__ void load_rows(Row (&r)[kRows], const T* p, int64_t ld, int live) {
    if (live == kRows) {   // warp-uniform
#pragma unroll
        for (int i = 0; i < kRows; ++i) ld_plain(r[i], p + i * ld);
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            r[i].zero();
            if (i < live) ld_plain(r[i], p + i * ld);
        }
    }
}

// Asks for a warp's rows of its next step in the L2, from the tile's first column p on: lane l its lines l, l + 32, ..
// of kRows rows of up to 128 columns.
template <typename T>
__device__ __forceinline__ void prefetch_rows(const T* p, int64_t ld, int live, int cols, int lane) {
    constexpr int kLines = kTileCols * sizeof(T) / 128;
#pragma unroll
    for (int k = 0; k < (kRows * kLines + 31) / 32; ++k) {
        const int l = lane + 32 * k, i = l / kLines, c = l % kLines * static_cast<int>(128 / sizeof(T));
        if (i < live && c < cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i * ld + c));
    }
}

// Hides from the compiler that loaded rows are unchanged: what was widened or raised from them before an exchange is
// computed again behind it, where keeping it would take twice the registers of the rows themselves.
__device__ __forceinline__ void forget(float& v) { asm volatile("" : "+f"(v)); }
__device__ __forceinline__ void forget(__nv_bfloat16& v) {
    uint16_t u = __bfloat16_as_ushort(v);
    asm volatile("" : "+h"(u));
    v = __ushort_as_bfloat16(u);
}
__device__ __forceinline__ void forget(Raw4<float>& r) {
    asm volatile("" : "+f"(r.v.x), "+f"(r.v.y), "+f"(r.v.z), "+f"(r.v.w));
}
__device__ __forceinline__ void forget(Raw4<__nv_bfloat16>& r) { asm volatile("" : "+r"(r.v.x), "+r"(r.v.y)); }
template <typename GT, bool PERCH, bool CENTER>
__device__ __forceinline__ void forget(RawGate<GT, PERCH, CENTER>& r) { forget(r.v); }
template <typename Row>
__device__ __forceinline__ void forget(Row (&r)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) forget(r[i]);
}

// How many of the kRows rows from t on lie before n.
__device__ __forceinline__ int live_rows(int64_t t, int64_t n) {
    return static_cast<int>(min(max(n - t, int64_t(0)), static_cast<int64_t>(kRows)));
}

// A store into the shared memory of another block of the cluster.
__device__ __forceinline__ void st_remote(const float* p, uint32_t rank, const Quad& q) {
    const uint32_t a = remote_address(p, rank);
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(a), "l"(q.lo), "l"(q.hi) : "memory");
}

// h = A h + B from a pair in shared memory
__device__ __forceinline__ void join(Quad& h, const float* A, const float* B) { h = fma4(quad_at(A), h, quad_at(B)); }

// One warp joins the block's warps' pairs and writes the block's pair into every block of the cluster, at its own rank.
template <bool REVERSE>
__device__ __forceinline__ void share_pair(const float (*A)[kTileCols], const float (*B)[kTileCols], float (*cA)[kTileCols],
                                           float (*cB)[kTileCols], uint32_t rank, int K, int lane) {
    Quad pa = quad(1.f), pb = quad(0.f);
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        const int k = REVERSE ? kWarps - 1 - j : j;
        const Quad ak = quad_at(&A[k][lane * 4]);
        pb = fma4(ak, pb, quad_at(&B[k][lane * 4]));
        pa = mul4(ak, pa);
    }
    for (int k = 0; k < K; ++k) {
        st_remote(&cA[rank][lane * 4], k, pa);
        st_remote(&cB[rank][lane * 4], k, pb);
    }
}

template <typename XT, typename GT, bool PERCH, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const GlrArgs a) {
    __shared__ __align__(16) float sA[2][kWarps][kTileCols], sB[2][kWarps][kTileCols];
    __shared__ __align__(16) float cA[2][CLUSTER ? kMaxCluster : 1][kTileCols], cB[2][CLUSTER ? kMaxCluster : 1][kTileCols];
    __shared__ __align__(16) float carry[2][kTileCols];
    if (CLUSTER) cluster_arrive_relaxed();
    start_dependent();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int K = CLUSTER ? a.cluster : 1, rank = CLUSTER ? cluster_rank() : 0;
    const int unit = blockIdx.x / K, id = unit / a.tiles;
    const Tile tl = tile_of<PERCH>(a, unit - id * a.tiles, lane);
    const Part part = part_of(a, id);
    if (part.n < 0) return;   // all of the cluster's blocks
    const int p = part.p;
    const int64_t b = part.b, n = part.n;
    Quad h = quad(0.f);   // the state before the step's rows
    if (part.of > 1)   // a segment's, its first one's too: h0 may be hT, which another block writes
        h = kept(static_cast<const XT*>(a.y) + b * a.y_ld + tl.col, a.y_ld, 2);
    else if (a.h0 != nullptr)
        h = quad(load4(a.h0 + static_cast<int64_t>(p) * a.D + tl.col));
    const int64_t step = static_cast<int64_t>(K) * SDM_GLR_CHUNK;
    int64_t t = rank * SDM_GLR_CHUNK + w * kRows;   // the warp's first row of the step
    const XT* x = static_cast<const XT*>(a.x) + (b + t) * a.x_ld;
    const GT* g = static_cast<const GT*>(a.g) + (b + t) * a.g_ld;
    XT* y = static_cast<XT*>(a.y) + (b + t) * a.y_ld + tl.col;
    float* const st = a.states == nullptr ? nullptr : a.states + part.chunk * a.D + tl.col;
    // bfloat16 rows: the next step's are loaded into registers over this one; float32 rows: asked for in the L2
    constexpr bool AHEAD = sizeof(XT) == 2;
    Raw4<XT> xr[kRows], xn[AHEAD ? kRows : 1];
    RawGate<GT, PERCH, sizeof(XT) == 4> gr[kRows], gn[AHEAD ? kRows : 1];
    int live = live_rows(t, n);
    if (AHEAD) {
        load_rows(gr, g + tl.gate, a.g_ld, live);
        load_rows(xr, x + tl.col, a.x_ld, live);
    }
    if (CLUSTER) cluster_wait();   // every block of the cluster runs
    int buf = 0;
    for (int64_t t0 = 0; t0 < n; t0 += step, t += step, buf ^= 1) {
        const int more = live_rows(t + step, n);
        if (!AHEAD) {
            load_rows(gr, g + tl.gate, a.g_ld, live);
            load_rows(xr, x + tl.col, a.x_ld, live);
        }
        x += step * a.x_ld;
        g += step * a.g_ld;
        if constexpr (AHEAD) {
            load_rows(gn, g + tl.gate, a.g_ld, more);
            load_rows(xn, x + tl.col, a.x_ld, more);
        } else {
            prefetch_rows(x + tl.col0, a.x_ld, more, tl.n, lane);
            if (PERCH) prefetch_rows(g + tl.col0, a.g_ld, more, tl.n, lane);
        }
        Quad A = quad(1.f), B = quad(0.f);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const Quad e = gr[i].exps();
            A = mul4(A, e);
            B = fma4(e, B, quad(xr[i]));
        }
        st4(&sA[buf][w][lane * 4], A);
        st4(&sB[buf][w][lane * 4], B);
        __syncthreads();   // the other buffer is written next: one barrier a step
        Quad hw = h;
        if (CLUSTER) {
            if (w == 0) {
                share_pair<false>(sA[buf], sB[buf], cA[buf], cB[buf], rank, K, lane);
                cluster_arrive();
            } else {
                cluster_arrive_relaxed();
            }
            cluster_wait();
#pragma unroll 1
            for (int k = 0; k < rank; ++k) join(h, &cA[buf][k][lane * 4], &cB[buf][k][lane * 4]);
            hw = h;
#pragma unroll 1
            for (int k = rank; k < K; ++k) join(h, &cA[buf][k][lane * 4], &cB[buf][k][lane * 4]);
            if (st != nullptr && w == 0 && tl.on && t < n) st4(st + t / SDM_GLR_CHUNK * a.D, hw);
        } else {
            // the state behind the step before: that step's last warp left it in the shared memory
            if (t0 > 0) hw = quad_at(&carry[buf][lane * 4]);
            if (st != nullptr && w == 0 && tl.on) st4(st + t0 / SDM_GLR_CHUNK * a.D, hw);
        }
#pragma unroll 1
        for (int j = 0; j < w; ++j) join(hw, &sA[buf][j][lane * 4], &sB[buf][j][lane * 4]);
        if (!CLUSTER && w == kWarps - 1) {
            h = hw;
            join(h, &sA[buf][w][lane * 4], &sB[buf][w][lane * 4]);
            st4(&carry[buf ^ 1][lane * 4], h);
        }
        if (AHEAD && PERCH) {
            forget(gr);
            forget(xr);
        }
        if (live == kRows) {
            if (tl.on) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    hw = fma4(gr[i].exps(), hw, quad(xr[i]));
                    st4(y + i * a.y_ld, hw);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                hw = fma4(gr[i].exps(), hw, quad(xr[i]));
                if (tl.on && i < live) st4(y + i * a.y_ld, hw);
            }
        }
        y += step * a.y_ld;
        live = more;
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                gr[i] = gn[i];
                xr[i] = xn[i];
            }
        }
    }
    // every thread of a cluster holds the state at the end; of a lone block, the last warp
    if (a.hT != nullptr && part.k + 1 == part.of && tl.on && (CLUSTER ? rank == 0 && w == 0 : w == kWarps - 1))
        st4(a.hT + static_cast<int64_t>(p) * a.D + tl.col, h);
}

// The sum of v over the lanes of its head in the tile, in the head's first lane.
__device__ __forceinline__ float head_sum(float v, int seg) {
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const float o = __shfl_down_sync(kFull, v, k);
        if (k < seg) v += o;   // lane + k lies in the same head
    }
    return v;
}

template <typename XT, typename GT, bool PERCH, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const GlrArgs a) {
    __shared__ __align__(16) float sA[2][kWarps][kTileCols], sF[2][kWarps][kTileCols], sR[2][kWarps][kTileCols];
    __shared__ __align__(16) float cA[2][CLUSTER ? kMaxCluster : 1][kTileCols], cR[2][CLUSTER ? kMaxCluster : 1][kTileCols];
    __shared__ __align__(16) float carry[2][kTileCols];
    if (CLUSTER) cluster_arrive_relaxed();
    start_dependent();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int K = CLUSTER ? a.cluster : 1, rank = CLUSTER ? cluster_rank() : 0;
    const int unit = blockIdx.x / K, id = unit / a.tiles;
    const Tile tl = tile_of<PERCH>(a, unit - id * a.tiles, lane);
    const Part part = part_of(a, id);
    if (part.n < 0) return;   // all of the cluster's blocks
    const int p = part.p;
    const int64_t b = part.b, n = part.n;
    Quad m = quad(0.f);   // the gradient of the state after the step's rows
    if (part.of > 1)
        m = kept(static_cast<const XT*>(a.dx) + b * a.dx_ld + tl.col, a.dx_ld, 2);
    else if (a.dhT != nullptr)
        m = quad(load4(a.dhT + static_cast<int64_t>(p) * a.D + tl.col));
    const float* const st = a.states + part.chunk * a.D + tl.col;
    const int64_t step = static_cast<int64_t>(K) * SDM_GLR_CHUNK;
    if (CLUSTER) cluster_wait();
    int buf = 0;
    bool first = true;
    for (int64_t t0 = (n + step - 1) / step * step - step; t0 >= 0; t0 -= step, buf ^= 1) {
        const int64_t tc = t0 + rank * SDM_GLR_CHUNK, t = tc + w * kRows;
        const int live = live_rows(t, n);
        const XT* const x = static_cast<const XT*>(a.x) + (b + t) * a.x_ld;
        const GT* const g = static_cast<const GT*>(a.g) + (b + t) * a.g_ld;
        const XT* const dy = static_cast<const XT*>(a.dy) + (b + t) * a.dy_ld;
        XT* const dx = static_cast<XT*>(a.dx) + (b + t) * a.dx_ld + tl.col;
        GT* const dg = static_cast<GT*>(a.dg) + (b + t) * a.dg_ld + tl.gate;
        Raw4<XT> xr[kRows], dr[kRows];
        RawGate<GT, PERCH, sizeof(XT) == 4> gr[kRows];
        load_rows(gr, g + tl.gate, a.g_ld, live);
        load_rows(dr, dy + tl.col, a.dy_ld, live);
        load_rows(xr, x + tl.col, a.x_ld, live);
        Quad h = quad(0.f);
        if (tc < n) h = quad(load4(st + tc / SDM_GLR_CHUNK * a.D));
        if (t0 > 0) {
            prefetch_rows(x - step * a.x_ld + tl.col0, a.x_ld, kRows, tl.n, lane);
            prefetch_rows(dy - step * a.dy_ld + tl.col0, a.dy_ld, kRows, tl.n, lane);
            if (PERCH) prefetch_rows(g - step * a.g_ld + tl.col0, a.g_ld, kRows, tl.n, lane);
        }
        Quad A = quad(1.f), F = quad(0.f), R = quad(0.f);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const Quad e = gr[i].exps();
            A = mul4(A, e);
            F = fma4(e, F, quad(xr[i]));
        }
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) R = mul4(gr[i].exps(), add4(quad(dr[i]), R));
        st4(&sA[buf][w][lane * 4], A);
        st4(&sF[buf][w][lane * 4], F);
        st4(&sR[buf][w][lane * 4], R);
        __syncthreads();
        Quad mw = m;
        if (CLUSTER) {
            if (w == 0) {
                share_pair<true>(sA[buf], sR[buf], cA[buf], cR[buf], rank, K, lane);
                cluster_arrive();
            } else {
                cluster_arrive_relaxed();
            }
#pragma unroll 1
            for (int j = 0; j < w; ++j) join(h, &sA[buf][j][lane * 4], &sF[buf][j][lane * 4]);
            cluster_wait();
#pragma unroll 1
            for (int k = K - 1; k > rank; --k) join(m, &cA[buf][k][lane * 4], &cR[buf][k][lane * 4]);
            mw = m;
#pragma unroll 1
            for (int k = rank; k >= 0; --k) join(m, &cA[buf][k][lane * 4], &cR[buf][k][lane * 4]);
        } else {
#pragma unroll 1
            for (int j = 0; j < w; ++j) join(h, &sA[buf][j][lane * 4], &sF[buf][j][lane * 4]);
            if (!first) mw = quad_at(&carry[buf][lane * 4]);
        }
#pragma unroll 1
        for (int j = kWarps - 1; j > w; --j) join(mw, &sA[buf][j][lane * 4], &sR[buf][j][lane * 4]);
        if (!CLUSTER && w == 0) {
            m = mw;
            join(m, &sA[buf][0][lane * 4], &sR[buf][0][lane * 4]);
            st4(&carry[buf ^ 1][lane * 4], m);
        }
        first = false;
        forget(gr);
        forget(xr);
        forget(dr);
        const bool all = live == kRows && tl.full;   // warp-uniform
        Quad hp[kRows];   // the state before each row
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            hp[i] = h;
            h = fma4(gr[i].exps(), h, quad(xr[i]));
        }
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            const Quad l = add4(quad(dr[i]), mw);
            mw = mul4(gr[i].exps(), l);
            const Quad q = mul4(mw, hp[i]);
            if (all || (tl.on && i < live)) st4(dx + i * a.dx_ld, l);
            if constexpr (PERCH) {
                if (all || (tl.on && i < live)) st4(dg + i * a.dg_ld, q);
            } else {
                float d[4];
                floats(q, d);
                const float s = head_sum(tl.on ? (d[0] + d[1]) + (d[2] + d[3]) : 0.f, tl.seg);
                if (tl.lead && i < live) {
                    if (a.tiles_per_head == 1)
                        st1(dg + i * a.dg_ld, s);
                    else
                        a.part[(tl.sub * a.rows + b + t + i) * a.H + tl.gate] = s;
                }
            }
        }
    }
    if (a.dh0 != nullptr && part.k == 0 && rank == 0 && w == 0 && tl.on)
        st4(a.dh0 + static_cast<int64_t>(p) * a.D + tl.col, m);
}

// The segments' pairs, kept in their outputs' first rows: forward (A, B) of all but a sequence's last segment,
// backward (A, R) of all but its first. A warp walks an eighth of the segment, and the first joins the eight.
template <typename XT, typename GT, bool PERCH, bool REVERSE>
__global__ void __launch_bounds__(256, 2) glr_pair_kernel(const GlrArgs a) {
    __shared__ __align__(16) float sA[8][kTileCols], sB[8][kTileCols];
    start_dependent();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int id = blockIdx.x / a.tiles;
    const Tile tl = tile_of<PERCH>(a, blockIdx.x - id * a.tiles, lane);
    const Part part = part_of(a, id);
    if (part.n < 0 || (REVERSE ? part.k == 0 : part.k + 1 == part.of)) return;   // block-uniform
    const int64_t each = (part.n + 63) / 64 * 8, t0 = w * each, n = min(each, part.n - t0);   // rows of the warp
    const XT* const v = static_cast<const XT*>(REVERSE ? a.dy : a.x) + (part.b + t0) * (REVERSE ? a.dy_ld : a.x_ld) + tl.col;
    const int64_t v_ld = REVERSE ? a.dy_ld : a.x_ld;
    const GT* const g = static_cast<const GT*>(a.g) + (part.b + t0) * a.g_ld + tl.gate;
    Quad A = quad(1.f), B = quad(0.f);
    for (int64_t i0 = 0; i0 < n; i0 += 8) {
        const int64_t t = REVERSE ? (n + 7) / 8 * 8 - 8 - i0 : i0;
        const int live = live_rows(t, n);
        Raw4<XT> xr[8];
        RawGate<GT, PERCH, sizeof(XT) == 4> gr[8];
        load_rows(gr, g + t * a.g_ld, a.g_ld, live);
        load_rows(xr, v + t * v_ld, v_ld, live);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = REVERSE ? 7 - j : j;
            const Quad e = gr[i].exps();
            A = mul4(A, e);
            B = REVERSE ? mul4(e, add4(quad(xr[i]), B)) : fma4(e, B, quad(xr[i]));
        }
    }
    st4(&sA[w][lane * 4], A);
    st4(&sB[w][lane * 4], B);
    __syncthreads();
    if (w != 0 || !tl.on) return;
    A = quad(1.f);
    B = quad(0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = REVERSE ? 7 - j : j;
        const Quad ak = quad_at(&sA[k][lane * 4]);
        B = fma4(ak, B, quad_at(&sB[k][lane * 4]));
        A = mul4(ak, A);
    }
    XT* const o = static_cast<XT*>(REVERSE ? a.dx : a.y) + part.b * (REVERSE ? a.dx_ld : a.y_ld) + tl.col;
    keep(o, REVERSE ? a.dx_ld : a.y_ld, 0, A);
    keep(o, REVERSE ? a.dx_ld : a.y_ld, 1, B);
}

// From the pairs, the state before (backward: the state's gradient behind) every segment, kept beside them. A block has
// 32 lanes of four channels of a sequence and kChain rows of threads that take a share of the segments each: they join
// their share's pairs, meet, and walk it again from their own start.
constexpr int kChain = 8;

template <typename XT, bool REVERSE>
__global__ void __launch_bounds__(32 * kChain) glr_chain_kernel(const GlrArgs a) {
    constexpr int kAhead = 8;   // pairs on their way at once
    __shared__ Quad sA[kChain][32], sB[kChain][32];
    start_dependent();
    const int quads = a.D / 4, blocks = (quads + 31) / 32, p = blockIdx.x / blocks;
    const int lane = threadIdx.x, share = threadIdx.y;
    const int q = min((blockIdx.x - p * blocks) * 32 + lane, quads - 1);
    const bool on = (blockIdx.x - p * blocks) * 32 + lane < quads;
    int64_t b, n;
    sequence(a, p, b, n);
    const int of = static_cast<int>(max(n / a.seg, int64_t(1)));
    if (of == 1) return;   // block-uniform
    const int64_t ld = REVERSE ? a.dx_ld : a.y_ld;
    const float* const first = REVERSE ? a.dhT : a.h0;
    XT* const o = static_cast<XT*>(REVERSE ? a.dx : a.y) + b * ld + q * 4;
    auto segment = [&](int i) { return o + (REVERSE ? of - 1 - i : i) * a.seg * ld; };   // i-th in the walk's order
    const int each = (of - 1 + kChain - 1) / kChain, from = share * each, to = min(of - 1, from + each);
    auto walk = [&](auto use) {
        for (int i0 = from; i0 < to; i0 += kAhead) {
            Quad A[kAhead], B[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i0 + i < to) {
                    A[i] = kept(segment(i0 + i), ld, 0);
                    B[i] = kept(segment(i0 + i), ld, 1);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (i0 + i < to) use(i0 + i, A[i], B[i]);
        }
    };
    Quad A = quad(1.f), B = quad(0.f);
    walk([&](int, const Quad& x, const Quad& y) {
        B = fma4(x, B, y);
        A = mul4(x, A);
    });
    sA[share][lane] = A;
    sB[share][lane] = B;
    __syncthreads();
    Quad h = quad(0.f);
    if (first != nullptr) h = quad(load4(first + static_cast<int64_t>(p) * a.D + q * 4));
    if (share == 0 && on) keep(segment(0), ld, 2, h);
    for (int k = 0; k < share; ++k) h = fma4(sA[k][lane], h, sB[k][lane]);
    walk([&](int i, const Quad& x, const Quad& y) {
        h = fma4(x, h, y);
        if (on) keep(segment(i + 1), ld, 2, h);
    });
}

// dg of a head wider than a tile: the sum of its tiles' parts, in tile order, of the rows from the first sequence's first to
// the last one's last. Rows of no sequence have no parts, and their dg stays as it is.
template <typename GT>
__global__ void __launch_bounds__(256) glr_dg_kernel(const GlrArgs a) {
    start_dependent();
    const int64_t n = a.rows * a.H;
    int64_t first = 0, end = a.rows;
    if (a.offsets != nullptr) {
        first = min(max(a.offsets[0], int64_t(0)), a.rows);
        end = min(a.offsets[a.P], a.rows);
    }
    for (int64_t i = first * a.H + blockIdx.x * int64_t(256) + threadIdx.x; i < end * a.H; i += gridDim.x * int64_t(256)) {
        float s = a.part[i];
        for (int k = 1; k < a.tiles_per_head; ++k) s += a.part[k * n + i];
        st1(static_cast<GT*>(a.dg) + i / a.H * a.dg_ld + i % a.H, s);
    }
}

struct StepArgs {
    const void* x;
    const void* g;
    const int32_t* slots;   // nullable: row i uses state i
    float* state;
    void* y;
    uint32_t* status;
    int64_t x_ld, g_ld, y_ld, s_ld;
    int64_t units;          // rows * (D / 4)
    int64_t states;
    int D, gw;
};

template <typename XT, typename GT, bool PERCH>
__global__ void __launch_bounds__(256) glr_step_kernel(const StepArgs a) {
    start_dependent();
    const int64_t u = blockIdx.x * int64_t(256) + threadIdx.x;
    if (u >= a.units) return;
    const int quads = a.D / 4;
    const int64_t r = u / quads;
    const int col = static_cast<int>(u - r * quads) * 4;
    const int64_t s = a.slots == nullptr ? r : static_cast<int64_t>(a.slots[r]);
    float h[4];
    Raw4<XT> x;
    XT* const y = static_cast<XT*>(a.y) + r * a.y_ld + col;
    if (s < 0 || s >= a.states) {   // a padding row, or an id that names no state
        if (s >= a.states && a.status != nullptr) atomicOr(a.status, kDevBadSlot);
        st4(y, quad(0.f));
        return;
    }
    float* const st = a.state + s * a.s_ld + col;
    ld4cg(st, h);
    ld_plain(x, static_cast<const XT*>(a.x) + r * a.x_ld + col);
    RawGate<GT, PERCH, sizeof(XT) == 4> gr;
    ld_plain(gr, static_cast<const GT*>(a.g) + r * a.g_ld + (PERCH ? col : col / a.gw));
    const Quad o = fma4(gr.exps(), quad(h), quad(x));
    st4(st, o);
    st4(y, o);
}

// ---- host side ------------------------------------------------------------------------------------
using checks::aligned16;
using checks::aligned_all;

int elem(int dtype) { return dtype == SDM_BF16 ? 2 : 4; }

sdm_status check(const sdm_glr_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->x_dtype < 0 || s->x_dtype > 1 || s->g_dtype < 0 || s->g_dtype > 1) return SDM_ERR_DTYPE;
    if (s->P < 1 || s->D < 1 || s->D > (1 << 20) || s->rows < 0 || s->rows > (int64_t(1) << 40) || s->gate_width < 1)
        return SDM_ERR_SHAPE;
    if (s->D % 4 != 0 || (s->gate_width != 1 && s->gate_width % 4 != 0)) return SDM_ERR_ALIGN;
    if (s->D % s->gate_width != 0) return SDM_ERR_SHAPE;
    return SDM_OK;
}

// A row array of `cols` columns: present, aligned to 4 elements (one where `vec` is false), its rows too.
sdm_status check_rows(const void* p, int64_t ld, int64_t cols, int dtype, bool vec, bool out) {
    if (p == nullptr) return SDM_ERR_ARG;
    const int v = vec ? 4 : 1;
    if (reinterpret_cast<uintptr_t>(p) % (v * elem(dtype)) != 0 || ld % v != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? cols : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

void geometry(const sdm_glr_shape* s, GlrArgs* a) {
    memset(a, 0, sizeof(*a));
    a->P = s->P;
    a->D = s->D;
    a->gw = s->gate_width;
    a->H = s->D / s->gate_width;
    a->rows = s->rows;
    a->len = s->rows / s->P;
    a->tiles_per_head = 1;
    if (s->gate_width == 1) {
        a->tile_cols = kTileCols;
        a->tiles = (s->D + kTileCols - 1) / kTileCols;
    } else if (s->gate_width <= kTileCols) {   // whole heads
        a->tile_cols = kTileCols / s->gate_width * s->gate_width;
        a->tiles = (s->D + a->tile_cols - 1) / a->tile_cols;
    } else {   // equal parts of a head, in multiples of 4 channels
        const int k = (s->gate_width + kTileCols - 1) / kTileCols;
        a->tile_cols = ((s->gate_width + k - 1) / k + 3) / 4 * 4;
        a->tiles_per_head = (s->gate_width + a->tile_cols - 1) / a->tile_cols;
        a->tiles = a->H * a->tiles_per_head;
    }
}

size_t part_bytes(const GlrArgs& a) {
    return a.tiles_per_head == 1 ? 0 : static_cast<size_t>(a.tiles_per_head) * a.rows * a.H * sizeof(float);
}

// How the rows are divided: by one block a part, or by clusters of 2, 4 or 8, whichever takes the fewest steps of 64 rows
// one after another on an SM's two blocks (152 SMs, kSlots blocks at once). Equal sequences: the waves of blocks times the
// steps of each. Unequal ones, whose lengths the host does not know: the larger of all steps over the slots and of the
// longest's steps, taken as four times the mean (24 sequences of 0 to 5526 rows, 30011 x 1920: 91 us with 1 block, 85
// with 4, 120 with 8; 8 x 8192 x 2048 bfloat16, forward and backward: 456 us with 1, 397 with 2, 444 with 4). Where even 8
// leave SMs idle and the sequences are long, they are cut into segments for two blocks an SM, at the price of reading
// the inputs twice (1 x 8192 x 1024: 97 us with clusters, 50 with segments; 1 x 4096 x 256: 48 and 47; 65537 x 512
// float32: 893 and 185), unequal ones four times earlier (8 sequences, 24000 x 256: 148 and 69).
//
// An output in place of an input (`in_place`) is not cut: the segments' pairs would lie over rows that are still to be
// read. Uncut, every row of a step is in registers before the step writes.
constexpr int64_t kSlots = 304, kBusy = 228, kSegmentRows = 256, kLong = 4096;

void divide(GlrArgs* a, bool in_place) {
    const int64_t units = static_cast<int64_t>(a->tiles) * a->P, steps = (a->len + SDM_GLR_CHUNK - 1) / SDM_GLR_CHUNK;
    const bool equal = a->offsets == nullptr || a->P == 1;
    a->cluster = 1;
    a->seg = 0;
    if (!in_place && units * kMaxCluster < kBusy && a->len * (equal ? 1 : 4) > kLong) {
        const int64_t cuts = kSlots / units;   // of a sequence
        a->seg = std::max(kSegmentRows, (a->len + cuts - 1) / cuts);
        a->seg = (a->seg + SDM_GLR_CHUNK - 1) / SDM_GLR_CHUNK * SDM_GLR_CHUNK;
        return;
    }
    auto cost = [&](int64_t k) {   // in steps
        if (equal) return static_cast<double>((units * k + kSlots - 1) / kSlots * ((steps + k - 1) / k));
        return std::max(static_cast<double>(units) * (steps + 0.5 * k) / kSlots, 4.0 * steps / k);
    };
    for (int k = 2; k <= kMaxCluster && k <= steps; k *= 2)
        if (cost(k) < cost(a->cluster)) a->cluster = k;
}

// Parts of the launch.
int64_t parts_of(const GlrArgs& a) {
    if (a.seg == 0) return a.P;
    return a.offsets == nullptr ? a.P * std::max<int64_t>(a.len / a.seg, 1) : a.rows / a.seg + a.P;
}

// Calls f(x type, g type, per-channel gates) with the shape's types.
template <typename F>
cudaError_t by_type(const sdm_glr_shape* s, F f) {
    const bool xb = s->x_dtype == SDM_BF16, gb = s->g_dtype == SDM_BF16, pc = s->gate_width == 1;
    auto with = [&](auto x, auto g) { return pc ? f(x, g, std::true_type{}) : f(x, g, std::false_type{}); };
    const __nv_bfloat16 b{};
    if (xb) return gb ? with(b, b) : with(b, 0.f);
    return gb ? with(0.f, b) : with(0.f, 0.f);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_glr_states_bytes(const sdm_glr_shape* shape) {
    if (check(shape) != SDM_OK) return 0;
    return static_cast<size_t>(shape->rows / SDM_GLR_CHUNK + shape->P) * shape->D * sizeof(float);
}

extern "C" size_t sdm_glr_workspace_bytes(const sdm_glr_shape* shape) {
    if (check(shape) != SDM_OK) return 0;
    GlrArgs a;
    geometry(shape, &a);
    return std::max<size_t>(part_bytes(a), 256);
}

extern "C" sdm_status sdm_glr_forward(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g,
                                      int64_t g_ld, const int64_t* offsets, const float* h0, void* y, int64_t y_ld,
                                      float* hT, float* states, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (offsets == nullptr && shape->rows % shape->P != 0) return SDM_ERR_SHAPE;
    const bool pc = shape->gate_width == 1;
    if (shape->rows > 0) {
        if ((st = check_rows(x, x_ld, shape->D, shape->x_dtype, true, false)) != SDM_OK) return st;
        if ((st = check_rows(g, g_ld, shape->D / shape->gate_width, shape->g_dtype, pc, false)) != SDM_OK) return st;
        if ((st = check_rows(y, y_ld, shape->D, shape->x_dtype, true, true)) != SDM_OK) return st;
    }
    if (!aligned_all(16, {h0, hT, states}) || !aligned_all(8, {offsets}) || !aligned_all(4, {status})) return SDM_ERR_ALIGN;
    GlrArgs a;
    geometry(shape, &a);
    if (static_cast<int64_t>(a.tiles) * (a.P + a.rows / SDM_GLR_CHUNK) > 0x7FFFFFFF / kMaxCluster) return SDM_ERR_SHAPE;
    a.x = x; a.x_ld = x_ld; a.g = g; a.g_ld = g_ld; a.y = y; a.y_ld = y_ld;
    a.offsets = offsets; a.h0 = h0; a.hT = hT; a.states = states; a.status = status;
    divide(&a, y == x || y == g);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(shape, [&](auto xt, auto gt, auto perch) {
        constexpr bool PC = decltype(perch)::value;
        const unsigned units = static_cast<unsigned>(a.tiles * parts_of(a));
        if (a.seg != 0) {
            using X = decltype(xt);
            cudaError_t e = launch_dependent(glr_pair_kernel<X, decltype(gt), PC, false>, dim3(units), dim3(256), 0, cs, a);
            if (e == cudaSuccess)
                e = launch_dependent(glr_chain_kernel<X, false>, dim3(static_cast<unsigned>(a.P) * ((a.D / 4 + 31) / 32)), dim3(32, kChain), 0,
                                     cs, a);
            if (e != cudaSuccess) return e;
        }
        const dim3 grid(units * a.cluster), block(kThreads);
        if (a.cluster > 1)
            return launch_cluster(glr_fwd_kernel<decltype(xt), decltype(gt), PC, true>, grid, block, a.cluster, cs, a);
        return launch_dependent(glr_fwd_kernel<decltype(xt), decltype(gt), PC, false>, grid, block, 0, cs, a);
    });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_glr_backward(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g,
                                       int64_t g_ld, const void* dy, int64_t dy_ld, const int64_t* offsets,
                                       const float* states, const float* dhT, void* dx, int64_t dx_ld, void* dg,
                                       int64_t dg_ld, float* dh0, void* ws, size_t ws_bytes, uint32_t* status,
                                       sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (offsets == nullptr && shape->rows % shape->P != 0) return SDM_ERR_SHAPE;
    const bool pc = shape->gate_width == 1;
    const int H = shape->D / shape->gate_width;
    if (shape->rows > 0) {
        if ((st = check_rows(x, x_ld, shape->D, shape->x_dtype, true, false)) != SDM_OK) return st;
        if ((st = check_rows(g, g_ld, H, shape->g_dtype, pc, false)) != SDM_OK) return st;
        if ((st = check_rows(dy, dy_ld, shape->D, shape->x_dtype, true, false)) != SDM_OK) return st;
        if ((st = check_rows(dx, dx_ld, shape->D, shape->x_dtype, true, true)) != SDM_OK) return st;
        if ((st = check_rows(dg, dg_ld, H, shape->g_dtype, pc, true)) != SDM_OK) return st;
        if (states == nullptr) return SDM_ERR_ARG;
    }
    if (!aligned_all(16, {states, dhT, dh0}) || !aligned_all(8, {offsets}) || !aligned_all(4, {status})) return SDM_ERR_ALIGN;
    GlrArgs a;
    geometry(shape, &a);
    if (static_cast<int64_t>(a.tiles) * (a.P + a.rows / SDM_GLR_CHUNK) > 0x7FFFFFFF / kMaxCluster) return SDM_ERR_SHAPE;
    if (part_bytes(a) > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < part_bytes(a))) return SDM_ERR_WORKSPACE;
    a.x = x; a.x_ld = x_ld; a.g = g; a.g_ld = g_ld; a.dy = dy; a.dy_ld = dy_ld;
    a.dx = dx; a.dx_ld = dx_ld; a.dg = dg; a.dg_ld = dg_ld;
    a.offsets = offsets; a.dhT = dhT; a.dh0 = dh0; a.states = const_cast<float*>(states); a.status = status;
    a.part = static_cast<float*>(ws);
    divide(&a, dx == x || dx == dy || dx == g);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = by_type(shape, [&](auto xt, auto gt, auto perch) {
        constexpr bool PC = decltype(perch)::value;
        const unsigned units = static_cast<unsigned>(a.tiles * parts_of(a));
        if (a.seg != 0) {
            using X = decltype(xt);
            cudaError_t e = launch_dependent(glr_pair_kernel<X, decltype(gt), PC, true>, dim3(units), dim3(256), 0, cs, a);
            if (e == cudaSuccess)
                e = launch_dependent(glr_chain_kernel<X, true>, dim3(static_cast<unsigned>(a.P) * ((a.D / 4 + 31) / 32)), dim3(32, kChain), 0,
                                     cs, a);
            if (e != cudaSuccess) return e;
        }
        const dim3 grid(units * a.cluster), block(kThreads);
        if (a.cluster > 1)
            return launch_cluster(glr_bwd_kernel<decltype(xt), decltype(gt), PC, true>, grid, block, a.cluster, cs, a);
        return launch_dependent(glr_bwd_kernel<decltype(xt), decltype(gt), PC, false>, grid, block, 0, cs, a);
    });
    if (e == cudaSuccess && part_bytes(a) > 0) {
        const int64_t blocks = std::min<int64_t>((a.rows * a.H + 255) / 256, 4096);
        e = launch_dependent(shape->g_dtype == SDM_BF16 ? glr_dg_kernel<__nv_bfloat16> : glr_dg_kernel<float>,
                             dim3(static_cast<unsigned>(blocks)), dim3(256), 0, cs, a);
    }
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_glr_step(const sdm_glr_shape* shape, const void* x, int64_t x_ld, const void* g, int64_t g_ld,
                                   const int32_t* slots, float* state, int64_t state_ld, int64_t states, void* y,
                                   int64_t y_ld, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (states < 0 || (slots == nullptr && states < shape->rows)) return SDM_ERR_SHAPE;
    if (shape->rows == 0) return SDM_OK;
    if (!aligned_all(4, {slots, status})) return SDM_ERR_ALIGN;
    if ((st = check_rows(x, x_ld, shape->D, shape->x_dtype, true, false)) != SDM_OK) return st;
    if ((st = check_rows(g, g_ld, shape->D / shape->gate_width, shape->g_dtype, shape->gate_width == 1, false)) != SDM_OK)
        return st;
    if ((st = check_rows(y, y_ld, shape->D, shape->x_dtype, true, true)) != SDM_OK) return st;
    if (states > 0 && (st = check_rows(state, state_ld, shape->D, SDM_F32, true, true)) != SDM_OK) return st;
    StepArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x; a.x_ld = x_ld; a.g = g; a.g_ld = g_ld; a.slots = slots; a.state = state; a.s_ld = state_ld;
    a.states = states; a.y = y; a.y_ld = y_ld; a.status = status;
    a.D = shape->D;
    a.gw = shape->gate_width;
    a.units = shape->rows * (shape->D / 4);
    const int64_t blocks = (a.units + 255) / 256;
    if (blocks > 0x7FFFFFFF) return SDM_ERR_SHAPE;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(shape, [&](auto xt, auto gt, auto perch) {
        return launch_dependent(glr_step_kernel<decltype(xt), decltype(gt), decltype(perch)::value>,
                                dim3(static_cast<unsigned>(blocks)), dim3(256), 0, cs, a);
    });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
