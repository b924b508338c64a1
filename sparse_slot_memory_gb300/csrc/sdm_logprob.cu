// sdm_logprob.cu -- log probabilities of given tokens with entropy and top alternatives, and the gradient of the
// logits: sdm_token_logprobs / sdm_token_logprobs_backward (include/sdm.h).
//
// Mathematics. For a row x of V logits, z = scale x, lse = log sum exp z, p = exp(z - lse), H = lse - sum p z.
// One pass keeps, per thread, a reference M, s = sum 2^t and u = sum t 2^t with t = x scale log2(e) - M, moved to a
// new M when a larger logit comes; the threads' triples join the same way. log p(target) = (t_target - log2 s) ln 2,
// H = (log2 s - u / s) ln 2. Backward: dz_v = dlogp (1[v = target] - p_v) - dH p_v (log p_v + H).
//
// The top alternatives: the same pass leaves the largest logit of every cell (64 bytes or more of a thread's share) in the
// shared memory. The K-th largest of 32 of those bounds the K-th largest logit from below; the few cells that hold as
// large a logit are read again, a vector a lane, their logits wait in the shared memory and join their warp's list of the 32 largest
// (value, id) sorted, 32 at a time, and the warps' lists join by halves.
//
// A row is one block's, or where there are fewer rows than the SMs hold blocks, a cluster's: each block takes a part
// of the row and the first joins their triples and lists through its shared memory.
//
// Bound by HBM: a read forward, a read and a write backward. Measured on a GB300 (6.7 TB/s copy): 4096 x 65536 bfloat16,
// forward and backward 238 us (1.61 GB: 6.8 TB/s, the second read partly from the L2); 1000 x 50001 float32 forward 33 us
// without alternatives (6.1 TB/s), 38 with 5; 8000 x 12000 bfloat16 32 us without, 58 with 20: a row's end (bound, cells,
// sort) is not hidden wholly where the blocks of an SM reach it together. Eight rows of 131072 with 20
// alternatives: 7.3 us in clusters of 8 blocks, its latency (loads, two list sorts, cluster barriers). A backward whose rows
// all have |lse| of 1024 or more pays for the plain look in every block of a row: 512 x 131072 float32 2.9 ms, otherwise 78 us.
//
// A row whose largest logit lies under -1e30 / scale (everything masked, by -inf or by a type's lowest value) leaves
// s = 0, one whose largest x scale log2(e) is past float32's range leaves NaN, and an M of 2^28 or more is rounded too
// coarsely: such rows take a second, plain look, whose differences hold for any finite logits. So does the backward of a row whose lse is too large for float32 differences. lse
// past the range is the largest or lowest finite value, so that -inf tells the backward that the row has nothing left.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

// Threads of a block that has a row to itself: as few as still fill the SMs, because the fixed part of a row (bound, cells,
// sort) costs a few warps little more than many, and more blocks on an SM hide one another's. All blocks run at 1024
// threads an SM. Measured at bfloat16 rows with 20 alternatives (us, blocks of 256 / 128 / 64 threads):
//   8000 x 6000: 84 / 55 / 42    8000 x 12000: 103 / 65 / 58    2000 x 12000: 30 / 20 / 18    600 x 12000: 9.3 / 8.5 / 9.7
//   8000 x 32000: 142 / 113 / 113    1000 x 32000: 23 / 19 / 24    600 x 32000: 13 / 15 / 21    1000 x 128000: 56 / 53 / 74
//   1800 x 128000: 92 / 95 / 94 (74 / 82 / 74 without alternatives)
// Long rows lose with narrow blocks where a few of them are left at the end, each read by few threads, but not where all
// run at once, when 256 threads would leave those few. That is so from 609 rows on; the rule begins at 760, a middle of (256 /
// 128 threads) rows with alternatives or of float32, which gain before (620 rows: 40000 bfloat16 with 20 alternatives
// 21.3 / 18.6, 32003 float32 without 17.0 / 14.6, 64000 float32 with 20 45 / 38), and bfloat16 rows without alternatives, which
// lose (620 rows of 128000: 30.2 / 33.9; 760: 32.3 / 35.9; 900: 44.0 / 39.8). Behind 1216 rows 256 are left some again
// (1230 rows of 128000 with 20: 74.5 / 80.0). Very short rows are two batches of two warps.
// A block of a cluster has the fewest rows and the most threads (150 rows of 131072: 21.7 us with 256, 18.2 with 512; 8 rows:
// 8.3 and 7.9).
constexpr int kRowThreads = 256, kClusterThreads = 512, kMidThreads = 128, kShortThreads = 64;
constexpr int64_t kMidBytes = 65536, kShortBytes = 24576, kBriefBytes = 8192, kSms = 152;
constexpr int blocks_of(int threads) { return 1024 / threads; }   // on an SM, at 64 registers
constexpr int kBatch = 4;             // vectors of a thread in flight
constexpr int kMaxK = 32;
constexpr int kCells = 16;            // cells of a thread's share of a row
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kFloor = -1e35f;      // what a masked logit counts as in the sums: its term is 0 beside any M
constexpr float kStart = -1e30f;      // the first M
constexpr float kFarM = 0x1p28f;      // |M| from which its rounding, which every term's t carries, is more than 16
constexpr float kFarLse = 1024.f;     // |lse| from which float32 z - lse is too coarse
// Where the gradient cuts z, and z - lse of far rows: p is 0 there beside any |lse| below kFarLse, and the products of what
// is left with scale and d_entropy, which p multiplies, stay as small as those of the other logits (-inf times 0 is NaN).
constexpr float kGradFloor = -2 * kFarLse;

struct LpArgs {
    const void* logits;
    const int32_t* targets;
    float* logp;
    float* entropy;        // nullable
    float* lse;            // nullable
    float* top_vals;       // nullable [rows, K]
    int32_t* top_idx;      // nullable
    const float* lse_in;
    const float* ent_in;      // nullable without d_entropy
    const float* d_logp;
    const float* d_entropy;   // nullable
    void* dlogits;
    uint32_t* status;      // nullable
    int64_t rows, ld, d_ld;
    int V, K;
    float scale;
    float floor;           // backward: the logit at kGradFloor
    int cluster;           // blocks of a row
    bool in_place;         // backward: dlogits is logits
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
    return o;
}

// A float's place in the order of the reals as an unsigned number (0 is no value's); -0 is +0, NaN is above all.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float ex2(float t) {   // 2^t, to 2 ulp; below 2^-126 it is 0
    float o;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(t));
    return o;
}

template <typename T>
struct Vec;   // 16 bytes of logits
template <>
struct Vec<float> {
    static constexpr int n = 4;
    float4 v;
    __device__ __forceinline__ void ld(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void none() { v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ void get(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
    __device__ __forceinline__ float most() const { return max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)); }
    // the pair i, no element below `floor`
    __device__ __forceinline__ uint64_t pair(int i, float floor) const {
        return i ? pack2(max_nan(v.z, floor), max_nan(v.w, floor)) : pack2(max_nan(v.x, floor), max_nan(v.y, floor));
    }
    __device__ __forceinline__ static void st(float* p, const float (&o)[4]) { st4(p, o); }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    uint4 v;
    __device__ __forceinline__ void ld(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void none() { v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t o;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
        return o;
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(word(i) << 16);
            o[2 * i + 1] = __uint_as_float(word(i) & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ float most() const {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    __device__ __forceinline__ uint64_t pair(int i, float floor) const {
        const uint32_t f = __float_as_uint(floor) >> 16, w = max2(word(i), f << 16 | f);
        return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ __forceinline__ static void st(__nv_bfloat16* p, const float (&o)[8]) { st8(p, o); }
};

// The online sums of some of a row's logits, in units of log2.
struct Sums {
    float M, s, u;
    __device__ __forceinline__ void clear() {
        M = kStart;
        s = u = 0.f;
    }
    __device__ __forceinline__ void raise(float m) {
        const float d = M - m, f = ex2(d);   // d <= 0
        u = f * fmaf(d, s, u);
        s *= f;
        M = m;
    }
    __device__ __forceinline__ void add(float x, float c) {   // M is at least x c
        const float t = fmaf(max_nan(x, kFloor), c, -M), e = ex2(t);
        s += e;
        u = fmaf(e, t, u);
    }
    template <int VECS, typename T>
    __device__ __forceinline__ void add(const Vec<T> (&r)[VECS], float c) {
        const uint64_t c2 = pack2(c, c), m2 = pack2(-M, -M);
        uint64_t s2 = pack2(s, 0.f), u2 = pack2(u, 0.f);
#pragma unroll
        for (int k = 0; k < VECS; ++k)
#pragma unroll
            for (int i = 0; i < Vec<T>::n / 2; ++i) {
                const uint64_t t2 = fma2(r[k].pair(i, kFloor), c2, m2);
                float a, b;
                unpack2(t2, a, b);
                const uint64_t e2 = pack2(ex2(a), ex2(b));
                s2 = add2(s2, e2);
                u2 = fma2(e2, t2, u2);
            }
        float a, b;
        unpack2(s2, a, b);
        s = a + b;
        unpack2(u2, a, b);
        u = a + b;
    }
    __device__ __forceinline__ void join(float oM, float os, float ou) {
        const float m = fmaxf(M, oM), d = M - m, od = oM - m, f = ex2(d), of = ex2(od);
        u = f * fmaf(d, s, u) + of * fmaf(od, os, ou);
        s = f * s + of * os;
        M = m;
    }
};

// A warp's 32 largest (order, ~id) so far, the i-th in lane i, and up to 63 logits that wait to join them.
struct TopList {
    uint64_t key;
    uint64_t* wait;   // [64] in shared memory
    uint32_t* bound;  // the block's: K logits at least this large are known
    int K, lane, n;   // n wait
    uint32_t pass;    // a logit enters only if its order is at least this
    float thr;        // the same as a value: logits below it do not enter (NaN: none is below)
    uint32_t last;    // and one of that order only if its id is below this
    __device__ __forceinline__ void raise(uint32_t p) {
        if (p > pass) {
            pass = p;
            thr = value_of(p);
            last = 0xFFFFFFFFu;
        }
    }
    // whether logits of at most x with ids from `id` on may enter
    __device__ __forceinline__ bool enters(float x, int id) const {
        return !(x < thr) && !(static_cast<uint32_t>(id) >= last && order_of(x) == pass);
    }
    __device__ __forceinline__ void clear(int k, int l, uint64_t* w, uint32_t* b) {
        key = 0;
        wait = w;
        bound = b;
        K = k;
        lane = l;
        n = 0;
        pass = 0;
        thr = value_of(0);
        last = 0xFFFFFFFFu;
    }
    // A step of a sorting network: the lane pairs at distance d, the larger first where `down`
    __device__ __forceinline__ static void step(uint64_t& k, int d, bool down, int lane) {
        const uint64_t x = __shfl_xor_sync(kFull, k, d);
        k = (k > x) == (((lane & d) == 0) == down) ? k : x;
    }
    // The 32 largest of this list and another, both descending over the lanes: the larger of lane i's and the other's
    // lane 31 - i are those 32, and five exchanges bring them in order.
    __device__ __forceinline__ void join(uint64_t other) {
        const uint64_t o = __shfl_xor_sync(kFull, other, 31);
        key = key > o ? key : o;
#pragma unroll
        for (int d = 16; d; d >>= 1) step(key, d, true, lane);
    }
    __device__ __forceinline__ static void sort(uint64_t& c, int lane) {
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int d = size >> 1; d; d >>= 1) step(c, d, (lane & size) == 0, lane);
    }
    // The first 32 that wait are sorted and join the list.
    __device__ __forceinline__ void flush() {
        __syncwarp();
        uint64_t c = lane < n ? wait[lane] : 0;
        const uint64_t rest = lane + 32 < n ? wait[lane + 32] : 0;
        __syncwarp();
        wait[lane] = rest;
        n = max(0, n - 32);
        sort(c, lane);
        join(c);
        const uint64_t kth = __shfl_sync(kFull, key, K - 1);
        const uint32_t k = static_cast<uint32_t>(kth >> 32);
        if (k != 0) {
            raise(k);
            if (k == pass) last = min(last, ~static_cast<uint32_t>(kth));   // K logits of this warp go before the others
            if (lane == 0) atomicMax(bound, k);
        }
        __syncwarp();
    }
    // N logits of each lane, ids id .. id + N - 1 (a lane whose id lies at or past `end` has none)
    template <int N>
    __device__ __forceinline__ void offer(const float (&x)[N], float most, int id, int end) {
        const bool want = id < end && enters(most, id);
        if (!__any_sync(kFull, want)) return;
        uint32_t mine = 0;   // the lane's logits that enter
        if (want) {
#pragma unroll
            for (int i = 0; i < N; ++i) mine |= enters(x[i], id + i) ? 1u << i : 0u;
        }
        while (true) {   // one logit of each lane that has one left, room for 32 of them behind the 31 that may wait
            const uint32_t b = __ballot_sync(kFull, mine != 0);
            if (b == 0) break;
            if (mine != 0) {
                const int i = __ffs(mine) - 1;
                mine &= mine - 1;
                float v = x[0];
#pragma unroll
                for (int k = 1; k < N; ++k) v = i == k ? x[k] : v;
                wait[n + __popc(b & ((1u << lane) - 1u))] =
                    static_cast<uint64_t>(order_of(v)) << 32 | static_cast<uint32_t>(~(id + i));
            }
            n += __popc(b);
            if (n >= 32) flush();
        }
    }
};

template <int WARPS, int CLUSTER, bool TOP>
struct Shared {
    static_assert(kMaxK % WARPS == 0, "each warp gives its share of the 32 logits that bound the alternatives");
    float M[WARPS], s[WARPS], u[WARPS], red[WARPS];
    union {
        uint64_t top[WARPS][kMaxK];
        uint16_t hit[WARPS][kMaxK * 4];   // before the lists: cells of a warp's threads to be read again, 32 cell + lane
    };
    uint64_t wait[WARPS][64];
    uint32_t least[kMaxK], bound;
    int pooled;
    float cell[TOP ? kCells : 1][WARPS * 32];   // the largest logit of a thread's cell
    // of the cluster's blocks, in the first one
    float cM[CLUSTER], cs[CLUSTER], cu[CLUSTER];
    uint64_t ctop[CLUSTER][kMaxK];
};

// The lists in rows 0 .. n - 1 (n a power of two, one row a warp) joined into row 0. Block-wide.
__device__ __forceinline__ void join_lists(uint64_t (*top)[kMaxK], int n, int w, int lane) {
    for (int h = n >> 1; h; h >>= 1) {
        if (w < h) {
            TopList l;
            l.lane = lane;
            l.key = top[w][lane];
            l.join(top[w + h][lane]);
            top[w][lane] = l.key;
        }
        __syncthreads();
    }
}

// The row's largest logit, then sum exp(z - z_max), sum exp(z - z_max) (z - z_max), from differences that hold for
// any finite logits. Block-wide, with a float of shared memory for each warp; every thread gets them.
template <typename T>
__device__ void plain_stats(const T* x, int V, float scale, float* red, float& m, float& s, float& u) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    auto block = [&](float v, bool sum) {
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            const float o = __shfl_xor_sync(kFull, v, k);
            v = sum ? v + o : max_nan(v, o);
        }
        __syncthreads();
        if (lane == 0) red[w] = v;
        __syncthreads();
        v = red[0];
        for (int k = 1; k < static_cast<int>(blockDim.x) / 32; ++k) v = sum ? v + red[k] : max_nan(v, red[k]);
        return v;
    };
    float most = -INFINITY;
    for (int i = threadIdx.x; i < V; i += blockDim.x) most = max_nan(most, widen(x[i]));
    m = block(most, false);
    float a = 0.f, b = 0.f;
    for (int i = threadIdx.x; i < V; i += blockDim.x) {
        const float d = (widen(x[i]) - m) * scale, e = expf(d);
        a += e;
        b += e > 0.f ? e * d : e;   // NaN stays
    }
    s = block(a, true);
    u = block(b, true);
}

template <typename T, bool TOP, bool CLUSTER, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_of(THREADS)) lp_fwd_kernel(const LpArgs a) {
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    __shared__ Shared<kWarps, CLUSTER ? kMaxCluster : 1, TOP> sh;
    if (CLUSTER) cluster_arrive_relaxed();
    start_dependent();
    constexpr int N = Vec<T>::n;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int C = CLUSTER ? a.cluster : 1, rank = CLUSTER ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const T* const x = static_cast<const T*>(a.logits) + row * a.ld;
    const float c = a.scale * kLog2e;
    Sums acc;
    acc.clear();
    TopList top;
    top.clear(a.K, lane, sh.wait[w], &sh.bound);
    if (TOP) {
        if (threadIdx.x == 0) {
            sh.bound = 0;
            sh.pooled = 0;
        }
        __syncthreads();
    }
    // vectors start at the row's first 16-byte boundary; the logits before it and behind the last vector are
    // taken one by one, by the first and the last block. Ids come in no order: among equal logits the lower ids win by the keys'
    // order, and by TopList::last, the id from which on logits equal to the K-th cannot enter
    const int head = min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
    const int nvec = (a.V - head) / N;
    const int each = CLUSTER ? (nvec + C - 1) / C : nvec;
    const int vb = rank * each, ve = CLUSTER ? min(nvec, vb + each) : nvec;   // this block's vectors
    const T* const xv = x + head;
    // at most 32 logits, by warp 0: their sums, and as alternatives
    auto scalar = [&](int b, int e) { return b + lane < e ? widen(x[b + lane]) : -INFINITY; };
    auto sum_scalars = [&](int b, int e) {
        const float v = scalar(b, e);
        if (b + lane < e) {
            if (!(v * c <= acc.M)) acc.raise(v * c);
            acc.add(v, c);
        }
    };
    auto offer_scalars = [&](int b, int e) {
        const float v[1] = {scalar(b, e)};
        top.offer<1>(v, v[0], b + lane, e);
    };
    const int tail = head + nvec * N;
    if (w == 0 && rank == 0) sum_scalars(0, head);
    // a cell of a thread: its vectors of `per` batches
    const int batches = (max(ve - vb, 0) + kThreads * kBatch - 1) / (kThreads * kBatch), per = (batches + kCells - 1) / kCells;
    float cell = -INFINITY, most_of_all = -INFINITY;
    int cells = 0;
    for (int v0 = vb, in = 0; v0 < ve; v0 += kThreads * kBatch) {
        Vec<T> r[kBatch];
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = v0 + k * kThreads + threadIdx.x;
            if (v < ve)
                r[k].ld(xv + static_cast<int64_t>(v) * N);
            else
                r[k].none();
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) most = max_nan(most, r[k].most());
        if (!(most * c <= acc.M)) acc.raise(most * c);
        acc.add(r, c);
        if (TOP) {
            cell = max_nan(cell, most);
            if (++in == per || v0 + kThreads * kBatch >= ve) {   // block-uniform
                sh.cell[cells++][threadIdx.x] = cell;
                most_of_all = max_nan(most_of_all, cell);
                cell = -INFINITY;
                in = 0;
            }
        }
    }
    if (w == 0 && rank == C - 1) sum_scalars(tail, a.V);
    if (TOP) {
        // The K-th largest logit is at least the K-th largest of any 32 of them: of the largest ones that a thread of each
        // warp saw, the largest few. Only cells that hold as large a logit are read again.
        constexpr int kEach = kMaxK / kWarps;
        uint32_t o = order_of(most_of_all);
#pragma unroll
        for (int r = 0; r < kEach; ++r) {
            const uint32_t m = __reduce_max_sync(kFull, o);
            if (__ffs(__ballot_sync(kFull, o == m)) - 1 == lane) o = 0;
            if (lane == 0) sh.least[w * kEach + r] = m;
        }
        __syncthreads();
        o = sh.least[lane];
        uint32_t kth = 0;
        if (a.K <= kMaxK / 2) {   // taken away from the top, or from the bottom
            for (int r = 0; r < a.K; ++r) {
                kth = __reduce_max_sync(kFull, o);
                if (__ffs(__ballot_sync(kFull, o == kth)) - 1 == lane) o = 0;
            }
        } else {
            for (int r = kMaxK; r >= a.K; --r) {
                kth = __reduce_min_sync(kFull, o);
                if (__ffs(__ballot_sync(kFull, o == kth)) - 1 == lane) o = 0xFFFFFFFFu;
            }
        }
        top.raise(kth);
        if (w == 0 && rank == 0) offer_scalars(0, head);
        // A cell has `size` vectors; those of a warp's cells are read again one a lane, whoever's cell they are of: a
        // few rounds of full warps instead of one for every cell and vector (8000 x 12000 bfloat16, 20 alternatives: 75 us,
        // then 58; 1000 x 50001 float32 with 32: 58, then 46; rows whose logits all rise with the id lose:
        // the latter with 20 42, then 51, 4000 x 12000 bfloat16 41, then 61).
        const int size = per * kBatch;
        int hits = 0;
        for (int q = 0; q < cells; ++q) {
            top.raise(*static_cast<volatile uint32_t*>(&sh.bound));
            const float best = sh.cell[q][threadIdx.x];
            if (__any_sync(kFull, !(best < top.thr))) {
                const int v = min(vb + q * size * kThreads + static_cast<int>(threadIdx.x), ve);
                const bool want = top.enters(best, head + v * N);
                const uint32_t all = __ballot_sync(kFull, want);
                if (want) sh.hit[w][hits + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(q * 32 + lane);
                hits += __popc(all);
            }
            while (hits >= 32 || (hits > 0 && q == cells - 1)) {   // the first 32
                const int n = min(hits, 32) * size;
                __syncwarp();
                for (int j0 = 0; j0 < n; j0 += 32) {
                    const int j = j0 + lane, h = min(j, n - 1) / size, code = sh.hit[w][h], col = w * 32 + (code & 31);
                    const int v = vb + ((code >> 5) * size + j - h * size) * kThreads + col;
                    const bool mine = j < n && v < ve && !(sh.cell[code >> 5][col] < top.thr);
                    Vec<T> r;
                    if (mine)
                        r.ld(xv + static_cast<int64_t>(v) * N);
                    else
                        r.none();
                    float f[N];
                    r.get(f);
                    top.offer<N>(f, r.most(), mine ? head + v * N : a.V, tail);
                }
                const uint16_t rest = lane + 32 < hits ? sh.hit[w][lane + 32] : uint16_t(0);
                __syncwarp();
                if (lane + 32 < hits) sh.hit[w][lane] = rest;
                hits = max(0, hits - 32);
            }
        }
        if (w == 0 && rank == C - 1) offer_scalars(tail, a.V);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        const float M = __shfl_xor_sync(kFull, acc.M, k), s = __shfl_xor_sync(kFull, acc.s, k),
                    u = __shfl_xor_sync(kFull, acc.u, k);
        acc.join(M, s, u);
    }
    if (lane == 0) {
        sh.M[w] = acc.M;
        sh.s[w] = acc.s;
        sh.u[w] = acc.u;
    }
    if (TOP) {
        // what waits in all warps is at most a row of 32 for each: together, the rows sorted by a warp each and joined.
        // Where a warp has a list already, every warp completes its own.
        uint64_t* const pool = &sh.top[0][0];
        const bool lists = __syncthreads_or(__any_sync(kFull, top.key != 0)) != 0;
        if (lists) {
            while (top.n > 0) top.flush();
            sh.top[w][lane] = top.key;
            __syncthreads();
            join_lists(sh.top, kWarps, w, lane);
        } else {
            int at = 0;
            if (lane == 0) at = atomicAdd(&sh.pooled, top.n);
            at = __shfl_sync(kFull, at, 0);
            if (lane < top.n) pool[at + lane] = top.wait[lane];
            __syncthreads();
            const int n = sh.pooled;
            int rows = 1;
            while (rows * 32 < n) rows *= 2;
            if (w < rows) {
                uint64_t key = w * 32 + lane < n ? pool[w * 32 + lane] : 0;
                TopList::sort(key, lane);
                sh.top[w][lane] = key;
            }
            __syncthreads();
            join_lists(sh.top, rows, w, lane);
        }
    } else {
        __syncthreads();
    }
    acc.clear();
    for (int k = 0; k < kWarps; ++k) acc.join(sh.M[k], sh.s[k], sh.u[k]);
    if (CLUSTER) {
        cluster_wait();   // every block of the cluster runs
        if (w == 0) {
            if (lane == 0) {
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote_address(&sh.cM[rank], 0)), "f"(acc.M) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote_address(&sh.cs[rank], 0)), "f"(acc.s) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote_address(&sh.cu[rank], 0)), "f"(acc.u) : "memory");
            }
            if (TOP)
                asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(remote_address(&sh.ctop[rank][lane], 0)),
                             "l"(sh.top[0][lane]) : "memory");
        }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        acc.clear();
        for (int k = 0; k < C; ++k) acc.join(sh.cM[k], sh.cs[k], sh.cu[k]);
        if (TOP) join_lists(sh.ctop, C, w, lane);
    }
    // z - lse = (x - ref) mul - sub for the row's logits
    float ref = 0.f, sub, lse, H, mul = 0.f;
    bool empty = false;
    if (!(acc.s > 0.f && fabsf(acc.M) < kFarM)) {   // block-uniform
        float m, s, u;
        plain_stats(x, a.V, a.scale, sh.red, m, s, u);
        empty = m == -INFINITY;
        ref = m;
        mul = a.scale;
        sub = logf(s);
        const float top = fmaf(m, a.scale, sub);
        lse = empty ? -INFINITY : isinf(top) ? copysignf(FLT_MAX, top) : top;
        H = empty ? 0.f : sub - u / s;
    } else {
        const float l2 = log2f(acc.s);
        sub = l2;
        lse = (acc.M + l2) * kLn2;
        H = (l2 - acc.u / acc.s) * kLn2;
        if (H < 0.f) H = 0.f;   // by rounding, where one logit holds everything
    }
    auto logp_of = [&](float v) {
        if (empty) return -INFINITY;
        if (mul != 0.f) {
            const float d = v - ref;   // of finite logits infinite beside a large ref alone: then the products do not cancel
            return (isinf(d) && ref > 0.f ? v * mul - ref * mul : d * mul) - sub;
        }
        const float t = fmaf(v, c, -acc.M) - sub;
        if (t < kStart) return v * a.scale - lse;   // a masked logit's t may have overflowed
        return t > 0.f ? 0.f : t * kLn2;            // M and the logit's product round apart: never above 0
    };
    if (threadIdx.x == 0) {
        const int t = a.targets[row];
        if (t >= a.V && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_TARGET);
        a.logp[row] = t >= 0 && t < a.V ? logp_of(widen(x[t])) : 0.f;
        if (a.entropy != nullptr) a.entropy[row] = H;
        if (a.lse != nullptr) a.lse[row] = lse;
    }
    if (TOP && w == 0 && lane < a.K) {
        const uint64_t key = CLUSTER ? sh.ctop[0][lane] : sh.top[0][lane];
        if (a.top_vals != nullptr) a.top_vals[row * a.K + lane] = logp_of(value_of(static_cast<uint32_t>(key >> 32)));
        if (a.top_idx != nullptr) a.top_idx[row * a.K + lane] = static_cast<int32_t>(~static_cast<uint32_t>(key));
    }
}

constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 4;   // vectors of a thread

template <typename T>
__global__ void __launch_bounds__(kBwdThreads) lp_bwd_kernel(const LpArgs a, int parts) {
    __shared__ float red[kBwdThreads / 32];
    start_dependent();
    constexpr int N = Vec<T>::n;
    const int64_t row = blockIdx.x / parts;
    const int part = static_cast<int>(blockIdx.x - row * parts);
    const T* const x = static_cast<const T*>(a.logits) + row * a.ld;
    T* const o = static_cast<T*>(a.dlogits) + row * a.d_ld;
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    const int head = min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
    const int nvec = (a.V - head) / N;
    // this part's vectors, on their way while the row's scalars arrive
    const int v0 = part * kBwdThreads * kBwdVecs + threadIdx.x;
    Vec<T> r[kBwdVecs];
#pragma unroll
    for (int k = 0; k < kBwdVecs; ++k)
        if (v0 + k * kBwdThreads < nvec) r[k].ld(x + head + static_cast<int64_t>(v0 + k * kBwdThreads) * N);
    const int t = a.targets[row];
    const float dl = t >= 0 && t < a.V ? a.d_logp[row] : 0.f;
    const float dh = a.d_entropy != nullptr ? a.d_entropy[row] : 0.f;
    const float H = a.d_entropy != nullptr ? a.ent_in[row] : 0.f, lse = a.lse_in[row];
    if (part == 0 && threadIdx.x == 0 && t >= a.V && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_TARGET);
    if (fabsf(lse) >= kFarLse) {
        // block-uniform and rare: z - lse from differences to the largest logit, or (lse -inf) a row of zeros. In place
        // the first block writes the whole row, which every block would read.
        if (a.in_place && part != 0) return;
        const bool empty = lse == -INFINITY;
        float m = 0.f, s = 1.f, u;
        if (!empty) plain_stats(x, a.V, a.scale, red, m, s, u);
        const float ls = logf(s);
        const int per = kBwdThreads * kBwdVecs * N;
        const int end = a.in_place || part + 1 == parts ? a.V : min(a.V, (part + 1) * per);
        for (int i = part * per + threadIdx.x; i < end; i += kBwdThreads) {
            const float d = max_nan((widen(x[i]) - m) * a.scale - ls, kGradFloor), p = empty ? 0.f : expf(d);
            const float g = -p * (dl + dh * (empty ? 0.f : d + H)) + (i == t ? dl : 0.f);
            st1(o + i, a.scale * g);
        }
        return;
    }
    // dlogits = p (k1 d + k0) with d = log p, and scale dl more at the target
    const float k0 = -a.scale * (dl + dh * H), k1 = -a.scale * dh;
    auto grad = [&](float v, int id) {
        const float d = fmaf(max_nan(v, a.floor), a.scale, -lse);
        return ex2(d * kLog2e) * fmaf(d, k1, k0) + (id == t ? a.scale * dl : 0.f);
    };
    if (part == 0) {   // the logits outside the vectors
        const int tail = head + nvec * N, i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
        if (i < a.V) st1(o + i, grad(widen(x[i]), i));
    }
    const uint64_t sc2 = pack2(a.scale, a.scale), ls2 = pack2(-lse, -lse), le2 = pack2(kLog2e, kLog2e),
                   k02 = pack2(k0, k0), k12 = pack2(k1, k1);
#pragma unroll
    for (int k = 0; k < kBwdVecs; ++k) {
        const int v = v0 + k * kBwdThreads;
        if (v >= nvec) continue;
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint64_t d2 = fma2(r[k].pair(i, a.floor), sc2, ls2);
            float p, q;
            unpack2(mul2(d2, le2), p, q);
            unpack2(mul2(pack2(ex2(p), ex2(q)), fma2(d2, k12, k02)), f[2 * i], f[2 * i + 1]);
        }
        const int base = head + v * N, at = t - base;
        if (at >= 0 && at < N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i == at) f[i] += a.scale * dl;
        }
        if (same) {
            Vec<T>::st(o + base, f);
        } else {   // the gradient's row lies differently on 16 bytes
#pragma unroll
            for (int i = 0; i < N; ++i) st1(o + base + i, f[i]);
        }
    }
}

// ---- host side ------------------------------------------------------------------------------------
sdm_status check(const sdm_logprob_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->dtype < 0 || s->dtype > 1) return SDM_ERR_DTYPE;
    if (s->rows < 0 || s->rows > (int64_t(1) << 31) - 1 || s->V < 1 || s->V > (1 << 28) || s->K < 0 || s->K > kMaxK ||
        s->K > s->V || !(s->scale >= 1e-3f && s->scale <= 1e3f))
        return SDM_ERR_SHAPE;
    return SDM_OK;
}

sdm_status check_logits(const sdm_logprob_shape* s, const void* p, int64_t ld, bool out) {
    if (p == nullptr) return SDM_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(p) % (s->dtype == SDM_BF16 ? 2 : 4) != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? s->V : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

// Blocks of a row: as many as leave each at least a batch, while the rows alone leave SMs idle.
int cluster_of(const sdm_logprob_shape* s) {
    const int64_t batch = kClusterThreads * 16 / (s->dtype == SDM_BF16 ? 2 : 4);
    int c = 1;
    while (c < kMaxCluster && s->rows * c < kSms && s->V >= 2 * c * batch) c *= 2;
    return c;
}

// Threads of a block that has a row to itself.
int threads_of(const sdm_logprob_shape* s) {
    const int64_t bytes = static_cast<int64_t>(s->V) * (s->dtype == SDM_BF16 ? 2 : 4);
    if (bytes <= kBriefBytes || (bytes <= kShortBytes && s->rows >= 8 * kSms)) return kShortThreads;
    const bool once = s->rows >= 5 * kSms && s->rows <= 8 * kSms;   // all at once at eight blocks an SM, not at four
    return once || (bytes <= kMidBytes && s->rows >= 4 * kSms) ? kMidThreads : kRowThreads;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" sdm_status sdm_token_logprobs(const sdm_logprob_shape* shape, const void* logits, int64_t ld,
                                         const int32_t* targets, float* logp, float* entropy, float* lse,
                                         float* top_vals, int32_t* top_idx, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->rows == 0) return SDM_OK;
    if ((st = check_logits(shape, logits, ld, false)) != SDM_OK) return st;
    if (targets == nullptr || logp == nullptr) return SDM_ERR_ARG;
    if (!checks::aligned_all(4, {targets, logp, entropy, lse, top_vals, top_idx, status})) return SDM_ERR_ALIGN;
    LpArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = logits; a.ld = ld; a.targets = targets; a.logp = logp; a.entropy = entropy; a.lse = lse;
    a.top_vals = top_vals; a.top_idx = top_idx; a.status = status;
    a.rows = shape->rows; a.V = shape->V; a.K = shape->K; a.scale = shape->scale;
    const bool top = shape->K > 0 && (top_vals != nullptr || top_idx != nullptr);
    const bool bf = shape->dtype == SDM_BF16;
    a.cluster = cluster_of(shape);
    if (shape->rows * a.cluster > 0x7FFFFFFF) return SDM_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(shape->rows * a.cluster));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    auto run = [&](auto t, auto with_top) {
        using T = decltype(t);
        constexpr bool TOP = decltype(with_top)::value;
        if (a.cluster > 1)
            return launch_cluster(lp_fwd_kernel<T, TOP, true, kClusterThreads>, grid, dim3(kClusterThreads), a.cluster, cs, a);
        auto go = [&](auto threads) {
            constexpr int N = decltype(threads)::value;
            return launch_dependent(lp_fwd_kernel<T, TOP, false, N>, grid, dim3(N), 0, cs, a);
        };
        const int threads = threads_of(shape);
        if (threads == kShortThreads) return go(std::integral_constant<int, kShortThreads>{});
        if (threads == kMidThreads) return go(std::integral_constant<int, kMidThreads>{});
        return go(std::integral_constant<int, kRowThreads>{});
    };
    const std::true_type yes;
    const std::false_type no;
    const cudaError_t e = bf ? (top ? run(__nv_bfloat16{}, yes) : run(__nv_bfloat16{}, no)) : (top ? run(0.f, yes) : run(0.f, no));
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_token_logprobs_backward(const sdm_logprob_shape* shape, const void* logits, int64_t ld,
                                                  const int32_t* targets, const float* lse, const float* entropy,
                                                  const float* d_logp, const float* d_entropy, void* dlogits,
                                                  int64_t d_ld, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->rows == 0) return SDM_OK;
    if ((st = check_logits(shape, logits, ld, false)) != SDM_OK) return st;
    if ((st = check_logits(shape, dlogits, d_ld, true)) != SDM_OK) return st;
    if (targets == nullptr || lse == nullptr || (entropy == nullptr && d_entropy != nullptr) || d_logp == nullptr)
        return SDM_ERR_ARG;
    if (!checks::aligned_all(4, {targets, lse, entropy, d_logp, d_entropy, status})) return SDM_ERR_ALIGN;
    LpArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = logits; a.ld = ld; a.targets = targets; a.lse_in = lse; a.ent_in = entropy; a.d_logp = d_logp;
    a.d_entropy = d_entropy; a.dlogits = dlogits; a.d_ld = d_ld; a.status = status;
    a.rows = shape->rows; a.V = shape->V; a.scale = shape->scale; a.floor = kGradFloor / shape->scale;
    a.in_place = dlogits == logits;
    const bool bf = shape->dtype == SDM_BF16;
    const int per = kBwdThreads * kBwdVecs * (bf ? 8 : 4);
    const int parts = (shape->V + per - 1) / per;
    const int64_t blocks = shape->rows * parts;
    if (blocks > 0x7FFFFFFF) return SDM_ERR_SHAPE;
    const cudaError_t e = launch_dependent(bf ? lp_bwd_kernel<__nv_bfloat16> : lp_bwd_kernel<float>,
                                           dim3(static_cast<unsigned>(blocks)), dim3(kBwdThreads), 0,
                                           reinterpret_cast<cudaStream_t>(stream), a, parts);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
