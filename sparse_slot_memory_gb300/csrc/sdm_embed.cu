// sdm_embed.cu -- the rows of an embedding table for tokens, scaled, and the table's gradient by sorted tokens:
// sdm_embed / sdm_embed_backward (include/sdm.h).
//
// The gradient's row v is scale times the sum of dy over the tokens with id v. The tokens are sorted by id, stably, by one
// cluster of 8 blocks (a radix sort of 10 bits a pass: histograms of contiguous parts, exchanged through the cluster's shared
// memory), which also lists the ids that there are and where their tokens begin and end; the other SMs write the table's zeros
// meanwhile, a kernel that starts with the sort and ends behind it. Then a warp adds the tokens of an id in their order, or of
// a part of 16 where an id has more, the frequent words; their parts' sums wait in the workspace and are joined in order by a
// last kernel. No sum depends on timing. Bound by HBM: the table's gradient is written once (float32, 131072 x 2048: 1.07 GB),
// the tokens' rows are read once. Measured: that step's 278 us of 238; the zeros alone run at 6.0 TB/s, the sort (38 us) beside them.
// The gradient alone of 16384, 32768, 65536, 131072 and 262144 tokens takes 209, 240, 295, 393 and 648 us of 168, 178, 198, 238 and 317.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

constexpr int kBits = 10, kDigits = 1 << kBits;   // of a pass
constexpr int kHeld = 4;        // rounds of a warp's tokens that stay in registers
constexpr int kSortBlocks = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSlice = 512;     // columns of a warp's unit: 16 a lane
constexpr int kPart = 16;       // tokens of an id that a warp adds
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct EmbedArgs {
    const int32_t* ids;
    const void* table;
    void* y;
    const void* dy;
    void* dtable;
    uint32_t* status;   // nullable
    int64_t tokens, t_ld, y_ld;
    int V, D, accumulate;
    float scale;
    // workspace of the backward
    int32_t* key[2];
    int32_t* tok[2];
    int2* range;        // [V]: where an id's tokens begin and end, of ids that there are
    int32_t* count;     // [2]: of work and joins
    int4* work;         // an id, or -1 - a part's number; where its tokens begin and end; the first token
    int4* joins;        // an id of several parts: id, first part, parts
    float* part;        // [tokens / 8][D]: their sums. Part p of an id whose tokens begin at b has the row b / 8 + p: an id of several parts
                        // has at least 17 tokens, so the rows of two ids never meet
    int passes;
};

// ---- forward ----------------------------------------------------------------------------------------------------------
// A warp takes a token's slice of kSlice columns, 16 a lane, and the next one's id ahead.
template <typename TT, typename T>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs a) {
    start_dependent();
    const int lane = threadIdx.x & 31, slices = (a.D + kSlice - 1) / kSlice;
    const int64_t units = a.tokens * slices, stride = gridDim.x * int64_t(8);
    int64_t u = blockIdx.x * int64_t(8) + (threadIdx.x >> 5), t = u / slices;
    int next = u < units ? a.ids[t] : 0;
    for (; u < units; u += stride) {
        const int id = next, c = static_cast<int>(u - t * slices) * kSlice + 4 * lane;
        const int64_t row = t;
        const bool real = id >= 0 && id < a.V;
        if (id >= a.V && lane == 0 && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_TOKEN);
        Raw4<TT> v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q].zero();
            if (real && c + 128 * q < a.D) ld_plain(v[q], static_cast<const TT*>(a.table) + id * a.t_ld + c + 128 * q);
        }
        if (u + stride < units) {
            t = (u + stride) / slices;
            next = a.ids[t];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (c + 128 * q < a.D)
                st4(static_cast<T*>(a.y) + row * a.y_ld + c + 128 * q, real ? mul4(quad(v[q]), quad(a.scale)) : quad(0.f));
    }
}

// The lanes whose digit (-1: none) is this lane's: a ballot for each bit.
__device__ __forceinline__ uint32_t same_digit(int d) {
    uint32_t m = __ballot_sync(kFull, d >= 0);
#pragma unroll
    for (int b = 0; b < kBits; ++b) {
        const uint32_t v = __ballot_sync(kFull, d >> b & 1);
        m &= d >> b & 1 ? v : ~v;
    }
    return d >= 0 ? m : 0u;
}

// ---- the sort -----------------------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ EmbedArgs a) {
    extern __shared__ int hist_of[];
    int (*const hist)[kDigits] = reinterpret_cast<int (*)[kDigits]>(hist_of);   // a warp's counts, then the places of the warps before it
    __shared__ int total[kDigits];          // of this block's part, which the cluster's other blocks read
    __shared__ int first[kDigits];
    __shared__ int carry[kSortWarps];
    static_assert(kDigits == kSortThreads, "a thread for each digit");
    start_dependent();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the zeros may start: what came before this sort is done
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rank = static_cast<int>(cluster_rank());
    const int n = static_cast<int>(a.tokens);
    // contiguous parts, so that their order is the tokens'
    const int64_t share = (static_cast<int64_t>(n) + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps);
    const int64_t lo = min((static_cast<int64_t>(rank) * kSortWarps + w) * share, int64_t(n)), hi = min(lo + share, int64_t(n));
    if (rank == 0 && tid < 2) a.count[tid] = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = kBits * pass;
        const int32_t* const kin = a.key[(pass + 1) & 1];
        const int32_t* const tin = a.tok[(pass + 1) & 1];
        int32_t* const kout = a.key[pass & 1];
        int32_t* const tout = a.tok[pass & 1];
        auto key_at = [&](int64_t i) {
            if (pass > 0) return __ldcg(kin + i);   // another block wrote it
            const int id = a.ids[i];
            if (id >= a.V && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_TOKEN);
            return id < 0 || id >= a.V ? a.V : id;   // padding sorts last
        };
        // a warp's tokens, 32 at a time; the first kHeld rounds' stay in registers for the second look
        auto round_of = [&](int64_t i, int (&k)[kHeld], int (&t)[kHeld]) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                const int64_t j = i + 32 * r;
                k[r] = j < hi ? key_at(j) : -1;
                t[r] = j < hi ? (pass > 0 ? __ldcg(tin + j) : static_cast<int>(j)) : 0;
            }
        };
        int k0[kHeld], t0[kHeld];
        round_of(lo + lane, k0, t0);
        for (int i = lane; i < kDigits; i += 32) hist[w][i] = 0;
        __syncwarp();
        auto count = [&](int64_t i, const int (&k)[kHeld]) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                if (i + 32 * r >= hi) break;
                const int d = k[r] >= 0 ? (k[r] >> shift) & (kDigits - 1) : -1;
                const uint32_t same = same_digit(d);
                if (d >= 0 && (same & ((1u << lane) - 1)) == 0) hist[w][d] += __popc(same);
                __syncwarp();
            }
        };
        count(lo, k0);
        for (int64_t i = lo + 32 * kHeld; i < hi; i += 32 * kHeld) {
            int k[kHeld], t[kHeld];
            round_of(i + lane, k, t);
            count(i, k);
        }
        __syncthreads();
        {
            int c[kSortWarps], sum = 0;
#pragma unroll
            for (int i = 0; i < kSortWarps; ++i) c[i] = hist[i][tid];
#pragma unroll
            for (int i = 0; i < kSortWarps; ++i) {
                hist[i][tid] = sum;
                sum += c[i];
            }
            total[tid] = sum;
        }
        cluster_arrive();
        cluster_wait();
        int all = 0, before = 0;
        {
            int c[kSortBlocks];
#pragma unroll
            for (int r = 0; r < kSortBlocks; ++r)
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[r]) : "r"(remote_address(&total[tid], r)) : "memory");
#pragma unroll
            for (int r = 0; r < kSortBlocks; ++r) {
                all += c[r];
                before += r < rank ? c[r] : 0;
            }
            int run = all;   // the digits' places: a scan over them
            for (int m = 1; m < 32; m *= 2) {
                const int o = __shfl_up_sync(kFull, run, m);
                if (lane >= m) run += o;
            }
            if (lane == 31) carry[w] = run;
            first[tid] = run - all + before;
        }
        __syncthreads();
        {
            int c = lane < w ? carry[lane] : 0;
#pragma unroll
            for (int m = 16; m > 0; m /= 2) c += __shfl_xor_sync(kFull, c, m);
            first[tid] += c;
        }
        __syncthreads();
        auto place = [&](int64_t i, const int (&k)[kHeld], const int (&t)[kHeld]) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                if (i + 32 * r >= hi) break;
                const int d = k[r] >= 0 ? (k[r] >> shift) & (kDigits - 1) : -1;
                const uint32_t same = same_digit(d);
                const int ahead = __popc(same & ((1u << lane) - 1));
                int at = 0;
                if (d >= 0) at = first[d] + hist[w][d] + ahead;
                __syncwarp();
                if (d >= 0 && ahead == 0) hist[w][d] += __popc(same);
                __syncwarp();
                if (d >= 0) {
                    kout[at] = k[r];
                    tout[at] = t[r];
                }
            }
        };
        place(lo, k0, t0);
        for (int64_t i = lo + 32 * kHeld; i < hi; i += 32 * kHeld) {
            int k[kHeld], t[kHeld];
            round_of(i + lane, k, t);
            place(i, k, t);
        }
        // the next pass reads what the cluster wrote, and writes the totals that it read
        cluster_arrive();
        cluster_wait();
    }
    const int32_t* const key = a.key[(a.passes + 1) & 1];
    const int32_t* const tok = a.tok[(a.passes + 1) & 1];
    for (int64_t i = rank * int64_t(kSortThreads) + tid; i < n; i += kSortBlocks * kSortThreads) {
        const int k = __ldcg(key + i);
        if (k >= a.V) continue;
        if (i == 0 || __ldcg(key + i - 1) != k) a.range[k].x = static_cast<int>(i);
        if (i + 1 == n || __ldcg(key + i + 1) != k) a.range[k].y = static_cast<int>(i) + 1;
    }
    cluster_arrive();
    cluster_wait();
    for (int64_t i = rank * int64_t(kSortThreads) + tid; i - lane < n; i += kSortBlocks * kSortThreads) {
        const int k = i < n ? __ldcg(key + i) : a.V, at = static_cast<int>(i);
        const int2 r = k < a.V ? __ldcg(a.range + k) : make_int2(0, 0);
        const bool several = r.y - r.x > kPart;
        // the lists' order is whatever it is; a warp takes its places together
        const bool starts = k < a.V && (several ? (at - r.x) % kPart == 0 : at == r.x), joins = starts && several && at == r.x;
        const uint32_t ms = __ballot_sync(kFull, starts), mj = __ballot_sync(kFull, joins), before = (1u << lane) - 1;
        int ws = 0, wj = 0;
        if (lane == 0 && ms != 0) ws = atomicAdd(a.count, __popc(ms));
        if (lane == 0 && mj != 0) wj = atomicAdd(a.count + 1, __popc(mj));
        ws = __shfl_sync(kFull, ws, 0) + __popc(ms & before);
        wj = __shfl_sync(kFull, wj, 0) + __popc(mj & before);
        if (starts) a.work[ws] = make_int4(several ? -1 - (r.x / 8 + (at - r.x) / kPart) : k, at, several ? min(at + kPart, r.y) : r.y, __ldcg(tok + i));
        if (joins) a.joins[wj] = make_int4(k, r.x / 8, (r.y - r.x + kPart - 1) / kPart, 0);
    }
}

// ---- the zeros --------------------------------------------------------------------------------------------------------------
// Rows of zeros, 16 bytes a store where rows lie without gaps. It starts with the sort and waits for its end before its own, so that
// what follows has both behind it.
template <typename TT>
__global__ void __launch_bounds__(256) embed_zero_kernel(const __grid_constant__ EmbedArgs a) {
    const int64_t stride = gridDim.x * int64_t(256), i0 = blockIdx.x * int64_t(256) + threadIdx.x;
    const Quad none = quad(0.f);
    if (a.t_ld == a.D && sizeof(TT) == 2 && reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0) {
        const int64_t n = static_cast<int64_t>(a.V) * a.D / 8;
        for (int64_t i = i0; i < n; i += stride) static_cast<uint4*>(a.dtable)[i] = make_uint4(0, 0, 0, 0);
        if (i0 == 0)
            for (int64_t i = n * 8; i < static_cast<int64_t>(a.V) * a.D; i += 4) st4(static_cast<TT*>(a.dtable) + i, none);
    } else if (a.t_ld == a.D) {
        const int64_t n = static_cast<int64_t>(a.V) * a.D / 4;
        for (int64_t i = i0; i < n; i += stride) st4(static_cast<TT*>(a.dtable) + 4 * i, none);
    } else {
        const int64_t per = a.D / 4, n = a.V * per;
        for (int64_t i = i0; i < n; i += stride) st4(static_cast<TT*>(a.dtable) + i / per * a.t_ld + i % per * 4, none);
    }
    start_dependent();
}

// ---- the sums ------------------------------------------------------------------------------------------------------------
// acc += dy of the tokens tok[b .. e), in order, at a lane's columns c + 128 q for q below n; F tokens on their way at once. The first
// token is known.
template <typename T, int Q, int F>
__device__ __forceinline__ void add_tokens(const EmbedArgs& a, const int32_t* tok, int first, int b, int e, int c, int n, Quad (&acc)[Q]) {
    for (int i = b; i < e; i += F) {
        Raw4<T> v[F][Q];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int64_t t = i + f >= e ? -1 : i + f == b ? first : tok[i + f];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                v[f][q].zero();
                if (t >= 0 && q < n) ld_plain(v[f][q], static_cast<const T*>(a.dy) + t * a.y_ld + c + 128 * q);
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int q = 0; q < Q; ++q) acc[q] = add4(acc[q], quad(v[f][q]));
    }
}

// The sums, scaled, to row v: n of a lane's four places of 4 columns lie in it.
template <typename TT, int Q>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int v, int c, int n, const Quad (&acc)[Q]) {
    TT* const out = static_cast<TT*>(a.dtable) + v * a.t_ld + c;
    const Quad s = quad(a.scale);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (q >= n) continue;
        Quad x = mul4(acc[q], s);
        if (a.accumulate) {
            Raw4<TT> old;
            ld_plain(old, out + 128 * q);
            x = fma4(acc[q], s, quad(old));
        }
        st4(out + 128 * q, x);
    }
}

template <typename TT, typename T>
__global__ void __launch_bounds__(kThreads, 4) embed_bwd_kernel(const __grid_constant__ EmbedArgs a) {
    start_dependent();
    constexpr int F = sizeof(T) == 2 ? 4 : 2;   // tokens of 512 columns on their way: what 64 registers hold but for 80 bytes a thread, which bfloat16 rows spill
    const int lane = threadIdx.x & 31, slices = (a.D + kSlice - 1) / kSlice;
    const int32_t* const tok = a.tok[(a.passes + 1) & 1];
    const int64_t units = static_cast<int64_t>(a.count[0]) * slices, stride = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t u = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5);
    int4 next = u < units ? a.work[u / slices] : make_int4(0, 0, 0, 0);   // known ahead
    for (; u < units; u += stride) {
        const int4 r = next;
        const int c = static_cast<int>(u % slices) * kSlice + 4 * lane, n = max(0, min(4, (a.D - c + 127) / 128));
        if (u + stride < units) next = a.work[(u + stride) / slices];
        Quad acc[4] = {};
        add_tokens<T, 4, F>(a, tok, r.w, r.y, r.z, c, n, acc);
        if (r.x >= 0) {
            put_row<TT>(a, r.x, c, n, acc);
        } else {
            float* const out = a.part + static_cast<int64_t>(-1 - r.x) * a.D + c;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < n) st4(out + 128 * q, acc[q]);
        }
    }
}

// An id's parts: a block's warps add contiguous shares of them, those are joined in order.
template <typename TT>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ EmbedArgs a) {
    __shared__ __align__(16) float sum[kWarps][kSlice];
    start_dependent();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, slices = (a.D + kSlice - 1) / kSlice;
    const int64_t units = static_cast<int64_t>(a.count[1]) * slices;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int4 r = a.joins[u / slices];
        const int c = static_cast<int>(u % slices) * kSlice + 4 * lane, n = max(0, min(4, (a.D - c + 127) / 128));
        const int share = (r.z + kWarps - 1) / kWarps, b = min(w * share, r.z), e = min(b + share, r.z);
        Quad acc[4] = {};
#pragma unroll 4
        for (int i = b; i < e; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < n) acc[q] = add4(acc[q], quad(load4(a.part + (static_cast<int64_t>(r.y) + i) * a.D + c + 128 * q)));
#pragma unroll
        for (int q = 0; q < 4; ++q) st4(&sum[w][4 * lane + 128 * q], acc[q]);
        __syncthreads();
        if (w == 0) {
            for (int i = 1; i < kWarps; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = add4(acc[q], quad_at(&sum[i][4 * lane + 128 * q]));
            put_row<TT>(a, r.x, c, n, acc);
        }
        __syncthreads();
    }
}

// ---- host side ------------------------------------------------------------------------------------
using checks::aligned16;
using checks::aligned_all;

sdm_status check(const sdm_embed_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->table_dtype < 0 || s->table_dtype > 1 || s->dtype < 0 || s->dtype > 1) return SDM_ERR_DTYPE;
    if (s->tokens < 0 || s->tokens >= (int64_t(1) << 31) - (1 << 20) || s->V < 1 || s->V > (1 << 28) || s->D < 1 || s->D > (1 << 20) ||
        !(s->scale == s->scale))
        return SDM_ERR_SHAPE;
    if (s->D % 4 != 0) return SDM_ERR_ALIGN;
    return SDM_OK;
}

sdm_status check_rows(const void* p, int64_t ld, int D, int dtype, bool out) {
    if (p == nullptr) return SDM_ERR_ARG;
    const int e = dtype == SDM_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(p) % (4 * e) != 0 || ld % 4 != 0) return SDM_ERR_ALIGN;
    if (ld < (out ? D : 0) || ld > (int64_t(1) << 40)) return SDM_ERR_ARG;
    return SDM_OK;
}

void fill(const sdm_embed_shape* s, EmbedArgs* a) {
    memset(a, 0, sizeof(*a));
    a->tokens = s->tokens;
    a->V = s->V;
    a->D = s->D;
    a->scale = s->scale;
    a->passes = 1;
    while (s->V >> (kBits * a->passes) != 0) ++a->passes;   // keys 0 .. V
}

int64_t up(int64_t n) { return (n + 255) / 256 * 256; }
// ids of several parts at most, and the rows of their parts
int64_t joins_of(int64_t tokens) { return tokens / (kPart + 1); }
int64_t parts_of(int64_t tokens) { return joins_of(tokens) > 0 ? tokens / 8 + 1 : 0; }

template <typename F>
cudaError_t by_type(const sdm_embed_shape* s, F f) {
    auto with = [&](auto tt) { return s->dtype == SDM_BF16 ? f(tt, __nv_bfloat16{}) : f(tt, 0.f); };
    return s->table_dtype == SDM_BF16 ? with(__nv_bfloat16{}) : with(0.f);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_embed_workspace_bytes(const sdm_embed_shape* shape) {
    if (check(shape) != SDM_OK) return 0;
    const int64_t T = shape->tokens, V = shape->V;
    return static_cast<size_t>(4 * up(4 * T) + up(8 * V) + 256 + up(16 * (std::min(T, V) + parts_of(T))) + up(16 * joins_of(T)) +
                               up(4 * parts_of(T) * shape->D));
}

extern "C" sdm_status sdm_embed(const sdm_embed_shape* shape, const int32_t* ids, const void* table, int64_t table_ld, void* y,
                                int64_t y_ld, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (shape->tokens == 0) return SDM_OK;
    if (ids == nullptr) return SDM_ERR_ARG;
    if ((st = check_rows(table, table_ld, shape->D, shape->table_dtype, false)) != SDM_OK) return st;
    if ((st = check_rows(y, y_ld, shape->D, shape->dtype, true)) != SDM_OK) return st;
    if (!aligned_all(4, {ids, status})) return SDM_ERR_ALIGN;
    EmbedArgs a;
    fill(shape, &a);
    a.ids = ids; a.table = table; a.t_ld = table_ld; a.y = y; a.y_ld = y_ld; a.status = status;
    const int64_t units = shape->tokens * ((shape->D + kSlice - 1) / kSlice);
    const int64_t blocks = std::min<int64_t>((units + 7) / 8, 152 * 8);
    const cudaError_t e = by_type(shape, [&](auto tt, auto t) {
        return launch_dependent(embed_kernel<decltype(tt), decltype(t)>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                reinterpret_cast<cudaStream_t>(stream), a);
    });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_embed_backward(const sdm_embed_shape* shape, const int32_t* ids, const void* dy, int64_t dy_ld, void* dtable,
                                         int64_t dtable_ld, int32_t accumulate, void* ws, size_t ws_bytes, uint32_t* status,
                                         sdm_stream_t stream) {
    sdm_status st = check(shape);
    if (st != SDM_OK) return st;
    if (accumulate < 0 || accumulate > 1) return SDM_ERR_ARG;
    if (shape->tokens > 0) {
        if (ids == nullptr) return SDM_ERR_ARG;
        if ((st = check_rows(dy, dy_ld, shape->D, shape->dtype, false)) != SDM_OK) return st;
    }
    if ((st = check_rows(dtable, dtable_ld, shape->D, shape->table_dtype, true)) != SDM_OK) return st;
    if (!aligned_all(4, {ids, status})) return SDM_ERR_ALIGN;
    if (ws == nullptr || !aligned16(ws) || ws_bytes < sdm_embed_workspace_bytes(shape)) return SDM_ERR_WORKSPACE;
    EmbedArgs a;
    fill(shape, &a);
    a.ids = ids; a.dy = dy; a.y_ld = dy_ld; a.dtable = dtable; a.t_ld = dtable_ld; a.accumulate = accumulate; a.status = status;
    unsigned char* w = static_cast<unsigned char*>(ws);
    for (int i = 0; i < 2; ++i) {
        a.key[i] = reinterpret_cast<int32_t*>(w);
        w += up(4 * shape->tokens);
        a.tok[i] = reinterpret_cast<int32_t*>(w);
        w += up(4 * shape->tokens);
    }
    a.range = reinterpret_cast<int2*>(w);
    w += up(8 * static_cast<int64_t>(shape->V));
    a.count = reinterpret_cast<int32_t*>(w);
    w += 256;
    a.work = reinterpret_cast<int4*>(w);
    w += up(16 * (std::min<int64_t>(shape->tokens, shape->V) + parts_of(shape->tokens)));
    a.joins = reinterpret_cast<int4*>(w);
    w += up(16 * joins_of(shape->tokens));
    a.part = reinterpret_cast<float*>(w);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    constexpr int smem = kSortWarps * kDigits * static_cast<int>(sizeof(int));
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_cluster_smem(embed_sort_kernel, dim3(kSortBlocks), dim3(kSortThreads), kSortBlocks, smem, cs, a);
    if (e == cudaSuccess && !accumulate) {
        const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(shape->V) * (shape->D / 4) + 1023) / 1024, 144 * 8);
        e = launch_dependent(shape->table_dtype == SDM_BF16 ? embed_zero_kernel<__nv_bfloat16> : embed_zero_kernel<float>,
                             dim3(static_cast<unsigned>(blocks)), dim3(256), 0, cs, a);
    }
    const int64_t slices = (shape->D + kSlice - 1) / kSlice;
    const int64_t blocks = std::min<int64_t>((shape->tokens * slices + kWarps - 1) / kWarps, 152 * 4);
    if (e == cudaSuccess && shape->tokens > 0)
        e = by_type(shape, [&](auto tt, auto t) {
            return launch_dependent(embed_bwd_kernel<decltype(tt), decltype(t)>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, cs, a);
        });
    if (e == cudaSuccess && joins_of(shape->tokens) > 0)
        e = launch_dependent(shape->table_dtype == SDM_BF16 ? embed_join_kernel<__nv_bfloat16> : embed_join_kernel<float>,
                             dim3(static_cast<unsigned>(std::min<int64_t>(joins_of(shape->tokens) * slices, 152 * 4))), dim3(kThreads), 0, cs, a);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
