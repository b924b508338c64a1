// sdm_embed.cu -- the rows of an embedding table for tokens, scaled, and the table's gradient by sorted tokens:
// sdm_embed / sdm_embed_backward (include/sdm.h).
//
// The gradient's row v is scale times the sum of dy over the tokens with id v. The tokens are sorted by id first, stably, by one
// cluster of 8 blocks (a radix sort of 8 bits a pass: histograms of contiguous parts, exchanged through the cluster's shared
// memory), which also notes where every id's tokens begin and end. Then every row has one writer that adds its tokens in order:
// no sum depends on timing. Rows with many tokens, the frequent words, are a block's: its warps take contiguous shares of the
// tokens, joined in order, and come first, so that the many rows of zeros hide them. Bound by HBM: the table's gradient is
// written once (float32, 131072 x 2048: 1.07 GB), the tokens' rows are read once.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "sdm_operators.cuh"

namespace sdm {
namespace {

using namespace rows;

constexpr int kHeld = 4;        // rounds of a warp's tokens that stay in registers
constexpr int kSortBlocks = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSlice = 512;     // columns of a warp's unit: 16 a lane
constexpr int kMany = 64;       // tokens from which a row is a block's
constexpr int kThreads = 512, kWarps = kThreads / 32;

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
    int2* range;        // [V]: where an id's tokens begin and end
    int32_t* many;      // [0] their number, then the ids with more than kMany tokens
    int passes;
};

// ---- forward ----------------------------------------------------------------------------------------------------------
// A thread takes 4 columns of up to 4 rows' places: independent loads in flight.
template <typename TT, typename T>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs a, int64_t units, int per) {
    start_dependent();
    const int64_t stride = gridDim.x * int64_t(256);
    for (int64_t base = blockIdx.x * int64_t(256) + threadIdx.x; base < units; base += 4 * stride) {
        Raw4<TT> v[4];
        int id[4];
        int64_t row[4];
        int c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t u = base + i * stride;
            row[i] = u < units ? u / per : -1;
            c[i] = static_cast<int>(u - row[i] * per) * 4;
            id[i] = row[i] >= 0 ? a.ids[row[i]] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i].zero();
            if (id[i] >= 0 && id[i] < a.V) ld_plain(v[i], static_cast<const TT*>(a.table) + id[i] * a.t_ld + c[i]);
            else if (id[i] >= a.V && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_TOKEN);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (row[i] < 0) continue;
            float x[4];
            v[i].get(x);
            const bool real = id[i] >= 0 && id[i] < a.V;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = real ? x[e] * a.scale : 0.f;
            st4(static_cast<T*>(a.y) + row[i] * a.y_ld + c[i], x);
        }
    }
}

// ---- the sort -----------------------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ EmbedArgs a) {
    __shared__ int hist[kSortWarps][256];   // a warp's counts, then the places of the warps before it
    __shared__ int total[256];              // of this block's part, which the cluster's other blocks read
    __shared__ int first[256];
    __shared__ int carry[8];
    start_dependent();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rank = static_cast<int>(cluster_rank());
    const int n = static_cast<int>(a.tokens);
    // contiguous parts, so that their order is the tokens'
    const int64_t share = (static_cast<int64_t>(n) + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps);
    const int64_t lo = min((static_cast<int64_t>(rank) * kSortWarps + w) * share, int64_t(n)), hi = min(lo + share, int64_t(n));
    for (int64_t i = rank * int64_t(kSortThreads) + tid; i < a.V; i += kSortBlocks * kSortThreads) a.range[i] = make_int2(0, 0);
    if (rank == 0 && tid == 0) a.many[0] = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass;
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
        for (int i = lane; i < 256; i += 32) hist[w][i] = 0;
        __syncwarp();
        auto count = [&](const int (&k)[kHeld]) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                const int d = k[r] >= 0 ? (k[r] >> shift) & 255 : 256;
                const uint32_t same = __match_any_sync(kFull, d);
                if (d < 256 && (same & ((1u << lane) - 1)) == 0) hist[w][d] += __popc(same);
                __syncwarp();
            }
        };
        count(k0);
        for (int64_t i = lo + 32 * kHeld; i < hi; i += 32 * kHeld) {
            int k[kHeld], t[kHeld];
            round_of(i + lane, k, t);
            count(k);
        }
        __syncthreads();
        if (tid < 256) {
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
        if (tid < 256) {
            int c[kSortBlocks];
#pragma unroll
            for (int r = 0; r < kSortBlocks; ++r)
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[r]) : "r"(remote_address(&total[tid], r)) : "memory");
#pragma unroll
            for (int r = 0; r < kSortBlocks; ++r) {
                all += c[r];
                before += r < rank ? c[r] : 0;
            }
            int run = all;   // the digits' places: a scan over 256
            for (int m = 1; m < 32; m *= 2) {
                const int o = __shfl_up_sync(kFull, run, m);
                if (lane >= m) run += o;
            }
            if (lane == 31) carry[w] = run;
            first[tid] = run - all + before;
        }
        __syncthreads();
        if (tid < 256) {
            int c = 0;
            for (int i = 0; i < w; ++i) c += carry[i];
            first[tid] += c;
        }
        __syncthreads();
        auto place = [&](const int (&k)[kHeld], const int (&t)[kHeld]) {
#pragma unroll
            for (int r = 0; r < kHeld; ++r) {
                const int d = k[r] >= 0 ? (k[r] >> shift) & 255 : 256;
                const uint32_t same = __match_any_sync(kFull, d);
                const int ahead = __popc(same & ((1u << lane) - 1));
                int at = 0;
                if (d < 256) at = first[d] + hist[w][d] + ahead;
                __syncwarp();
                if (d < 256 && ahead == 0) hist[w][d] += __popc(same);
                __syncwarp();
                if (d < 256) {
                    kout[at] = k[r];
                    tout[at] = t[r];
                }
            }
        };
        place(k0, t0);
        for (int64_t i = lo + 32 * kHeld; i < hi; i += 32 * kHeld) {
            int k[kHeld], t[kHeld];
            round_of(i + lane, k, t);
            place(k, t);
        }
        // the next pass reads what the cluster wrote, and writes the totals that it read
        cluster_arrive();
        cluster_wait();
    }
    const int32_t* const key = a.key[(a.passes + 1) & 1];
    for (int64_t i = rank * int64_t(kSortThreads) + tid; i < n; i += kSortBlocks * kSortThreads) {
        const int k = __ldcg(key + i);
        if (k >= a.V) continue;
        if (i == 0 || __ldcg(key + i - 1) != k) a.range[k].x = static_cast<int>(i);
        if (i + 1 == n || __ldcg(key + i + 1) != k) a.range[k].y = static_cast<int>(i) + 1;
    }
    cluster_arrive();
    cluster_wait();
    for (int64_t i = rank * int64_t(kSortThreads) + tid; i < n; i += kSortBlocks * kSortThreads) {
        const int k = __ldcg(key + i);
        if (k >= a.V || !(i == 0 || __ldcg(key + i - 1) != k)) continue;
        if (__ldcg(&a.range[k].y) - static_cast<int>(i) > kMany) a.many[1 + atomicAdd(a.many, 1)] = k;   // in whatever order
    }
}

// ---- the sums ------------------------------------------------------------------------------------------------------------
// acc += dy of the tokens tok[b .. e), in order, at a lane's columns c0 + 4 lane + 128 i
template <typename T>
__device__ __forceinline__ void add_tokens(const EmbedArgs& a, const int32_t* tok, int b, int e, int c, int n, Quad (&acc)[4]) {
    constexpr int kFlight = 4;
    for (int i = b; i < e; i += kFlight) {
        Raw4<T> v[kFlight][4];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t t = i + f < e ? tok[i + f] : -1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[f][q].zero();
                if (t >= 0 && q < n) ld_plain(v[f][q], static_cast<const T*>(a.dy) + t * a.y_ld + c + 128 * q);
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = add4(acc[q], quad(v[f][q]));
    }
}

// The sums, scaled, to row v: n of a lane's four places of 4 columns lie in it.
template <typename TT>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int v, int c, int n, const Quad (&acc)[4]) {
    TT* const out = static_cast<TT*>(a.dtable) + v * a.t_ld + c;
    const Quad s = quad(a.scale);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
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
__global__ void __launch_bounds__(kThreads, 2) embed_bwd_kernel(const __grid_constant__ EmbedArgs a) {
    __shared__ __align__(16) float part[kWarps][kSlice];
    start_dependent();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int slices = (a.D + kSlice - 1) / kSlice;
    const int32_t* const tok = a.tok[(a.passes + 1) & 1];
    auto places = [&](int c0) { return max(0, min(4, (a.D - c0 - 4 * lane + 127) / 128)); };
    const int64_t many = static_cast<int64_t>(a.many[0]) * slices;
    for (int64_t u = blockIdx.x; u < many; u += gridDim.x) {
        const int v = a.many[1 + u / slices], c0 = static_cast<int>(u % slices) * kSlice, c = c0 + 4 * lane, n = places(c0);
        const int2 r = a.range[v];
        const int share = (r.y - r.x + kWarps - 1) / kWarps, b = min(r.x + w * share, r.y);
        Quad acc[4] = {};
        add_tokens<T>(a, tok, b, min(b + share, r.y), c, n, acc);
#pragma unroll
        for (int q = 0; q < 4; ++q) st4(&part[w][4 * lane + 128 * q], acc[q]);
        __syncthreads();
        if (w == 0) {
            for (int i = 1; i < kWarps; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = add4(acc[q], quad_at(&part[i][4 * lane + 128 * q]));
            put_row<TT>(a, v, c, n, acc);
        }
        __syncthreads();
    }
    const int64_t units = static_cast<int64_t>(a.V) * slices, stride = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + w; u < units; u += stride) {
        const int v = static_cast<int>(u / slices), c0 = static_cast<int>(u - static_cast<int64_t>(v) * slices) * kSlice;
        const int2 r = a.range[v];
        if (r.y - r.x > kMany || (a.accumulate && r.y == r.x)) continue;
        const int c = c0 + 4 * lane, n = places(c0);
        Quad acc[4] = {};
        if (r.y > r.x) add_tokens<T>(a, tok, r.x, r.y, c, n, acc);
        put_row<TT>(a, v, c, n, acc);
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
    while (a->passes < 4 && s->V >> (8 * a->passes) != 0) ++a->passes;   // keys 0 .. V
}

int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

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
    const int64_t T = shape->tokens;
    return static_cast<size_t>(4 * up(4 * T) + up(8 * static_cast<int64_t>(shape->V)) + up(4 * (T / kMany + 2)));
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
    const int64_t units = shape->tokens * (shape->D / 4);
    const int64_t blocks = std::min<int64_t>((units + 255) / 256, 152 * 8);
    const cudaError_t e = by_type(shape, [&](auto tt, auto t) {
        return launch_dependent(embed_kernel<decltype(tt), decltype(t)>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                                reinterpret_cast<cudaStream_t>(stream), a, units, shape->D / 4);
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
    a.many = reinterpret_cast<int32_t*>(w);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_cluster(embed_sort_kernel, dim3(kSortBlocks), dim3(kSortThreads), kSortBlocks, cs, a);
    const int64_t units = static_cast<int64_t>(shape->V) * ((shape->D + kSlice - 1) / kSlice);
    const int64_t blocks = std::min<int64_t>((units + kWarps - 1) / kWarps, 152 * 2);
    if (e == cudaSuccess)
        e = by_type(shape, [&](auto tt, auto t) {
            return launch_dependent(embed_bwd_kernel<decltype(tt), decltype(t)>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, cs, a);
        });
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
