// sdm_gdr.cu -- the gated delta rule: the forward over sequences in blocks of 64 rows, and one token of every request:
// sdm_gdr_forward / sdm_gdr_step (include/sdm.h; the backward: sdm_gdr_bwd.cu; mathematics and numbers: sdm_gdr.cuh).
//
// Two kernels. What a block's rows give without the state (T, A T and the decays) is computed for all blocks at once; then
// every sequence and value head is walked block by block, its state's columns divided among blocks of threads where there are few.
#include "sdm_gdr.cuh"

namespace sdm {
namespace gdr {
namespace {

// ---- float32 rows as three planes of bfloat16 ------------------------------------------------------------------
__global__ void __launch_bounds__(256) gdr_split_kernel(const float* x, int64_t ld, int64_t rows, int cols, __nv_bfloat16* out) {
    start_dependent();
    const int units = cols / 4;
    const int64_t n = rows * units;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n; i += gridDim.x * int64_t(256)) {
        const int64_t r = i / units;
        const int c = static_cast<int>(i - r * units) * 4;
        float v[4];
        load4(x + r * ld + c).get(v);
        uint32_t a[3], b[3];
        split2<3>(v[0], v[1], a);
        split2<3>(v[2], v[3], b);
#pragma unroll
        for (int t = 0; t < 3; ++t) *reinterpret_cast<uint2*>(out + (t * rows + r) * cols + c) = make_uint2(a[t], b[t]);
    }
}

// ---- what a block's rows give without the state ---------------------------------------------------------------
// A block of 4 warps for each block of rows and key head; warp w holds rows 16 w .. of K K^T and Q K^T, and for each value head of
// the key head weighs them by its decays. T is built from its 16 x 16 blocks: those on the diagonal row by row in float32 (a
// column a lane), those below by T_21 = -T_22 (N_21 T_11), first for 32 rows, then for 64, in products of terms. Bound by the waits of
// this chain at four blocks an SM (41 % of the issue slots): 8320 blocks of a head of 128 in 185 us; the bytes would take 80.
template <int XT, int DKP>
__global__ void __launch_bounds__(128, XT == 1 ? 4 : 2) gdr_prepare_kernel(const __grid_constant__ Args a) {
    constexpr int kTile = kC * DKP * 2, kPlane = kC * kC * 2, NS = XT == 1 ? 2 : 3;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float gh[kC], gl[kC], be[kC];
    __shared__ float diag[4][16][17];
    start_dependent();
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
    const int64_t id = blockIdx.x / a.Hk;
    const int kh = blockIdx.x - static_cast<int>(id) * a.Hk;
    int64_t b;
    int n;
    block_rows(a, id, b, n);
    if (n <= 0) return;
    // N and T take the place of K and Q, which the accumulators have taken in
    const uint32_t K = smem_of(smem), Q = K + XT * kTile, N = K, T = N + NS * kPlane, A = T + NS * kPlane;
    load_rows<DKP, 128>(K, a.k, XT, b, n, kh * a.dk, a.dk, tid);
    load_rows<DKP, 128>(Q, a.q, XT, b, n, kh * a.dk, a.dk, tid);
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    const Lane L(lane);
    float kk[8][4] = {}, qk[8][4] = {};
#pragma unroll
    for (int kt = 0; kt < DKP / 16; ++kt) {
        uint32_t ka[XT][4], qa[XT][4];
#pragma unroll
        for (int x = 0; x < XT; ++x) {
            ldsm4(ka[x], K + x * kTile + tile_at<DKP>(16 * w + L.rA, 2 * kt + L.uA));
            ldsm4(qa[x], Q + x * kTile + tile_at<DKP>(16 * w + L.rA, 2 * kt + L.uA));
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > w) continue;
            uint32_t f[XT][4];
#pragma unroll
            for (int x = 0; x < XT; ++x) ldsm4(f[x], K + x * kTile + tile_at<DKP>(16 * np + L.rB, 2 * kt + L.uB));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                auto step = [&](float (&sum)[4], const uint32_t (&a)[XT][4]) {
                    add_step<XT>(sum, [&](float (&t)[4]) {
#pragma unroll
                        for (int x = XT - 1; x >= 0; --x)
#pragma unroll
                            for (int y = XT - 1 - x; y >= 0; --y) mma(t, a[y], f[x][2 * e], f[x][2 * e + 1]);
                    });
                };
                step(kk[2 * np + e], ka);
                step(qk[2 * np + e], qa);
            }
        }
    }
    __syncthreads();
    const int R = a.Hv / a.Hk;
    for (int rv = 0; rv < R; ++rv) {
        const int h = kh * R + rv;
        __nv_bfloat16* const tri = a.tri + (id * a.Hv + h) * (2 * NS) * int64_t(kC * kC);
        float* const vec = a.vec + (id * a.Hv + h) * kVecs * kC;
        if (w == 0) {
            // gates below -150 are 0 to float32 like -150 (a product with them is), and their sums stay finite. Sums in 64
            // bits, kept as two floats: e^(gam_i - gam_j) then has the error of one exponential.
            double s[2];
            float bt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                const float x = r < n ? gate_at(a.g, (b + r) * a.g_ld + h, a.g_bf16) : 0.f;
                s[e] = x < -150.f ? -150.f : x;
                bt[e] = strength(r < n ? gate_at(a.beta, (b + r) * a.b_ld + h, a.g_bf16) : 0.f);
            }
            s[1] += s[0];
            double run = s[1];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const double o = __shfl_up_sync(kFull, run, d);
                if (lane >= d) run += o;
            }
            const double last = __shfl_sync(kFull, run, 31);
            const double before = run - s[1];   // exact enough: both are sums of the same terms in 53 bits
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                const double gam = e ? run : before + s[0];
                const float hi = static_cast<float>(gam), lo = static_cast<float>(gam - hi);
                gh[r] = hi;
                gl[r] = lo;
                be[r] = bt[e];
                vec[3 * kC + r] = hi;
                vec[4 * kC + r] = lo;
                const float x = expf(hi);
                vec[r] = fmaf(x, lo, x);
                vec[kC + r] = bt[e];
                vec[2 * kC + r] = expf(static_cast<float>(last - gam));
            }
        }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            if (nt > 2 * w + 1) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // the two rows of a lane's accumulators
                const int i = 16 * w + g + 8 * e, j = 8 * nt + 2 * qd;
                float av[2], nv[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float d = decay<XT>((gh[i] - gh[j + c]) + (gl[i] - gl[j + c]));
                    av[c] = j + c <= i ? d * qk[nt][2 * e + c] : 0.f;
                    nv[c] = j + c < i ? be[i] * (d * kk[nt][2 * e + c]) : 0.f;
                    if (nt >> 1 == w) diag[w][g + 8 * e][j + c - 16 * w] = nv[c];
                }
                uint32_t t[NS];
                split2<NS>(av[0], av[1], t);
#pragma unroll
                for (int pl = 0; pl < NS; ++pl) {
                    if (XT == 1) st_word(A + pl * kPlane + tile_at<kC>(i, j >> 3) + (j & 7) * 2, t[pl]);
                    else *reinterpret_cast<uint32_t*>(tri + (NS + pl) * kC * kC + i * kC + j) = t[pl];
                }
                uint32_t u[NS];
                split2<NS>(nv[0], nv[1], u);
#pragma unroll
                for (int pl = 0; pl < NS; ++pl) st_word(N + pl * kPlane + tile_at<kC>(i, j >> 3) + (j & 7) * 2, u[pl]);
            }
        }
        __syncwarp();
        {   // the diagonal block: column c of (I + N)^-1, from the top down
            const int c = lane & 15;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == c ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) s = fmaf(-diag[w][i][j], x[j], s);
                x[i] = s;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // lane c and c + 1 share a word: the even one writes
                const float other = __shfl_down_sync(kFull, x[i], 1);
                uint32_t t[NS];
                split2<NS>(x[i], other, t);
                if (lane < 16 && !(lane & 1)) {
#pragma unroll
                    for (int pl = 0; pl < NS; ++pl)
                        st_word(T + pl * kPlane + tile_at<kC>(16 * w + i, 2 * w + (c >> 3)) + (c & 7) * 2, t[pl]);
                }
            }
        }
        __syncthreads();
        // 8 columns of a warp: y = N_21 T_11, out = -T_22 y. M: tiles of 16 rows (and of 16 summands) of a side.
        auto below = [&](auto mt, int r0, int c0, int c) {
            constexpr int M = decltype(mt)::value;
            float y[M][4] = {};
#pragma unroll
            for (int kt = 0; kt < M; ++kt) {
                if (kt < (c - c0) / 16) continue;   // T_11 is zero above the diagonal
                uint32_t t[NS][4];
#pragma unroll
                for (int p = 0; p < NS; ++p) ldsm4t(t[p], T + p * kPlane + tile_at<kC>(c0 + 16 * kt + L.rBt, c / 8));
#pragma unroll
                for (int m = 0; m < M; ++m)
                    add_step<NS>(y[m], [&](float (&sum)[4]) {
#pragma unroll
                        for (int x = 0; x < NS; ++x) {
                            const int p = NS == 3 ? NS - 1 - x : x;
                            uint32_t f[4];
                            ldsm4(f, N + p * kPlane + tile_at<kC>(r0 + 16 * m + L.rA, c0 / 8 + 2 * kt + L.uA));
#pragma unroll
                            for (int z = 0; z < NS - p; ++z) {
                                const int q = NS == 3 ? NS - 1 - p - z : z;
                                mma(sum, f, t[q][0], t[q][1]);
                            }
                        }
                    });
            }
            uint32_t yt[M][2][NS];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    split2<NS>(-y[m][2 * e], -y[m][2 * e + 1], yt[m][e]);
#pragma unroll
                    for (int p = 0; p < NS; ++p) yt[m][e][p] = transposed(yt[m][e][p]);
                }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                float o[4] = {};
#pragma unroll
                for (int kt = 0; kt <= m; ++kt)
                    add_step<NS>(o, [&](float (&sum)[4]) {
#pragma unroll
                        for (int x = 0; x < NS; ++x) {
                            const int p = NS == 3 ? NS - 1 - x : x;
                            uint32_t f[4];
                            ldsm4(f, T + p * kPlane + tile_at<kC>(r0 + 16 * m + L.rA, r0 / 8 + 2 * kt + L.uA));
#pragma unroll
                            for (int z = 0; z < NS - p; ++z) {
                                const int q = NS == 3 ? NS - 1 - p - z : z;
                                mma(sum, f, yt[kt][0][q], yt[kt][1][q]);
                            }
                        }
                    });
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t t[NS];
                    split2<NS>(o[2 * e], o[2 * e + 1], t);
#pragma unroll
                    for (int p = 0; p < NS; ++p) st_word(T + p * kPlane + tile_at<kC>(r0 + 16 * m + g + 8 * e, c / 8) + qd * 4, t[p]);
                }
            }
        };
        below(std::integral_constant<int, 1>{}, 32 * (w >> 1) + 16, 32 * (w >> 1), 32 * (w >> 1) + 8 * (w & 1));
        __syncthreads();
        below(std::integral_constant<int, 2>{}, 32, 0, 8 * w);
        __syncthreads();
        if constexpr (XT == 1) {   // scale A T, over A, whose rows are this warp's own
            float at[8][4] = {};
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                if (kt > w) continue;
                uint32_t f[NS][4];
#pragma unroll
                for (int p = 0; p < NS; ++p) ldsm4(f[p], A + p * kPlane + tile_at<kC>(16 * w + L.rA, 2 * kt + L.uA));
                products<NS, NS, NS, true, 4>(at, f, kPlane, [&](int np) { return T + tile_at<kC>(16 * kt + L.rBt, 2 * np + L.uBt); }, 0, kt + 1);
            }
            __syncwarp();
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                if (nt > 2 * w + 1) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t t[NS];
                    split2<NS>(a.scale * at[nt][2 * e], a.scale * at[nt][2 * e + 1], t);
#pragma unroll
                    for (int p = 0; p < NS; ++p) st_word(A + p * kPlane + tile_at<kC>(16 * w + g + 8 * e, nt) + qd * 4, t[p]);
                }
            }
            __syncthreads();
            // [T; scale A T] in cores of 8 rows: a term's 128 rows x 64
            for (int i = tid; i < 2 * NS * kC * 8; i += 128) {
                const int r = i & 63, u = i >> 6 & 7, lower = i >> 9 & 1, p = i >> 10;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (u <= (r >> 4) * 2 + 1) v = *reinterpret_cast<const uint4*>(smem + ((lower ? A : T) - K) + p * kPlane + tile_at<kC>(r, u));
                *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(tri) + p * 16384 + stacked_at(64 * lower + r, u)) = v;
            }
        } else {
            for (int i = tid; i < NS * kC * 8; i += 128) {
                const int p = i >> 9, r = (i >> 3) & 63, u = i & 7;
                if (u > (r >> 4) * 2 + 1) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(smem + (T - K) + p * kPlane + tile_at<kC>(r, u));
                *reinterpret_cast<uint4*>(tri + p * kC * kC + r * kC + u * 8) = v;
            }
        }
        if (rv + 1 < R) __syncthreads();
    }
}

// ---- the walk, float32 rows ---------------------------------------------------------------------------------------
// A warp owns 16 of a head's value columns and keeps its part of the state transposed, S^T [16 x dk], in the accumulators of its
// matrix instructions (mma.sync): an accumulator's layout is an operand's too, so the chain S -> R -> U -> S' never leaves the
// warp's registers. A block of rows takes 17 us (a sequence of 21 of them in both directions 815), which is this one chain: two warps a
// block, a stage of 160 KB, of which the tensor core's operands in three terms would leave room for no second one either.
template <int DKP>
struct Walk {
    static constexpr int BV = 32;   // value columns of a block
    static constexpr int kTile = kC * DKP * 2, kVal = kC * BV * 2, kPlane = kC * kC * 2;
    static constexpr int K = 0, Q = K + kTerms * kTile, V = Q + kTerms * kTile, T = V + kTerms * kVal, A = T + kTerms * kPlane,
                         vec = A + kTerms * kPlane, keep = vec + 3 * kC * 4, kKeep = kTerms * 16 * DKP * 2;
    static constexpr int warps = BV / 16, threads = warps * 32;
    static constexpr int bytes(bool saving) { return keep + (saving ? warps * kKeep : 0); }
};

template <int DKP>
__global__ void __launch_bounds__(Walk<DKP>::threads) gdr_walk_kernel(const __grid_constant__ Args a) {
    using W = Walk<DKP>;
    constexpr int KT = DKP / 16, NS = kTerms, BV = W::BV;
    extern __shared__ __align__(1024) unsigned char smem[];
    start_dependent();
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
    const int slices = (a.dv + BV - 1) / BV;
    const int rank = blockIdx.x / (a.Hv * slices), rest = blockIdx.x - rank * a.Hv * slices;
    const int h = rest / slices, c0 = (rest - h * slices) * BV;
    const int p = by_length(a, rank), kh = h / (a.Hv / a.Hk);
    int64_t b, len;
    sequence(a, p, b, len);
    const int64_t blocks = (len + kC - 1) / kC, id0 = first_block(b, p);
    const uint32_t base = smem_of(smem);
    const int cols = min(BV, a.dv - c0), groups = (a.dv + 15) / 16;

    auto load = [&](int64_t j) {
        const int n = static_cast<int>(min(len - j * kC, int64_t(kC)));
        const int64_t r0 = b + j * kC;
        load_rows<DKP, W::threads>(base + W::K, a.k, NS, r0, n, kh * a.dk, a.dk, tid);
        load_rows<DKP, W::threads>(base + W::Q, a.q, NS, r0, n, kh * a.dk, a.dk, tid);
        load_rows<BV, W::threads>(base + W::V, a.v, NS, r0, n, h * a.dv + c0, cols, tid);
        const int64_t at = (id0 + j) * a.Hv + h;
        const __nv_bfloat16* const tri = a.tri + at * (2 * NS) * int64_t(kC * kC);
#pragma unroll
        for (int pl = 0; pl < 2 * NS; ++pl) load_tri<W::threads>(base + W::T + pl * W::kPlane, tri + pl * kC * kC, tid);
        if (tid < 48) copy16(base + W::vec + tid * 16, a.vec + at * kVecs * kC + tid * 4, true);
        copies_commit();
    };

    const Lane L(lane);
    float S[2 * KT][4];   // S^T: 16 value columns x dk
    const int vc = c0 + 16 * w + g;   // this lane's value columns: vc and vc + 8
    {
        const float* const h0 = a.h0 == nullptr ? nullptr : a.h0 + (static_cast<int64_t>(p) * a.Hv + h) * a.dk * a.dv;
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = 8 * t + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                S[t][e] = h0 != nullptr && d < a.dk && c < a.dv ? h0[static_cast<int64_t>(d) * a.dv + c] : 0.f;
            }
    }
    const uint32_t keep = base + W::keep + w * W::kKeep;
    const float* const vec = reinterpret_cast<const float*>(smem + W::vec);
    for (int64_t j = 0; j < blocks; ++j) {
        __syncthreads();
        load(j);
        copies_wait<0>();
        __syncthreads();
        if (16 * w >= cols) continue;   // a warp without columns
        if (a.states != nullptr) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
        }
        float r[8][4] = {}, o[8][4] = {};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {   // K S and Q S
            uint32_t s[NS][4];
            terms_of<NS>(S[2 * kt], S[2 * kt + 1], s);
            if (a.states != nullptr) {
#pragma unroll
                for (int t = 0; t < NS; ++t) stsm4(keep + t * (16 * DKP * 2) + state_at(L.rA, 2 * kt + L.uA), s[t]);
            }
            products<NS, NS, NS, false, 4>(r, s, W::kTile, [&](int np) { return base + W::K + tile_at<DKP>(16 * np + L.rB, 2 * kt + L.uB); });
            products<NS, NS, NS, false, 4>(o, s, W::kTile, [&](int np) { return base + W::Q + tile_at<DKP>(16 * np + L.rB, 2 * kt + L.uB); });
        }
        if (a.states != nullptr) {   // the state before the block, for the backward
            async_fence();
            __syncwarp();
            if (lane == 0) {
                bulk_store(a.states + (((id0 + j) * a.Hv + h) * groups + c0 / 16 + w) * int64_t(NS * 16 * DKP), keep, W::kKeep);
                bulk_commit();
            }
        }
        // r = beta (v - e^gam K S); o = e^gam Q S
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t f[NS][4];
#pragma unroll
            for (int x = 0; x < NS; ++x) ldsm4t(f[x], base + W::V + x * W::kVal + tile_at<BV>(16 * np + L.rAt, 2 * w + L.uAt));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int nt = 2 * np + t;
                const float2 eg = *reinterpret_cast<const float2*>(vec + 8 * nt + 2 * qd);
                const float2 bt = *reinterpret_cast<const float2*>(vec + kC + 8 * nt + 2 * qd);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = 0.f;
#pragma unroll
                    for (int x = NS - 1; x >= 0; --x) {
                        const uint32_t word = f[x][2 * t + (e >> 1)];
                        v += __uint_as_float(e & 1 ? word & 0xFFFF0000u : word << 16);
                    }
                    const float x = e & 1 ? eg.y : eg.x;
                    r[nt][e] = (e & 1 ? bt.y : bt.x) * fmaf(-x, r[nt][e], v);
                    o[nt][e] *= x;
                }
            }
        }
        float u[8][4] = {};
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {   // U = T r
            uint32_t f[NS][4];
            terms_of<NS>(r[2 * kt], r[2 * kt + 1], f);
            products<NS, NS, NS, false, 4>(u, f, W::kPlane, [&](int np) { return base + W::T + tile_at<kC>(16 * np + L.rB, 2 * kt + L.uB); }, kt);
        }
        const float last = vec[kC - 1];
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[t][e] *= last;
        if (a.states != nullptr) {   // the state's tile has left long ago
            if (lane == 0) bulk_wait_read();
            __syncwarp();
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {   // A U, and K^T (e^(gam_last - gam) U)
            uint32_t f[NS][4];
            terms_of<NS>(u[2 * kt], u[2 * kt + 1], f);
            if (a.states != nullptr) {
#pragma unroll
                for (int t = 0; t < NS; ++t) stsm4t(keep + t * (kC * 32) + rows_at(16 * kt + L.rAt, L.uAt), f[t]);
            }
            products<NS, NS, NS, false, 4>(o, f, W::kPlane, [&](int np) { return base + W::A + tile_at<kC>(16 * np + L.rB, 2 * kt + L.uB); }, kt);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float2 c = *reinterpret_cast<const float2*>(vec + 2 * kC + 16 * kt + 8 * t + 2 * qd);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[2 * kt + t][e] *= e & 1 ? c.y : c.x;
            }
            terms_of<NS>(u[2 * kt], u[2 * kt + 1], f);
            products<NS, NS, NS, true, KT>(S, f, W::kTile, [&](int np) { return base + W::K + tile_at<DKP>(16 * kt + L.rBt, 2 * np + L.uBt); });
        }
        if (a.states != nullptr) {   // the writes, for the backward
            async_fence();
            __syncwarp();
            if (lane == 0) {
                bulk_store(a.writes + (((id0 + j) * a.Hv + h) * groups + c0 / 16 + w) * int64_t(NS * kC * 16), keep, NS * kC * 32);
                bulk_commit();
            }
        }
        // the rows' answers
        const int64_t r0 = b + j * kC;
        const int n = static_cast<int>(min(len - j * kC, int64_t(kC)));
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 8 * nt + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                if (row < n && c < a.dv) static_cast<float*>(a.y)[(r0 + row) * a.y_ld + h * a.dv + c] = o[nt][e] * a.scale;
            }
    }
    if (a.hT != nullptr && 16 * w < cols) {
        float* const hT = a.hT + (static_cast<int64_t>(p) * a.Hv + h) * a.dk * a.dv;
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = 8 * t + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                if (d < a.dk && c < a.dv) hT[static_cast<int64_t>(d) * a.dv + c] = S[t][e];
            }
    }
    if (a.states != nullptr && lane == 0) bulk_wait();
}

// ---- the walk, bfloat16 rows ---------------------------------------------------------------------------------------
// A block walks a sequence of a value head, BV of its value columns, with the state in its threads' registers in float32: thread
// (row r of 128, 32 columns) holds S[r]. Per block of rows three products follow one another on the fifth-generation tensor core,
//   [K; Q] S   ->  beta R = beta (V - e^gam K S)  ->  [T; scale A T] (beta R) = [U; scale A U]  ->  K^T (e^(gam_last - gam) U),
// their sums in tensor memory, their computed operands (S, R, U) as two terms in shared memory, in cores that their own threads
// write without conflicts. What bounds it is this chain: with 128 columns 2300 cycles of products, then 4 turns of a barrier,
// loads from tensor memory and the cut into terms. Tiles of K and Q arrive a block ahead, V and T while the state is brought up
// to date, in boxes of a tensor map and bulk copies; saved states leave in bulk copies of their operands. Measured, 8 x 4096 rows of 16
// heads of 128: 290 us with what is saved for the backward (1.6 GB: 5.5 TB/s).
//
// Where the walks are few and long, every sequence is cut into segments that are walked side by side, twice. A segment makes
// M S + B of the state S before it: the first time (FIRST) blocks start from zeros for B, and others, without V, from the identity
// for M; gdr_chain_kernel joins them to the states before the segments, from which the second walk starts. One sequence of 32769
// rows, 8 heads of 64 x 128: 952 us whole, 406 in 16 segments. Keys longer than 1 may grow M out of float32's range where the states
// stay in it, so the second walk of a head does not start from a state that came out as not finite: the segment before walks on to the
// sequence's end (4 us of the 406, and 1 to 4 of walks of whole sequences).
template <int DKP, int BV, bool FIRST>
__global__ void __launch_bounds__(BV * 4) gdr_walk_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps,
                                                             const __grid_constant__ Segments sg) {
    using W = WalkTc<DKP, BV>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(128) float vecs[2][kVecs * kC];
    __shared__ __align__(8) uint64_t bars[6];   // the three products', then the copies' (WalkLoads)
    __shared__ uint32_t tmem;
    start_dependent();
    const int tid = threadIdx.x, w = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const int own = (a.dv + BV - 1) / BV, slices = own + (FIRST ? (a.dk + BV - 1) / BV : 0), walks = sg.n - (FIRST ? 1 : 0);
    const int rank = blockIdx.x / (a.Hv * slices * walks), rest = blockIdx.x - rank * a.Hv * slices * walks;
    const int seg = rest / (a.Hv * slices), rest2 = rest - seg * a.Hv * slices;
    const int h = rest2 / slices, slice = rest2 - h * slices;
    const bool moving = FIRST && slice >= own;                       // the identity's columns
    const int width = moving ? a.dk : a.dv, c0 = (moving ? slice - own : slice) * BV;
    const int p = by_length(a, rank), kh = h / (a.Hv / a.Hk);
    int64_t b, len;
    sequence(a, p, b, len);
    const int64_t blocks = (len + kC - 1) / kC, id0 = first_block(b, p);
    if (FIRST && seg + slice + tid == 0) sg.ends[p * a.Hv + h] = sg.n;
    const int ends = FIRST || sg.n == 1 ? sg.n : sg.ends[p * a.Hv + h];
    if (seg >= ends) return;
    const bool last_one = seg == ends - 1;
    const uint32_t base = smem_of(smem), bar = smem_of(bars);
    const int64_t per = (blocks + sg.n - 1) / sg.n, j0 = min(seg * per, blocks), j1 = !FIRST && last_one ? blocks : min(j0 + per, blocks);
    const int cols = min(BV, width - c0), nb = (a.dv + 15) / 16 * 2;   // units of 8 value columns that are saved

    const WalkLoads<DKP, BV> loads{a, maps, a.v, b, len, id0, base, smem_of(vecs), smem_of(bars) + 24, h, kh, c0, cols, tid, w, moving};
    auto load_kq = [&](int64_t j) {
        if (j < j1) loads.kq(j);
    };
    auto load_vt = [&](int64_t j) {
        if (j < j1) loads.vt(j);
    };
    // what no copy reaches is a number
    for (int i = tid; i < W::bytes / 16; i += W::threads) *reinterpret_cast<uint4*>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    if (tid == 32) {
        for (int x = 0; x < 6; ++x) tensor::barrier_init(bar + 8 * x, 1);
        tensor::barrier_fence();
    }
    async_fence();
    __syncthreads();
    load_kq(j0);
    load_vt(j0);

    const int r = 32 * (w & 3) + lane, part = w >> 2, i = r & 63;   // a row of tensor memory, 32 columns, a token
    const bool key = r < kC;
    const int vc = c0 + 32 * part;                                  // this thread's first value column
    uint64_t S[16];   // 32 columns of a row of the state, in pairs
    {
        const float* const h0 =
            FIRST || sg.start == nullptr ? nullptr : sg.start + (((static_cast<int64_t>(p) * a.Hv + h) * sg.n + seg) * a.dk + r) * a.dv + vc;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float v[4] = {};
            if (h0 != nullptr && r < a.dk && vc + 4 * q < a.dv) load4(h0 + 4 * q).get(v);
            if (moving && r < a.dk) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = vc + 4 * q + e == r ? 1.f : 0.f;
            }
            S[2 * q] = pack2(v[0], v[1]);
            S[2 * q + 1] = pack2(v[2], v[3]);
        }
    }
    unsigned char* const Sp = smem + W::S + part * 4 * (DKP * 16) + r * 16;   // a unit of 8 columns: DKP rows of 16 bytes
    unsigned char* const Rp = smem + W::R + part * 4 * 1024 + i * 16;
    auto put_state = [&]() {   // S as operand
        if (r < DKP) put_terms(Sp, Sp + W::kS, DKP * 16, S);
    };
    const bool saving = !FIRST && a.states != nullptr && w == 2;   // this warp's elected thread sends it off, for the backward
    put_state();
    if (w == 0) tensor::allocate<W::cols>(smem_of(&tmem));
    tensor::fence_before();
    __syncthreads();
    tensor::fence_after();
    const uint32_t Da = tmem, Db = tmem + W::N, Dc = Da;
    const uint32_t mine = (static_cast<uint32_t>(w & 3) << 21) + 32 * part;
    // the products' operands. Per 16 summands: 32 bytes of [K; Q]'s rows (a tile for 64), 4096 of T's; 2048 along swizzled tokens, 256 of
    // the others
    const uint64_t KQd = tensor::swizzled(base + W::KQ, 0), KTd = tensor::swizzled(base + W::KQ, 16384);
    const uint64_t Sd = tensor::operand(base + W::S, 128, DKP * 16), Td = tensor::operand(base + W::T, 2048, 128);
    const uint64_t Rd = tensor::operand(base + W::R, 128, 1024);
    uint32_t phase = 0, full = 0;
    bool bad = false;
    for (int64_t j = j0; j < j1; ++j) {
        const uint64_t kq = static_cast<uint64_t>((j & 1) * W::kKQ) >> 4;   // the stage's distance, in a descriptor's units
        const float* const vec = vecs[j & 1];
        bad |= !tensor::barrier_wait(bar + 24 + 8 * (j & 1), full >> (j & 1) & 1);
        full ^= 1u << (j & 1);
        copies_wait<0>();
        async_fence();
        if (__syncthreads_or(bad)) break;
        if (saving && tensor::elect()) {
            unsigned char* const to = reinterpret_cast<unsigned char*>(a.states) + (((id0 + j) * a.Hv + h) * 2 * nb + c0 / 8) * int64_t(DKP * 16);
            const int bytes = min(BV / 8, nb - c0 / 8) * (DKP * 16);
            bulk_store(to, base + W::S, bytes);
            bulk_store(to + static_cast<int64_t>(nb) * (DKP * 16), base + W::S + W::kS, bytes);
            bulk_commit();
        }
        __syncwarp();
        if (w == 0 && tensor::elect()) {
            tensor::fence_after();
#pragma unroll
            for (int ks = 0; ks < DKP / 16; ++ks)
#pragma unroll
                for (int t = 0; t < W::terms; ++t)
                    tensor::mma(Da, KQd + kq + (ks >> 2) * 1024 + (ks & 3) * 2, Sd + (t * W::kS + ks * 256) / 16, tensor::shape(128, W::N, false, true), ks + t > 0);
            tensor::commit(bar);
        }
        load_kq(j + 1);
        bad |= !tensor::barrier_wait(bar, phase);
        bad |= !tensor::barrier_wait(bar + 40, phase);
        if (!loads.boxed(j)) {   // V came by the threads' own copies
            copies_wait<0>();
            async_fence();
            __syncthreads();
        }
        tensor::fence_after();
        uint64_t x[16];
        W::sums(Da + mine, x);
        const float eg = vec[i];
        if (key) {   // beta R
            const float bt = vec[kC + i];
            const uint64_t f = pack2(-bt * eg, -bt * eg), bt2 = pack2(bt, bt);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(smem + W::V + (part >> 1) * 8192 + swizzled_at(i, loads.first() + (part & 1) * 4 + q));
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q + e] = fma2(f, x[4 * q + e], mul2(bt2, widen2(vw[e])));
            }
            put_terms(Rp, Rp + W::kR, 1024, x);
        }
        async_fence();
        tensor::fence_before();
        __syncthreads();
        if (w == 0 && tensor::elect()) {
            tensor::fence_after();
#pragma unroll
            for (int t = 0; t < W::terms; ++t)   // T's first term with both of R's, its second with the first
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tensor::mma(Db, Td + ks * 256, Rd + (t * W::kR + ks * 256) / 16, tensor::shape(128, W::N, false, true), t + ks > 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) tensor::mma(Db, Td + 1024 + ks * 256, Rd + ks * 16, tensor::shape(128, BV, false, true), true);
            tensor::commit(bar + 8);
        }
        bad |= !tensor::barrier_wait(bar + 8, phase);
        tensor::fence_after();
        uint64_t u[16];
        W::sums(Db + mine, u);
        if (key) {
            const float c = vec[2 * kC + i];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = mul2(pack2(c, c), u[e]);
            put_terms(Rp, Rp + W::kR, 1024, x);
        }
        if (saving && tensor::elect()) bulk_wait_read();   // before the state is written anew
        __syncwarp();
        async_fence();
        tensor::fence_before();
        __syncthreads();
        if (w == 0 && tensor::elect()) {
            tensor::fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int t = 0; t < W::terms; ++t)
                    tensor::mma(Dc, KTd + kq + ks * 128, Rd + (t * W::kR + ks * 256) / 16, tensor::shape(128, W::N, true, true), ks + t > 0);
            tensor::commit(bar + 16);
        }
        load_vt(j + 1);
        const int64_t r0 = b + j * kC;
        const int n = static_cast<int>(min(len - j * kC, int64_t(kC)));
        if (key) {
            if (!FIRST && a.states != nullptr) {   // the writes, for the backward
                unsigned char* const to = reinterpret_cast<unsigned char*>(a.writes) + (((id0 + j) * a.Hv + h) * 2 * nb + vc / 8) * int64_t(1024) + i * 16;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (vc / 8 + q >= nb) continue;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) terms2(u[4 * q + e], hi[e], lo[e]);
                    *reinterpret_cast<uint4*>(to + q * 1024) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(to + (nb + q) * 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        } else if (!FIRST) {   // the row's answer
            const uint64_t f = pack2(a.scale * eg, a.scale * eg);
            __nv_bfloat16* const y = static_cast<__nv_bfloat16*>(a.y) + r0 * a.y_ld + h * a.dv;
            // Of 128 columns through the place of Q, which the first product has read, to leave in whole rows (8 x 4096 rows of 16 heads:
            // 288 us, 308 in 16 bytes a thread); fewer are not worth the barrier (12 prompts in 64 columns: 314 and 294).
            constexpr bool whole = BV == 128 && DKP == 128;
            unsigned char* const Q = smem + W::KQ + (j & 1) * W::kKQ + 8192;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s, t;
                    unpack2(fma2(f, x[4 * q + e], u[4 * q + e]), s, t);
                    o[e] = round2(s, t);
                }
                const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                if (whole) *reinterpret_cast<uint4*>(Q + (part >> 1) * 16384 + swizzled_at(i, (part & 1) * 4 + q)) = v;
                else if (i < n && vc + 8 * q < a.dv) *reinterpret_cast<uint4*>(y + i * a.y_ld + vc + 8 * q) = v;
            }
            if (whole) {
                asm volatile("bar.sync 1, %0;" ::"n"(W::threads / 2) : "memory");
#pragma unroll
                for (int t = 64 * part + i; t < kC * (BV / 8); t += W::threads / 2) {
                    const int row = t / (BV / 8), un = t % (BV / 8);
                    if (row < n && c0 + 8 * un < a.dv)
                        *reinterpret_cast<uint4*>(y + row * a.y_ld + c0 + 8 * un) = *reinterpret_cast<const uint4*>(Q + (un >> 3) * 16384 + swizzled_at(row, un & 7));
                }
            }
        }
        __syncwarp();
        const float last = vec[kC - 1];
        bad |= !tensor::barrier_wait(bar + 16, phase);
        phase ^= 1;
        tensor::fence_after();
        W::sums(Dc + mine, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = fma2(pack2(last, last), S[e], u[e]);
        put_state();
        tensor::fence_before();
    }
    const int64_t head = static_cast<int64_t>(p) * a.Hv + h;
    float* to = nullptr;
    if (FIRST) to = moving ? sg.move + (head * walks + seg) * a.dk * a.dk : sg.start + (head * sg.n + seg + 1) * a.dk * a.dv;
    else if (a.hT != nullptr && last_one) to = a.hT + head * a.dk * a.dv;
    if (to != nullptr && r < a.dk) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (vc + 4 * q < width) st4(to + static_cast<int64_t>(r) * width + vc + 4 * q, Quad{S[2 * q], S[2 * q + 1]});
    }
    if (saving && tensor::elect()) bulk_wait();
    __syncwarp();
    copies_wait<0>();
    if (__syncthreads_or(bad)) {
        if (tid == 0 && a.status != nullptr) atomicOr(a.status, SDM_DEV_STALLED);
        tensor::drain(bar, 6);
        __syncthreads();
    }
    tensor::fence_after();
    if (w == 0) tensor::release<W::cols>(tmem);
}

// The states before a sequence's segments, one after another: S' = M S + B in float32, 32 value columns a block. Rows of M are read
// by whole warps at once; the next M is on its way meanwhile. R: rows of a thread, dk / 8 or more (the last ones are computed again).
template <int R>
__global__ void __launch_bounds__(256) gdr_chain_kernel(const __grid_constant__ Args a, const __grid_constant__ Segments sg) {
    extern __shared__ __align__(1024) unsigned char smem[];
    start_dependent();
    const int slices = (a.dv + 31) / 32, tid = threadIdx.x, c = tid & 31, w = tid >> 5;
    const int64_t head = blockIdx.x / slices;
    const int col = (static_cast<int>(blockIdx.x - head * slices)) * 32 + c;
    const bool there = col < a.dv;
    float* const M = reinterpret_cast<float*>(smem);                 // two of [dk][dk]
    float* const S = M + 2 * a.dk * a.dk;                            // [dk][32]
    const int64_t size = static_cast<int64_t>(a.dk) * a.dv;
    float* const start = sg.start + head * sg.n * size;
    const float* const move = sg.move + head * (sg.n - 1) * a.dk * a.dk;
    auto load = [&](int s) {
        if (s < sg.n - 1)
            for (int i = tid * 4; i < a.dk * a.dk; i += 1024)
                copy16(smem_of(M + (s & 1) * a.dk * a.dk + i), move + static_cast<int64_t>(s) * a.dk * a.dk + i, true);
        copies_commit();
    };
    load(0);
    for (int r = w; r < a.dk; r += 8) {
        const float x = a.h0 != nullptr && there ? a.h0[head * size + static_cast<int64_t>(r) * a.dv + col] : 0.f;
        S[r * 32 + c] = x;
        if (there) start[static_cast<int64_t>(r) * a.dv + col] = x;
    }
    float x[R], ahead[R];   // rows w, w + 8 ..: dk is a multiple of 8
    auto fetch = [&](int s) {
        const float* const from = start + s * size;
#pragma unroll
        for (int i = 0; i < R; ++i) ahead[i] = s < sg.n && 8 * i < a.dk && there ? from[static_cast<int64_t>(w + 8 * i) * a.dv + col] : 0.f;
    };
    fetch(1);
    int ends = sg.n;
    for (int s = 0; s + 1 < sg.n; ++s) {
        load(s + 1);
        float* const next = start + (s + 1) * size;
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = ahead[i];
        fetch(s + 2);
        copies_wait<1>();
        __syncthreads();
        const float* const m = M + (s & 1) * a.dk * a.dk + w * a.dk;
#pragma unroll 2
        for (int k = 0; k < a.dk; k += 4) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = S[(k + e) * 32 + c];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(m + min(8 * i, a.dk - 8) * a.dk + k);
                x[i] = fmaf(f.x, y[0], x[i]);
                x[i] = fmaf(f.y, y[1], x[i]);
                x[i] = fmaf(f.z, y[2], x[i]);
                x[i] = fmaf(f.w, y[3], x[i]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (8 * i >= a.dk) continue;
            if (!isfinite(x[i])) ends = min(ends, s + 1);
            S[(w + 8 * i) * 32 + c] = x[i];
            if (there) next[static_cast<int64_t>(w + 8 * i) * a.dv + col] = x[i];
        }
    }
    if (there && ends < sg.n) atomicMin(sg.ends + head, ends);
    copies_wait<0>();
}

// ---- one token of every request -----------------------------------------------------------------------------------
// y = scale (e^g S^T q + (k.q) u), so one look at the state gives S^T k and S^T q together; it stays in registers until
// u is known, and is written once. Bound by HBM: 8 bytes an element of the state. 32 requests of 16 heads of 128 x 128: 11.0 us in a
// graph (6.1 TB/s), 15.7 with the host's call.
struct StepArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* g;
    const void* beta;
    const int32_t* slots;   // nullable
    float* state;
    void* y;
    uint32_t* status;       // nullable
    int64_t q_ld, k_ld, v_ld, g_ld, b_ld, s_ld, y_ld, states;
    int Hk, Hv, dk, dv, g_bf16;
    float scale;
};

template <typename X>
__device__ __forceinline__ float value_at(const void* p, int64_t i) {
    return widen(static_cast<const X*>(p)[i]);
}

// A block holds `cols` value columns of a head's state (a multiple of 4): thread t the columns 4 (t % (cols / 4)) .. and RPT
// rows from RPT (t / (cols / 4)) on.
template <typename X, int RPT>
__global__ void __launch_bounds__(256) gdr_step_kernel(const __grid_constant__ StepArgs a, int cols) {
    __shared__ float sk[kMaxD], sq[kMaxD];
    __shared__ __align__(16) float part[2][32][kMaxD];
    start_dependent();
    const int tid = threadIdx.x, slices = (a.dv + cols - 1) / cols;
    const int64_t unit = blockIdx.x / slices;
    const int c0 = (blockIdx.x - static_cast<int>(unit) * slices) * cols;
    const int64_t i = unit / a.Hv;
    const int h = static_cast<int>(unit - i * a.Hv), kh = h / (a.Hv / a.Hk);
    const int64_t slot = a.slots == nullptr ? i : a.slots[i];
    const int n = min(cols, a.dv - c0), cg = cols / 4;
    const int c = (tid % cg) * 4, part_of = tid / cg, parts = (a.dk + RPT - 1) / RPT, d0 = part_of * RPT;
    if (slot < 0 || slot >= a.states) {
        if (slot >= a.states && tid == 0 && a.status != nullptr) atomicOr(a.status, SDM_DEV_BAD_SLOT);
        for (int e = tid; e < n; e += 256) st1(static_cast<X*>(a.y) + i * a.y_ld + h * a.dv + c0 + e, 0.f);
        return;
    }
    const bool on = part_of < parts && c < n;
    float* const st = a.state + slot * a.s_ld + static_cast<int64_t>(h) * a.dk * a.dv + c0 + c;
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r)
        s[r] = on && d0 + r < a.dk ? *reinterpret_cast<const float4*>(st + static_cast<int64_t>(d0 + r) * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int d = tid; d < a.dk; d += 256) {
        sk[d] = value_at<X>(a.k, i * a.k_ld + kh * a.dk + d);
        sq[d] = value_at<X>(a.q, i * a.q_ld + kh * a.dk + d);
    }
    const float decay = expf(gate_at(a.g, i * a.g_ld + h, a.g_bf16)), beta = gate_at(a.beta, i * a.b_ld + h, a.g_bf16);
    float v[4] = {};
    if (on) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = value_at<X>(a.v, i * a.v_ld + h * a.dv + c0 + c + e);
    }
    __syncthreads();
    float pk[4] = {}, pq[4] = {}, kq = 0.f;
    if (on) {
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            if (d0 + r >= a.dk) break;
            const float k = sk[d0 + r], q = sq[d0 + r];
            pk[0] = fmaf(s[r].x, k, pk[0]); pk[1] = fmaf(s[r].y, k, pk[1]); pk[2] = fmaf(s[r].z, k, pk[2]); pk[3] = fmaf(s[r].w, k, pk[3]);
            pq[0] = fmaf(s[r].x, q, pq[0]); pq[1] = fmaf(s[r].y, q, pq[1]); pq[2] = fmaf(s[r].z, q, pq[2]); pq[3] = fmaf(s[r].w, q, pq[3]);
        }
        st4(&part[0][part_of][c], pk);
        st4(&part[1][part_of][c], pq);
    }
    for (int d = tid & 31; d < a.dk; d += 32) kq = fmaf(sk[d], sq[d], kq);
#pragma unroll
    for (int m = 16; m > 0; m /= 2) kq += __shfl_xor_sync(kFull, kq, m);
    __syncthreads();
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) pk[e] = pq[e] = 0.f;
    for (int p = 0; p < parts; ++p) {
        float x[4];
        get4(&part[0][p][c], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[e] += x[e];
        if (part_of == 0) {
            get4(&part[1][p][c], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) pq[e] += x[e];
        }
    }
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = beta * fmaf(-decay, pk[e], v[e]);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        if (d0 + r >= a.dk) break;
        const float k = sk[d0 + r];
        const float4 t = {fmaf(k, u[0], decay * s[r].x), fmaf(k, u[1], decay * s[r].y), fmaf(k, u[2], decay * s[r].z),
                          fmaf(k, u[3], decay * s[r].w)};
        *reinterpret_cast<float4*>(st + static_cast<int64_t>(d0 + r) * a.dv) = t;
    }
    if (part_of == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) pq[e] = a.scale * fmaf(kq, u[e], decay * pq[e]);
        st4(static_cast<X*>(a.y) + i * a.y_ld + h * a.dv + c0 + c, pq);
    }
}

// ---- host side ------------------------------------------------------------------------------------------------------
using checks::aligned16;
using checks::aligned_all;

int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

template <typename K>
cudaError_t big_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int XT, int DKP>
cudaError_t prepare(const Args& a, int64_t blocks, cudaStream_t cs) {
    constexpr int tiles = 2 * XT * kC * DKP * 2, planes = (XT == 1 ? 3 * 2 : 2 * 3) * kC * kC * 2, bytes = tiles > planes ? tiles : planes;
    auto* const k = gdr_prepare_kernel<XT, DKP>;
    const cudaError_t e = big_smem(k, bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(k, dim3(static_cast<unsigned>(blocks * a.Hk)), dim3(128), bytes, cs, a);
}

template <int DKP>
cudaError_t walk(const Args& a, cudaStream_t cs) {
    using W = Walk<DKP>;
    auto* const k = gdr_walk_kernel<DKP>;
    const int bytes = W::bytes(a.states != nullptr);
    const cudaError_t e = big_smem(k, bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(a.P) * a.Hv * ((a.dv + W::BV - 1) / W::BV);
    return launch_dependent(k, dim3(static_cast<unsigned>(grid)), dim3(W::threads), bytes, cs, a);
}

template <int DKP, int BV, bool FIRST>
cudaError_t walk_tc(const Args& a, const Segments& sg, cudaStream_t cs) {
    using W = WalkTc<DKP, BV>;
    auto* const k = gdr_walk_tc_kernel<DKP, BV, FIRST>;
    cudaError_t e = big_smem(k, W::bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(a.P) * a.Hv * (FIRST ? (sg.n - 1) * ((a.dv + BV - 1) / BV + (a.dk + BV - 1) / BV) : sg.n * ((a.dv + BV - 1) / BV));
    Maps m;
    e = make_maps(&m, a, a.v, BV);
    if (e != cudaSuccess) return e;
    return launch_dependent(k, dim3(static_cast<unsigned>(grid)), dim3(W::threads), W::bytes, cs, a, m, sg);
}

template <int DKP, bool FIRST>
cudaError_t walk_tc(const Args& a, const Segments& sg, cudaStream_t cs) {
    const int64_t walks = static_cast<int64_t>(a.P) * a.Hv * (FIRST ? sg.n - 1 : sg.n);
    switch (columns(walks, a.dv, FIRST ? a.dk : 0)) {
        case 32: return walk_tc<DKP, 32, FIRST>(a, sg, cs);
        case 64: return walk_tc<DKP, 64, FIRST>(a, sg, cs);
        default: return walk_tc<DKP, 128, FIRST>(a, sg, cs);
    }
}

template <int DKP>
cudaError_t walk_bf16(const Args& a, const Segments& sg, cudaStream_t cs) {
    if (sg.n > 1) {
        cudaError_t e = walk_tc<DKP, true>(a, sg, cs);
        if (e != cudaSuccess) return e;
        const int smem = (2 * a.dk * a.dk + a.dk * 32) * 4;
        auto* const chain = gdr_chain_kernel<DKP / 8>;
        e = big_smem(chain, smem);
        if (e == cudaSuccess) e = launch_dependent(chain, dim3(static_cast<unsigned>(a.P * a.Hv * ((a.dv + 31) / 32))), dim3(256), smem, cs, a, sg);
        if (e != cudaSuccess) return e;
    }
    return walk_tc<DKP, false>(a, sg, cs);
}

// Segments of a sequence's walk, of 16 blocks of rows each at least: two walks of a segment and the chain's 3 us a segment and 10
// against one walk of all rows (columns(), a fifth on top for what that leaves out). Measured, heads of 128 but for the first: one
// sequence of 4096 rows, 2 heads of 64, 80 us in 4 segments and 110 whole; 32768 rows, 4 heads, 374 in 16 and 931 whole; 4096 rows, 16
// heads, 163 in 4 and 140 whole; 2 of 8192, 16 heads, 494 in 4 and 330 whole.
int segments(const sdm_gdr_shape* s) {
    const int64_t walks = static_cast<int64_t>(s->P) * s->v_heads, blocks = s->rows / s->P / kC;
    if (s->x_dtype != SDM_BF16 || walks > 152) return 1;
    int best = 1;
    int64_t whole, first, second;   // in 0.01 us
    columns(walks, s->dv, 0, &whole);
    int64_t least = whole * blocks * 36;
    for (int n : {4, 8, 16}) {
        if (blocks < 16 * n) break;
        columns(walks * (n - 1), s->dv, s->dk, &first);
        columns(walks * n, s->dv, 0, &second);
        const int64_t t = ((first + second) * ((blocks + n - 1) / n) * 36 + n * 300 + 1000) * 6 / 5;
        if (t < least) best = n, least = t;
    }
    return best;
}

}  // namespace

sdm_status check_shape(const sdm_gdr_shape* s) {
    if (s == nullptr) return SDM_ERR_ARG;
    if (s->x_dtype < 0 || s->x_dtype > 1 || s->g_dtype < 0 || s->g_dtype > 1) return SDM_ERR_DTYPE;
    if (s->P < 1 || s->rows < 0 || s->rows > (int64_t(1) << 40) || s->k_heads < 1 || s->v_heads < 1 || s->v_heads > 65536 ||
        s->v_heads % s->k_heads != 0 || s->dk < 1 || s->dk > kMaxD || s->dv < 1 || s->dv > kMaxD || !(s->scale == s->scale))
        return SDM_ERR_SHAPE;
    if (s->dk % 8 != 0 || s->dv % 8 != 0) return SDM_ERR_ALIGN;
    if (blocks_of(s) > (int64_t(1) << 30) / s->v_heads || static_cast<int64_t>(s->P) * s->v_heads > (int64_t(1) << 28))
        return SDM_ERR_SHAPE;
    return SDM_OK;
}

// Bytes of a head's block of rows
int64_t tri_bytes(const sdm_gdr_shape* s) { return 2 * terms(s) * int64_t(kC * kC) * 2; }
constexpr int64_t kVecBytes = kVecs * kC * 4;
int64_t state_bytes(const sdm_gdr_shape* s) { return (s->dv + 15) / 16 * 16 * int64_t(padded(s->dk)) * 2 * terms(s); }
int64_t write_bytes(const sdm_gdr_shape* s) { return (s->dv + 15) / 16 * 16 * int64_t(kC) * 2 * terms(s); }

Layout layout(const sdm_gdr_shape* s, bool backward) {
    Layout l;
    memset(&l, 0, sizeof(l));
    const int64_t heads = blocks_of(s) * s->v_heads;
    const bool f32 = s->x_dtype == SDM_F32;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes);
        return here;
    };
    if (!backward) {   // from the end on they are read where the forward saved them
        l.tri = take(heads * tri_bytes(s));
        l.vec = take(heads * kVecBytes);
    }
    if (const int n = segments(s); n > 1) {
        l.start = take(static_cast<int64_t>(s->P) * s->v_heads * n * s->dk * s->dv * 4);
        l.move = take(static_cast<int64_t>(s->P) * s->v_heads * (n - 1) * s->dk * s->dk * 4);
        l.ends = take(static_cast<int64_t>(s->P) * s->v_heads * 4);
    }
    if (f32) {
        l.q = take(s->rows * s->k_heads * s->dk * 6);
        l.k = take(s->rows * s->k_heads * s->dk * 6);
        l.v = take(s->rows * s->v_heads * s->dv * 6);
    }
    if (backward) {
        if (f32) l.dy = take(s->rows * s->v_heads * s->dv * 6);
        l.dstates = take(heads * state_bytes(s));
        l.du = take(heads * write_bytes(s));
        if (s->v_heads != s->k_heads) l.part = take(2 * s->rows * s->v_heads * s->dk * 4);
    }
    l.bytes = std::max<int64_t>(at, backward ? layout(s, false).bytes : 256);   // a forward can use it too
    return l;
}

void set_states(const sdm_gdr_shape* s, void* states, Args* a) {
    a->states = static_cast<__nv_bfloat16*>(states);
    if (states == nullptr) return;
    const int64_t heads = blocks_of(s) * s->v_heads;
    unsigned char* at = static_cast<unsigned char*>(states) + heads * state_bytes(s);
    a->writes = reinterpret_cast<__nv_bfloat16*>(at);
    at += heads * write_bytes(s);
    a->tri = reinterpret_cast<__nv_bfloat16*>(at);
    a->vec = reinterpret_cast<float*>(at + heads * tri_bytes(s));
}

cudaError_t launch_split(const void* x, int64_t ld, int64_t rows, int cols, __nv_bfloat16* out, cudaStream_t cs) {
    const int64_t blocks = std::min<int64_t>((rows * (cols / 4) + 255) / 256, 152 * 8);
    return launch_dependent(gdr_split_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, cs, static_cast<const float*>(x), ld, rows,
                            cols, out);
}

sdm_status check_inputs(const sdm_gdr_shape* s, const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                        const void* g, int64_t g_ld, const void* beta, int64_t b_ld, const int64_t* offsets, void* ws,
                        size_t ws_bytes, bool backward, uint32_t* status, Args* a) {
    sdm_status st = check_shape(s);
    if (st != SDM_OK) return st;
    if (offsets == nullptr && s->rows % s->P != 0) return SDM_ERR_SHAPE;
    const int xe = s->x_dtype == SDM_BF16 ? 2 : 4, ge = s->g_dtype == SDM_BF16 ? 2 : 4;
    const int64_t kn = static_cast<int64_t>(s->k_heads) * s->dk, vn = static_cast<int64_t>(s->v_heads) * s->dv;
    if (s->rows > 0) {
        if ((st = check_array(q, q_ld, kn, xe, 16, false)) != SDM_OK) return st;
        if ((st = check_array(k, k_ld, kn, xe, 16, false)) != SDM_OK) return st;
        if ((st = check_array(v, v_ld, vn, xe, 16, false)) != SDM_OK) return st;
        if ((st = check_array(g, g_ld, s->v_heads, ge, ge, false)) != SDM_OK) return st;
        if ((st = check_array(beta, b_ld, s->v_heads, ge, ge, false)) != SDM_OK) return st;
    }
    if (!aligned_all(8, {offsets}) || !aligned_all(4, {status})) return SDM_ERR_ALIGN;
    const Layout l = layout(s, backward);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < static_cast<size_t>(l.bytes)) return SDM_ERR_WORKSPACE;
    memset(a, 0, sizeof(*a));
    a->P = s->P; a->Hk = s->k_heads; a->Hv = s->v_heads; a->dk = s->dk; a->dv = s->dv; a->rows = s->rows;
    a->len = s->rows / s->P; a->scale = s->scale; a->g_bf16 = s->g_dtype == SDM_BF16;
    a->g = g; a->g_ld = g_ld; a->beta = beta; a->b_ld = b_ld; a->offsets = offsets; a->status = status;
    unsigned char* const w = static_cast<unsigned char*>(ws);
    a->tri = reinterpret_cast<__nv_bfloat16*>(w + l.tri);
    a->vec = reinterpret_cast<float*>(w + l.vec);
    return SDM_OK;
}

cudaError_t make_maps(Maps* m, const Args& a, const Planes& v, int bv) {
    static const auto encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess || found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
    }();
    if (encode == nullptr) return cudaErrorNotSupported;
    memset(m, 0, sizeof(*m));
    constexpr int64_t far = int64_t(1) << 38;   // elements between rows
    m->boxes = a.dk == padded(a.dk) && a.dv % (bv < 64 ? 64 : bv) == 0 && a.rows >= kC && a.rows < (int64_t(1) << 31) && a.k.ld >= a.Hk * a.dk &&
               a.q.ld >= a.Hk * a.dk && v.ld >= a.Hv * a.dv && a.k.ld < far && a.q.ld < far && v.ld < far;
    if (!m->boxes) return cudaSuccess;
    auto map = [&](CUtensorMap* to, const Planes& x, int cols) {
        const cuuint64_t size[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(a.rows)}, stride[1] = {static_cast<cuuint64_t>(x.ld) * 2};
        const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
        return encode(to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16*>(x.p), size, stride, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&m->k, a.k, a.Hk * a.dk) && map(&m->q, a.q, a.Hk * a.dk) && map(&m->v, v, a.Hv * a.dv) ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_planes(const sdm_gdr_shape* s, const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                          void* ws, bool backward, Args* a, cudaStream_t cs) {
    const Layout l = layout(s, backward);
    const int64_t kn = static_cast<int64_t>(s->k_heads) * s->dk, vn = static_cast<int64_t>(s->v_heads) * s->dv;
    cudaError_t e = cudaSuccess;
    auto take = [&](Planes* p, const void* x, int64_t ld, int64_t n, int64_t at) {
        if (s->x_dtype == SDM_BF16) {
            *p = {static_cast<const __nv_bfloat16*>(x), ld, 0};
            return;
        }
        __nv_bfloat16* const to = reinterpret_cast<__nv_bfloat16*>(static_cast<unsigned char*>(ws) + at);
        *p = {to, n, s->rows * n};
        if (e == cudaSuccess) e = launch_split(x, ld, s->rows, static_cast<int>(n), to, cs);
    };
    take(&a->q, q, q_ld, kn, l.q);
    take(&a->k, k, k_ld, kn, l.k);
    take(&a->v, v, v_ld, vn, l.v);
    return e;
}

cudaError_t launch_prepare(const Args& a, const sdm_gdr_shape* s, cudaStream_t cs) {
    const int64_t n = blocks_of(s);
    if (s->x_dtype == SDM_BF16) return padded(s->dk) == 64 ? prepare<1, 64>(a, n, cs) : prepare<1, 128>(a, n, cs);
    return padded(s->dk) == 64 ? prepare<3, 64>(a, n, cs) : prepare<3, 128>(a, n, cs);
}

}  // namespace gdr
}  // namespace sdm

using namespace sdm;
using namespace sdm::gdr;

extern "C" size_t sdm_gdr_states_bytes(const sdm_gdr_shape* shape) {
    if (check_shape(shape) != SDM_OK) return 0;
    return static_cast<size_t>(blocks_of(shape) * shape->v_heads * (state_bytes(shape) + write_bytes(shape) + tri_bytes(shape) + kVecBytes));
}

extern "C" size_t sdm_gdr_workspace_bytes(const sdm_gdr_shape* shape, int32_t backward) {
    if (check_shape(shape) != SDM_OK) return 0;
    return static_cast<size_t>(layout(shape, backward != 0).bytes);
}

extern "C" sdm_status sdm_gdr_forward(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                      const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta,
                                      int64_t beta_ld, const int64_t* offsets, const float* h0, void* y, int64_t y_ld,
                                      float* hT, void* states, void* ws, size_t ws_bytes, uint32_t* status,
                                      sdm_stream_t stream) {
    Args a;
    sdm_status st = check_inputs(shape, q, q_ld, k, k_ld, v, v_ld, g, g_ld, beta, beta_ld, offsets, ws, ws_bytes, false, status, &a);
    if (st != SDM_OK) return st;
    const int64_t vn = static_cast<int64_t>(shape->v_heads) * shape->dv;
    if (shape->rows > 0 && (st = check_array(y, y_ld, vn, shape->x_dtype == SDM_BF16 ? 2 : 4, 16, true)) != SDM_OK) return st;
    if (!aligned_all(16, {h0, hT, states})) return SDM_ERR_ALIGN;
    a.h0 = h0; a.y = y; a.y_ld = y_ld; a.hT = hT;
    set_states(shape, states, &a);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (shape->rows > 0) {
        e = launch_planes(shape, q, q_ld, k, k_ld, v, v_ld, ws, false, &a, cs);
        if (e == cudaSuccess) e = launch_prepare(a, shape, cs);
    }
    const bool narrow = padded(shape->dk) == 64;
    if (e == cudaSuccess) {
        Segments sg = {segments(shape), const_cast<float*>(h0), nullptr, nullptr};
        if (sg.n > 1) {
            const Layout l = layout(shape, false);
            sg.start = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + l.start);
            sg.move = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + l.move);
            sg.ends = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + l.ends);
        }
        if (shape->x_dtype == SDM_BF16) e = narrow ? walk_bf16<64>(a, sg, cs) : walk_bf16<128>(a, sg, cs);
        else e = narrow ? walk<64>(a, cs) : walk<128>(a, cs);
    }
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

extern "C" sdm_status sdm_gdr_step(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                   const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta,
                                   int64_t beta_ld, const int32_t* slots, float* state, int64_t state_ld, int64_t states,
                                   void* y, int64_t y_ld, uint32_t* status, sdm_stream_t stream) {
    sdm_status st = check_shape(shape);
    if (st != SDM_OK) return st;
    if (states < 0 || (slots == nullptr && states < shape->rows)) return SDM_ERR_SHAPE;
    if (shape->rows == 0) return SDM_OK;
    if (!aligned_all(4, {slots, status})) return SDM_ERR_ALIGN;
    const int xe = shape->x_dtype == SDM_BF16 ? 2 : 4, ge = shape->g_dtype == SDM_BF16 ? 2 : 4;
    const int64_t kn = static_cast<int64_t>(shape->k_heads) * shape->dk, vn = static_cast<int64_t>(shape->v_heads) * shape->dv;
    if ((st = check_array(q, q_ld, kn, xe, 16, false)) != SDM_OK) return st;
    if ((st = check_array(k, k_ld, kn, xe, 16, false)) != SDM_OK) return st;
    if ((st = check_array(v, v_ld, vn, xe, 16, false)) != SDM_OK) return st;
    if ((st = check_array(g, g_ld, shape->v_heads, ge, ge, false)) != SDM_OK) return st;
    if ((st = check_array(beta, beta_ld, shape->v_heads, ge, ge, false)) != SDM_OK) return st;
    if ((st = check_array(y, y_ld, vn, xe, 16, true)) != SDM_OK) return st;
    if (states > 0 && (st = check_array(state, state_ld, vn * shape->dk, 4, 16, true)) != SDM_OK) return st;
    StepArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.v = v; a.v_ld = v_ld; a.g = g; a.g_ld = g_ld; a.beta = beta; a.b_ld = beta_ld;
    a.slots = slots; a.state = state; a.s_ld = state_ld; a.states = states; a.y = y; a.y_ld = y_ld; a.status = status;
    a.Hk = shape->k_heads; a.Hv = shape->v_heads; a.dk = shape->dk; a.dv = shape->dv; a.g_bf16 = shape->g_dtype == SDM_BF16;
    a.scale = shape->scale;
    // 64 columns of a head to a block: 16 threads across, so 8 rows of up to 128 to each; narrower heads leave threads idle
    const int cols = std::min(64, shape->dv), parts = 256 / (cols / 4);
    const int64_t blocks = shape->rows * shape->v_heads * ((shape->dv + cols - 1) / cols);
    if (blocks > 0x7FFFFFFF) return SDM_ERR_SHAPE;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    auto launch = [&](auto x, auto rpt) {
        return launch_dependent(gdr_step_kernel<decltype(x), decltype(rpt)::value>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, cs, a, cols);
    };
    auto by_rows = [&](auto x) {
        return (shape->dk + 3) / 4 <= std::min(parts, 32) ? launch(x, std::integral_constant<int, 4>{}) : launch(x, std::integral_constant<int, 8>{});
    };
    const cudaError_t e = shape->x_dtype == SDM_BF16 ? by_rows(__nv_bfloat16{}) : by_rows(0.f);
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
