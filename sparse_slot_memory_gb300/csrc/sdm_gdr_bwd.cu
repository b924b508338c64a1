// sdm_gdr_bwd.cu -- the gated delta rule's backward: sdm_gdr_backward (include/sdm.h; mathematics and numbers: sdm_gdr.cuh).
//
// With S and S' the states before and behind a block, dS' the gradient of the latter, W the gradients of the writes u (so that
// dV = beta o W), and the forward's R, U, A, G, T:
//   W  = T^T (scale A^T dY + e^(gam_last - gam) o K dS')
//   dS = e^gam_last dS' + scale Q^T (e^gam o dY) - K^T (e^gam o dV)
//   M  = dV U^T, N = scale dY U^T
//   dQ = scale e^gam o dY S^T + (N o D) K
//   dK = (N o D)^T Q - (M o D) K - (M o D)^T K - e^gam o dV S^T + e^(gam_last - gam) o U dS'^T     (M o D strictly below the diagonal)
//   dbeta_i = W_i . U_i / beta_i      (a strength is never 0: sdm_gdr.cuh)
// and dg_t sums what every decay over row t brings, never a difference of such sums, so that strong decays keep their digits:
//   dg_t = sum_{j < t <= i} (N o A - M o G)_ij + sum_{i >= t} a_i + sum_{j < t} e_j + e^gam_last <dS', S>,
//   a_i = e^gam_i (scale q_i . (S dY_i) - dV_i . (S^T k_i)),   e_j = e^(gam_last - gam_j) u_j . (dS'^T k_j).
//
// Two kernels: a walk from each sequence's end that carries dS as the forward's carries S and writes dV, W and every block's dS';
// and one for all blocks at once that has the rest, from what the forward saved: the states, the writes, T, A T and the decays.
#include "sdm_gdr.cuh"

namespace sdm {
namespace gdr {
namespace {

// ---- the walk from the end, float32 rows ------------------------------------------------------------------------------
template <int DKP>
struct Back {
    static constexpr int BV = 32;
    static constexpr int kTile = kC * DKP * 2, kVal = kC * BV * 2, kPlane = kC * kC * 2;
    static constexpr int K = 0, Q = K + kTerms * kTile, Y = Q + kTerms * kTile, T = Y + kTerms * kVal, A = T + kTerms * kPlane,
                         vec = A + kTerms * kPlane, keep = vec + 3 * kC * 4, kKeep = kTerms * 16 * DKP * 2;
    static constexpr int warps = BV / 16, threads = warps * 32, bytes = keep + warps * kKeep;
};

template <int DKP>
__global__ void __launch_bounds__(Back<DKP>::threads) gdr_back_kernel(const __grid_constant__ Args a) {
    using W = Back<DKP>;
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
        load_rows<BV, W::threads>(base + W::Y, a.dy, NS, r0, n, h * a.dv + c0, cols, tid);
        const int64_t at = (id0 + j) * a.Hv + h;
        const __nv_bfloat16* const tri = a.tri + at * (2 * NS) * int64_t(kC * kC);
#pragma unroll
        for (int pl = 0; pl < 2 * NS; ++pl) load_tri<W::threads>(base + W::T + pl * W::kPlane, tri + pl * kC * kC, tid);
        if (tid < 48) copy16(base + W::vec + tid * 16, a.vec + at * kVecs * kC + tid * 4, true);
        copies_commit();
    };

    const Lane L(lane);
    float S[2 * KT][4];   // dS^T: 16 value columns x dk
    const int vc = c0 + 16 * w + g;
    {
        const float* const d = a.dhT == nullptr ? nullptr : a.dhT + (static_cast<int64_t>(p) * a.Hv + h) * a.dk * a.dv;
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 8 * t + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                S[t][e] = d != nullptr && i < a.dk && c < a.dv ? d[static_cast<int64_t>(i) * a.dv + c] : 0.f;
            }
    }
    const uint32_t keep = base + W::keep + w * W::kKeep;
    const float* const vec = reinterpret_cast<const float*>(smem + W::vec);
    for (int64_t it = 0; it < blocks; ++it) {
        const int64_t j = blocks - 1 - it;
        __syncthreads();
        load(j);
        copies_wait<0>();
        __syncthreads();
        if (16 * w >= cols) continue;
        if (lane == 0) bulk_wait_read();
        __syncwarp();
        const int64_t tile = ((id0 + j) * a.Hv + h) * groups + c0 / 16 + w;
        float x[8][4] = {};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {   // K dS'
            uint32_t s[NS][4];
            terms_of<NS>(S[2 * kt], S[2 * kt + 1], s);
#pragma unroll
            for (int t = 0; t < NS; ++t) stsm4(keep + t * (16 * DKP * 2) + state_at(L.rA, 2 * kt + L.uA), s[t]);
            products<NS, NS, NS, false, 4>(x, s, W::kTile, [&](int np) { return base + W::K + tile_at<DKP>(16 * np + L.rB, 2 * kt + L.uB); });
        }
        async_fence();
        __syncwarp();
        if (lane == 0) {
            bulk_store(a.dstates + tile * int64_t(NS * 16 * DKP), keep, W::kKeep);
            bulk_commit();
        }
        const float last = vec[kC - 1];
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[t][e] *= last;
        float u[8][4] = {};
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {   // A^T dY, and Q^T (scale e^gam dY)
            uint32_t y[NS][4];
#pragma unroll
            for (int t = 0; t < NS; ++t) ldsm4t(y[t], base + W::Y + t * W::kVal + tile_at<BV>(16 * kt + L.rAt, 2 * w + L.uAt));
            products<NS, NS, NS, true, 4>(u, y, W::kPlane, [&](int np) { return base + W::A + tile_at<kC>(16 * kt + L.rBt, 2 * np + L.uBt); }, 0, kt + 1);
            // the operand's columns are rows: 16 kt + 2 qd + {0, 1}, and 8 on
            uint32_t f[NS][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 eg = *reinterpret_cast<const float2*>(vec + 16 * kt + 8 * (i >> 1) + 2 * qd);
                float v0 = 0.f, v1 = 0.f;
#pragma unroll
                for (int t = NS - 1; t >= 0; --t) {
                    v0 += __uint_as_float(y[t][i] << 16);
                    v1 += __uint_as_float(y[t][i] & 0xFFFF0000u);
                }
                uint32_t o[NS];
                split2<NS>(a.scale * eg.x * v0, a.scale * eg.y * v1, o);
#pragma unroll
                for (int t = 0; t < NS; ++t) f[t][i] = o[t];
            }
            products<NS, NS, NS, true, KT>(S, f, W::kTile, [&](int np) { return base + W::Q + tile_at<DKP>(16 * kt + L.rBt, 2 * np + L.uBt); });
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const float2 c = *reinterpret_cast<const float2*>(vec + 2 * kC + 8 * nt + 2 * qd);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[nt][e] = fmaf(e & 1 ? c.y : c.x, x[nt][e], a.scale * u[nt][e]);
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {   // W = T^T dU
            uint32_t f[NS][4];
            terms_of<NS>(u[2 * kt], u[2 * kt + 1], f);
            products<NS, NS, NS, true, 4>(x, f, W::kPlane, [&](int np) { return base + W::T + tile_at<kC>(16 * kt + L.rBt, 2 * np + L.uBt); }, 0, kt + 1);
        }
        if (lane == 0) bulk_wait_read();   // the state's tile has left long ago
        __syncwarp();
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {   // W leaves; dV = beta W; - K^T (e^gam dV)
            uint32_t f[NS][4], o[NS][4];
            terms_of<NS>(x[2 * kt], x[2 * kt + 1], f);
#pragma unroll
            for (int t = 0; t < NS; ++t) stsm4t(keep + t * (kC * 32) + rows_at(16 * kt + L.rAt, L.uAt), f[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float2 bt = *reinterpret_cast<const float2*>(vec + kC + 16 * kt + 8 * t + 2 * qd);
                const float2 eg = *reinterpret_cast<const float2*>(vec + 16 * kt + 8 * t + 2 * qd);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * kt + t][e] *= e & 1 ? bt.y : bt.x;
                    u[2 * kt + t][e] = -(e & 1 ? eg.y : eg.x) * x[2 * kt + t][e];
                }
            }
            terms_of<NS>(u[2 * kt], u[2 * kt + 1], o);
            products<NS, NS, NS, true, KT>(S, o, W::kTile, [&](int np) { return base + W::K + tile_at<DKP>(16 * kt + L.rBt, 2 * np + L.uBt); });
        }
        async_fence();
        __syncwarp();
        if (lane == 0) {
            bulk_store(a.du + tile * int64_t(NS * kC * 16), keep, NS * kC * 32);
            bulk_commit();
        }
        const int64_t r0 = b + j * kC;
        const int n = static_cast<int>(min(len - j * kC, int64_t(kC)));
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 8 * nt + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                if (row < n && c < a.dv) static_cast<float*>(a.dv_out)[(r0 + row) * a.dv_ld + h * a.dv + c] = x[nt][e];
            }
    }
    if (a.dh0 != nullptr && 16 * w < cols) {
        float* const d = a.dh0 + (static_cast<int64_t>(p) * a.Hv + h) * a.dk * a.dv;
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 8 * t + 2 * qd + (e & 1), c = vc + (e >> 1) * 8;
                if (i < a.dk && c < a.dv) d[static_cast<int64_t>(i) * a.dv + c] = S[t][e];
            }
    }
    if (lane == 0) bulk_wait();
}

// ---- the walk from the end, bfloat16 rows ------------------------------------------------------------------------------
// As the forward's walk (sdm_gdr.cu), with dS in the threads' registers: per block of rows
//   K dS'  ->  x = e^(gam_last - gam) o K dS'  ->  W = T^T x + (scale A T)^T dY  ->  dS = e^gam_last dS' + Q^T (scale e^gam o dY) - K^T (e^gam o beta o W).
// What dY gives by itself is multiplied beside the chain; its scaled rows take the place of the state's terms while those are not needed.
// Measured, 8 x 4096 rows of 16 heads of 128: 344 us (1.6 GB: 4.6 TB/s). dV leaves in 16 bytes a thread, which the forward's answers
// do not: no place in shared memory is free for whole rows at that point.
template <int DKP, int BV>
__global__ void __launch_bounds__(BV * 4) gdr_back_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using W = WalkTc<DKP, BV>;
    static_assert(W::kR <= W::kS, "dY's terms lie over the state's");
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(128) float vecs[2][kVecs * kC];
    __shared__ __align__(8) uint64_t bars[6];   // the three products', then the copies' (WalkLoads)
    __shared__ uint32_t tmem;
    start_dependent();
    const int tid = threadIdx.x, w = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const int slices = (a.dv + BV - 1) / BV;
    const int rank = blockIdx.x / (a.Hv * slices), rest = blockIdx.x - rank * a.Hv * slices;
    const int h = rest / slices, c0 = (rest - h * slices) * BV;
    const int p = by_length(a, rank), kh = h / (a.Hv / a.Hk);
    int64_t b, len;
    sequence(a, p, b, len);
    const int64_t blocks = (len + kC - 1) / kC, id0 = first_block(b, p);
    const uint32_t base = smem_of(smem), bar = smem_of(bars);
    const int cols = min(BV, a.dv - c0), nb = (a.dv + 15) / 16 * 2;

    const WalkLoads<DKP, BV> loads{a, maps, a.dy, b, len, id0, base, smem_of(vecs), smem_of(bars) + 24, h, kh, c0, cols, tid, w, false};
    auto load_kq = [&](int64_t j) {
        if (j >= 0) loads.kq(j);
    };
    auto load_yt = [&](int64_t j) {
        if (j >= 0) loads.vt(j);
    };
    // what no copy reaches is a number
    for (int i = tid; i < W::bytes / 16; i += W::threads) *reinterpret_cast<uint4*>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    if (tid == 32) {
        for (int x = 0; x < 6; ++x) tensor::barrier_init(bar + 8 * x, 1);
        tensor::barrier_fence();
    }
    async_fence();
    __syncthreads();
    load_kq(blocks - 1);
    load_yt(blocks - 1);

    const int r = 32 * (w & 3) + lane, part = w >> 2, i = r & 63;
    const bool key = r < kC;
    const int vc = c0 + 32 * part;
    uint64_t S[16];
    {
        const float* const d = a.dhT == nullptr ? nullptr : a.dhT + ((static_cast<int64_t>(p) * a.Hv + h) * a.dk + r) * a.dv + vc;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float v[4] = {};
            if (d != nullptr && r < a.dk && vc + 4 * q < a.dv) load4(d + 4 * q).get(v);
            S[2 * q] = pack2(v[0], v[1]);
            S[2 * q + 1] = pack2(v[2], v[3]);
        }
    }
    unsigned char* const Sp = smem + W::S + part * 4 * (DKP * 16) + r * 16;
    unsigned char* const Yp = smem + W::S + part * 4 * 1024 + i * 16;
    unsigned char* const Xp = smem + W::R + part * 4 * 1024 + i * 16;
    auto put_state = [&]() {   // dS as operand
        if (r < DKP) put_terms(Sp, Sp + W::kS, DKP * 16, S);
    };
    const bool saving = w == 2;   // this warp's elected thread sends it off, for the other gradients
    put_state();
    if (w == 0) tensor::allocate<W::cols>(smem_of(&tmem));
    tensor::fence_before();
    __syncthreads();
    tensor::fence_after();
    const uint32_t Da = tmem, Db = tmem + W::N, Dc = Da;
    const uint32_t mine = (static_cast<uint32_t>(w & 3) << 21) + 32 * part;
    const uint64_t KQd = tensor::swizzled(base + W::KQ, 0), KTd = tensor::swizzled(base + W::KQ, 16384);
    const uint64_t Sd = tensor::operand(base + W::S, 128, DKP * 16), Yd = tensor::operand(base + W::S, 128, 1024);
    const uint64_t Td = tensor::operand(base + W::T, 128, 2048), dYd = tensor::swizzled(base + W::V + loads.first() * 16, 8192);
    const uint64_t Rd = tensor::operand(base + W::R, 128, 1024);
    uint32_t phase = 0, full = 0;
    bool bad = false;
    for (int64_t j = blocks - 1; j >= 0; --j) {
        const uint64_t kq = static_cast<uint64_t>((j & 1) * W::kKQ) >> 4;
        const float* const vec = vecs[j & 1];
        bad |= !tensor::barrier_wait(bar + 24 + 8 * (j & 1), full >> (j & 1) & 1);
        full ^= 1u << (j & 1);
        copies_wait<0>();
        async_fence();
        if (__syncthreads_or(bad)) break;
        if (saving && tensor::elect()) {
            unsigned char* const to = reinterpret_cast<unsigned char*>(a.dstates) + (((id0 + j) * a.Hv + h) * 2 * nb + c0 / 8) * int64_t(DKP * 16);
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
        load_kq(j - 1);
        bad |= !tensor::barrier_wait(bar, phase);
        bad |= !tensor::barrier_wait(bar + 40, phase);
        if (!loads.boxed(j)) {   // dY came by the threads' own copies
            copies_wait<0>();
            async_fence();
            __syncthreads();
        }
        tensor::fence_after();
        if (w == 0 && tensor::elect()) {   // what dY gives by A T: by the thread that commits it with T's products
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tensor::mma(W::terms == 1 ? Db + t * BV : Db, Td + (t * 16384 + 1024 + ks * 256) / 16, dYd + ks * 128, tensor::shape(128, BV, true, true), W::terms == 1 ? ks > 0 : t + ks > 0);
        }
        __syncwarp();
        uint64_t x[16];
        const float eg = vec[i], bt = vec[kC + i];
        if (key) {
            W::sums(Da + mine, x);
            const float c = vec[2 * kC + i];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = mul2(pack2(c, c), x[e]);
            put_terms(Xp, Xp + W::kR, 1024, x);
        } else {
            if (saving && tensor::elect()) bulk_wait_read();   // the state's terms, whose place dY's take
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(W::threads / 2) : "memory");
            const float f = a.scale * eg;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(smem + W::V + (part >> 1) * 8192 + swizzled_at(i, loads.first() + (part & 1) * 4 + q));
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q + e] = mul2(pack2(f, f), widen2(vw[e]));
            }
            put_terms(Yp, Yp + W::kR, 1024, x);
        }
        async_fence();
        tensor::fence_before();
        __syncthreads();
        if (w == 0 && tensor::elect()) {
            tensor::fence_after();
#pragma unroll
            for (int t = 0; t < W::terms; ++t)   // T's first term with both of x's, its second with the first
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tensor::mma(Db, Td + ks * 16, Rd + (t * W::kR + ks * 256) / 16, tensor::shape(128, W::N, true, true), true);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) tensor::mma(Db, Td + 1024 + ks * 16, Rd + ks * 16, tensor::shape(128, BV, true, true), true);
            tensor::commit(bar + 8);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int t = 0; t < W::terms; ++t)
                    tensor::mma(Dc, KTd + kq + 512 + ks * 128, Yd + (t * W::kR + ks * 256) / 16, tensor::shape(128, W::N, true, true), ks + t > 0);
        }
        bad |= !tensor::barrier_wait(bar + 8, phase);
        tensor::fence_after();
        uint64_t u[16];
        if (key) {
            W::sums(Db + mine, u);
            const float f = -eg * bt;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = mul2(pack2(f, f), u[e]);
            put_terms(Xp, Xp + W::kR, 1024, x);
        }
        async_fence();
        tensor::fence_before();
        __syncthreads();
        if (w == 0 && tensor::elect()) {
            tensor::fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int t = 0; t < W::terms; ++t)
                    tensor::mma(Dc, KTd + kq + ks * 128, Rd + (t * W::kR + ks * 256) / 16, tensor::shape(128, W::N, true, true), true);
            tensor::commit(bar + 16);
        }
        load_yt(j - 1);
        if (key) {
            unsigned char* const to = reinterpret_cast<unsigned char*>(a.du) + (((id0 + j) * a.Hv + h) * 2 * nb + vc / 8) * int64_t(1024) + i * 16;
            const bool there = i < min(len - j * kC, int64_t(kC));
            __nv_bfloat16* const dv = static_cast<__nv_bfloat16*>(a.dv_out) + (b + j * kC + i) * a.dv_ld + h * a.dv + vc;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (vc / 8 + q >= nb) continue;
                uint32_t hi[4], lo[4], o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    terms2(u[4 * q + e], hi[e], lo[e]);
                    float s, t;
                    unpack2(mul2(pack2(bt, bt), u[4 * q + e]), s, t);
                    o[e] = round2(s, t);
                }
                *reinterpret_cast<uint4*>(to + q * 1024) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(to + (nb + q) * 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (there && vc + 8 * q < a.dv) *reinterpret_cast<uint4*>(dv + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
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
    if (a.dh0 != nullptr && r < a.dk) {
        float* const d = a.dh0 + ((static_cast<int64_t>(p) * a.Hv + h) * a.dk + r) * a.dv + vc;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (vc + 4 * q < a.dv) st4(d + 4 * q, Quad{S[2 * q], S[2 * q + 1]});
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

// ---- all blocks at once, float32 rows ---------------------------------------------------------------------------------
// 16 warps: warp w has rows 16 (w % 4) .. of everything, and of each product's columns the (w / 4)-th part: 16 of the 64 columns
// of M and N, a quarter of dk. A block walks the value columns in slices of SL, the next ones' states, writes and gradients on
// their way; all operands come from shared memory as they were stored, so a slice needs one barrier.
template <int DKP>
struct Grad {
    static constexpr int NS = kTerms, SL = 16, stages = 2;
    static constexpr int kTile = kC * DKP * 2, kPlane = kC * kC * 2, kVal = kC * SL * 2;
    static constexpr int kState = SL / 16 * NS * 16 * DKP * 2, kRows = SL / 16 * NS * kC * 32;
    // within a stage
    static constexpr int S = 0, dS = kState, W = 2 * kState, U = W + kRows, Y = U + kRows, stage = Y + NS * kVal;
    // the whole
    static constexpr int K = 0, Q = NS * kTile, slices = 2 * NS * kTile, end = slices + stages * stage;
    // over the slices when they are done: N o D and - M o D, and the sums of dg
    static constexpr int ND = slices, XD = ND + NS * kPlane, Z = XD + NS * kPlane, last = Z + kC * 65 * 4;
    static constexpr int bytes = end > last ? end : last;
    static constexpr int threads = 512;
};

template <int DKP>
__global__ void __launch_bounds__(512) gdr_grad_kernel(const __grid_constant__ Args a) {
    using W = Grad<DKP>;
    constexpr int NS = W::NS, SL = W::SL, KT = DKP / 16, DN = DKP / 64;   // DN: tiles of 16 columns of dk of a warp
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(16) float vec[kVecs * kC];
    __shared__ float sums[2][4][kC];   // a, e by quarters
    __shared__ float diag[kC];         // W . U
    __shared__ float inner[16];
    start_dependent();
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3, mi = w & 3, qf = w >> 2;
    const int64_t id = blockIdx.x / a.Hv;
    const int h = blockIdx.x - static_cast<int>(id) * a.Hv, kh = h / (a.Hv / a.Hk);
    int64_t b;
    int n;
    block_rows(a, id, b, n);
    if (n <= 0) return;
    const uint32_t base = smem_of(smem);
    const int groups = (a.dv + 15) / 16, nslices = (a.dv + SL - 1) / SL;
    const int64_t unit = id * a.Hv + h;

    auto load = [&](int s) {
        if (s < nslices) {
            const uint32_t st = base + W::slices + s % W::stages * W::stage;
            const int c0 = s * SL, cols = min(SL, a.dv - c0);
            const int have = min(SL / 16, groups - c0 / 16);   // groups of 16 value columns that there are; the others are zeros
            const __nv_bfloat16* const sp = a.states + (unit * groups + c0 / 16) * (NS * 16 * DKP);
            const __nv_bfloat16* const dp = a.dstates + (unit * groups + c0 / 16) * (NS * 16 * DKP);
            const __nv_bfloat16* const wp = a.du + (unit * groups + c0 / 16) * (NS * kC * 16);
            const __nv_bfloat16* const up = a.writes + (unit * groups + c0 / 16) * (NS * kC * 16);
#pragma unroll
            for (int i = tid; i < W::kState / 16; i += W::threads) {
                const bool there = i < have * NS * 16 * DKP / 8;
                copy16(st + W::S + i * 16, there ? sp + i * 8 : sp, there);
                copy16(st + W::dS + i * 16, there ? dp + i * 8 : dp, there);
            }
#pragma unroll
            for (int i = tid; i < W::kRows / 16; i += W::threads) {
                const bool there = i < have * NS * kC * 2;
                copy16(st + W::W + i * 16, there ? wp + i * 8 : wp, there);
                copy16(st + W::U + i * 16, there ? up + i * 8 : up, there);
            }
            load_rows<SL, W::threads>(st + W::Y, a.dy, NS, b, n, h * a.dv + c0, cols, tid);
        }
        copies_commit();
    };
    load_rows<DKP, W::threads>(base + W::K, a.k, NS, b, n, kh * a.dk, a.dk, tid);
    load_rows<DKP, W::threads>(base + W::Q, a.q, NS, b, n, kh * a.dk, a.dk, tid);
#pragma unroll
    for (int s = 0; s + 1 < W::stages; ++s) load(s);
    for (int i = tid; i < kVecs * kC; i += W::threads) vec[i] = a.vec[unit * kVecs * kC + i];

    const Lane L(lane);
    const int row[2] = {16 * mi + g, 16 * mi + g + 8};   // of a lane's accumulators
    float dq[2 * DN][4] = {}, k2[2 * DN][4] = {}, k3[2 * DN][4] = {}, m[2][4] = {}, nn[2][4] = {};
    float ss = 0.f;
    for (int s = 0; s < nslices; ++s) {
        copies_wait<W::stages - 2>();
        __syncthreads();
        load(s + W::stages - 1);
        const int so = W::slices + s % W::stages * W::stage;
        const uint32_t st = base + so;
#pragma unroll
        for (int kt = 0; kt < SL / 16; ++kt) {
            const uint32_t Sg = st + W::S + kt * (NS * 16 * DKP * 2), Dg = st + W::dS + kt * (NS * 16 * DKP * 2);
            const uint32_t Ug = st + W::U + kt * (NS * kC * 32);
            uint32_t wa[NS][4], ya[NS][4], ua[NS][4];
#pragma unroll
            for (int t = 0; t < NS; ++t) {
                ldsm4(wa[t], st + W::W + kt * (NS * kC * 32) + t * (kC * 32) + rows_at(16 * mi + L.rA, L.uA));
                ldsm4(ua[t], Ug + t * (kC * 32) + rows_at(16 * mi + L.rA, L.uA));
            }
#pragma unroll
            for (int t = 0; t < NS; ++t) ldsm4(ya[t], st + W::Y + t * W::kVal + tile_at<SL>(16 * mi + L.rA, 2 * kt + L.uA));
            if (qf <= mi) {   // W U^T and dY U^T
                auto at = [&](int) { return Ug + rows_at(16 * qf + L.rB, L.uB); };
                products<NS, NS, NS, false, 1>(m, wa, kC * 32, at);
                products<NS, NS, NS, false, 1>(nn, ya, kC * 32, at);
            }
            // dY S^T, W S^T, U dS'^T
            auto sa = [&](int np) { return Sg + state_at(L.rBt, 2 * (DN * qf + np) + L.uBt); };
            auto da = [&](int np) { return Dg + state_at(L.rBt, 2 * (DN * qf + np) + L.uBt); };
            products<NS, NS, NS, true, DN>(dq, ya, 16 * DKP * 2, sa);
            products<NS, NS, NS, true, DN>(k2, wa, 16 * DKP * 2, sa);
            products<NS, NS, NS, true, DN>(k3, ua, 16 * DKP * 2, da);
        }
        if (vec[kC - 1] != 0.f) {   // <dS', S>, both in the same tiles
            for (int i = tid; i < SL / 16 * 16 * DKP / 8; i += W::threads) {
                const int gr = i / (16 * DKP / 8), o = gr * (NS * 16 * DKP * 2) + (i - gr * (16 * DKP / 8)) * 16;
                float x[8] = {}, y[8] = {};
#pragma unroll
                for (int t = NS - 1; t >= 0; --t) {
                    const uint4 p = *reinterpret_cast<const uint4*>(smem + so + W::S + o + t * (16 * DKP * 2));
                    const uint4 q = *reinterpret_cast<const uint4*>(smem + so + W::dS + o + t * (16 * DKP * 2));
                    const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[2 * e] += __uint_as_float(pw[e] << 16);
                        x[2 * e + 1] += __uint_as_float(pw[e] & 0xFFFF0000u);
                        y[2 * e] += __uint_as_float(qw[e] << 16);
                        y[2 * e + 1] += __uint_as_float(qw[e] & 0xFFFF0000u);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], y[e], ss);
            }
        }
    }
    // A and G once more, in float32
    float kk[2][4] = {}, qk[2][4] = {};
    if (qf <= mi) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            uint32_t ka[NS][4], qa[NS][4];
#pragma unroll
            for (int t = 0; t < NS; ++t) {
                ldsm4(ka[t], base + W::K + t * W::kTile + tile_at<DKP>(16 * mi + L.rA, 2 * kt + L.uA));
                ldsm4(qa[t], base + W::Q + t * W::kTile + tile_at<DKP>(16 * mi + L.rA, 2 * kt + L.uA));
            }
            auto at = [&](int) { return base + W::K + tile_at<DKP>(16 * qf + L.rB, 2 * kt + L.uB); };
            products<NS, NS, NS, false, 1>(kk, ka, W::kTile, at);
            products<NS, NS, NS, false, 1>(qk, qa, W::kTile, at);
        }
    }
    __syncthreads();   // every slice is done: their place is free
    float* const Z = reinterpret_cast<float*>(smem + W::Z);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = row[e], j = 16 * qf + 8 * t + 2 * qd;
            float x[2], y[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float d = 0.f;
                if (j + c <= i) d = decay<kTerms>((vec[3 * kC + i] - vec[3 * kC + j + c]) + (vec[4 * kC + i] - vec[4 * kC + j + c]));
                const float N = a.scale * nn[t][2 * e + c], M = vec[kC + i] * m[t][2 * e + c];
                if (j + c == i) diag[i] = m[t][2 * e + c];
                x[c] = j + c <= i ? d * N : 0.f;
                y[c] = j + c < i ? -d * M : 0.f;
                Z[i * 65 + j + c] = j + c < i ? fmaf(x[c], qk[t][2 * e + c], y[c] * kk[t][2 * e + c]) : 0.f;
            }
            uint32_t o[NS];
            split2<NS>(x[0], x[1], o);
#pragma unroll
            for (int p = 0; p < NS; ++p) st_word(base + W::ND + p * W::kPlane + tile_at<kC>(i, j >> 3) + qd * 4, o[p]);
            split2<NS>(y[0], y[1], o);
#pragma unroll
            for (int p = 0; p < NS; ++p) st_word(base + W::XD + p * W::kPlane + tile_at<kC>(i, j >> 3) + qd * 4, o[p]);
        }
    // the rows' scalars: a = e^gam (scale q . (S dY) - beta k . (S W)), e = e^(gam_last - gam) k . (dS' u)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = row[e];
        float qd1 = 0.f, kd2 = 0.f, kd3 = 0.f;
#pragma unroll
        for (int t = 0; t < 2 * DN; ++t) {
            const uint32_t at = tile_at<DKP>(r, 2 * DN * qf + t) + qd * 4;
            float q[2] = {}, k[2] = {};
#pragma unroll
            for (int p = NS - 1; p >= 0; --p) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(smem + W::Q + p * W::kTile + at);
                const uint32_t y = *reinterpret_cast<const uint32_t*>(smem + W::K + p * W::kTile + at);
                q[0] += __uint_as_float(x << 16);
                q[1] += __uint_as_float(x & 0xFFFF0000u);
                k[0] += __uint_as_float(y << 16);
                k[1] += __uint_as_float(y & 0xFFFF0000u);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qd1 = fmaf(q[c], dq[t][2 * e + c], qd1);
                kd2 = fmaf(k[c], k2[t][2 * e + c], kd2);
                kd3 = fmaf(k[c], k3[t][2 * e + c], kd3);
            }
        }
        const float eg = vec[r], be = vec[kC + r], c = vec[2 * kC + r];
        float x[2] = {eg * (a.scale * qd1 - be * kd2), c * kd3};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] += __shfl_xor_sync(kFull, x[i], 1);
            x[i] += __shfl_xor_sync(kFull, x[i], 2);
            if (qd == 0) sums[i][qf][r] = x[i];
        }
        // the rows' gradients so far
#pragma unroll
        for (int t = 0; t < 2 * DN; ++t)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                dq[t][2 * e + p] *= a.scale * eg;
                k3[t][2 * e + p] = fmaf(-eg * be, k2[t][2 * e + p], c * k3[t][2 * e + p]);
            }
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) ss += __shfl_xor_sync(kFull, ss, o);
    if (lane == 0) inner[w] = ss;
    __syncthreads();
    // dQ += (N o D) K; dK += (N o D)^T Q - (M o D) K - (M o D)^T K
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        auto ka = [&](int np) { return base + W::K + tile_at<DKP>(16 * kt + L.rBt, 2 * (DN * qf + np) + L.uBt); };
        auto qa = [&](int np) { return base + W::Q + tile_at<DKP>(16 * kt + L.rBt, 2 * (DN * qf + np) + L.uBt); };
        uint32_t f[NS][4];
        if (kt <= mi) {
#pragma unroll
            for (int p = 0; p < NS; ++p) ldsm4(f[p], base + W::ND + p * W::kPlane + tile_at<kC>(16 * mi + L.rA, 2 * kt + L.uA));
            products<NS, NS, NS, true, DN>(dq, f, W::kTile, ka);
#pragma unroll
            for (int p = 0; p < NS; ++p) ldsm4(f[p], base + W::XD + p * W::kPlane + tile_at<kC>(16 * mi + L.rA, 2 * kt + L.uA));
            products<NS, NS, NS, true, DN>(k3, f, W::kTile, ka);
        }
        if (kt >= mi) {
#pragma unroll
            for (int p = 0; p < NS; ++p) ldsm4t(f[p], base + W::XD + p * W::kPlane + tile_at<kC>(16 * kt + L.rAt, 2 * mi + L.uAt));
            products<NS, NS, NS, true, DN>(k3, f, W::kTile, ka);
#pragma unroll
            for (int p = 0; p < NS; ++p) ldsm4t(f[p], base + W::ND + p * W::kPlane + tile_at<kC>(16 * kt + L.rAt, 2 * mi + L.uAt));
            products<NS, NS, NS, true, DN>(k3, f, W::kTile, qa);
        }
    }
    // dg. Column by column sums from the bottom (8 rows a thread, then what lies below them), then row by row up to the diagonal.
    {
        const int j = tid & 63, s8 = tid >> 6;
        float run = 0.f;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            run += Z[(8 * s8 + i) * 65 + j];
            Z[(8 * s8 + i) * 65 + j] = run;
        }
        __syncthreads();
        float below = 0.f;
        for (int q = 7; q > s8; --q) below += Z[8 * q * 65 + j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) Z[(8 * s8 + i) * 65 + j] += below;
        __syncthreads();
        const int t = tid >> 3, part = tid & 7;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 8 * part + i;   // a column before row t, its end's share, and a row from t on
            if (c < t) {
                x += Z[t * 65 + c];
                x += sums[1][0][c] + sums[1][1][c] + sums[1][2][c] + sums[1][3][c];
            } else {
                x += sums[0][0][c] + sums[0][1][c] + sums[0][2][c] + sums[0][3][c];
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o /= 2) x += __shfl_xor_sync(kFull, x, o);
        if (part == 0 && t < n) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += inner[i];
            x = fmaf(vec[kC - 1], s, x);
            const float db = diag[t] / vec[kC + t];
            const int64_t gi = (b + t) * a.dg_ld + h, bi = (b + t) * a.db_ld + h;
            if (a.g_bf16) {
                static_cast<__nv_bfloat16*>(a.dg)[gi] = __float2bfloat16_rn(x);
                static_cast<__nv_bfloat16*>(a.dbeta)[bi] = __float2bfloat16_rn(db);
            } else {
                static_cast<float*>(a.dg)[gi] = x;
                static_cast<float*>(a.dbeta)[bi] = db;
            }
        }
    }
    // the rows' gradients: of a head's own queries and keys, or a value head's share of them in float32
    const int64_t HD = static_cast<int64_t>(a.Hv) * a.dk;
#pragma unroll
    for (int t = 0; t < 2 * DN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row[e], c = 16 * DN * qf + 8 * t + 2 * qd;
            if (r >= n || c >= a.dk) continue;
            float* const q = a.part != nullptr ? a.part + (b + r) * HD + h * a.dk + c : static_cast<float*>(a.dq) + (b + r) * a.dq_ld + kh * a.dk + c;
            float* const k = a.part != nullptr ? a.part + (a.rows + b + r) * HD + h * a.dk + c
                                               : static_cast<float*>(a.dk_out) + (b + r) * a.dk_ld + kh * a.dk + c;
            *reinterpret_cast<float2*>(q) = make_float2(dq[t][2 * e], dq[t][2 * e + 1]);
            *reinterpret_cast<float2*>(k) = make_float2(k3[t][2 * e], k3[t][2 * e + 1]);
        }
}

// ---- all blocks at once, bfloat16 rows --------------------------------------------------------------------------------
// All of the slices' products read what is stored as it is, so they are the fifth-generation tensor core's: one thread issues them,
// the sums stay in tensor memory, and the threads turn to them when a block's slices are through. Rows are stacked to the
// instruction's 128, [W; dY] against S and U, [U; .] against dS' (its lower half is not used), [K; Q] against K:
//   D1 = [W; dY] S^T, D2 = [U; .] dS'^T, D3 = [W; dY] U^T, D4 = [K; Q] K^T, then with the decays in
//   D5 = [-(M o D); N o D] K, D6 = (N o D)^T Q - (M o D)^T K,
// so a thread that has row r of tensor memory has row r of the key's side (r < 64) or row r - 64 of the query's, and a quarter of its
// columns. Resident blocks take (block of rows, head) after (block, head); the next ones' rows and states arrive, two slices of 32
// value columns ahead, while these are finished. Its floor is HBM: 272 KB a block of a head of 128, of which the states are 128 (6.7
// us on each of 152 SMs; measured 12.0). What bounds it is the chain of a block's phases: four slices of copies, products (1400
// cycles, in which shared memory is read all the time) and <dS', S>; the decays; then the gates' gradients beside the rows'. A
// block's sums fill tensor memory, so the next block's products wait until these are taken in. Left out one at a time, <dS', S> was
// worth 36 us of 725, the sums with queries and keys 19, the slices' products 50; the gates' gradients 118 and the rows' 147 before
// half of the warps took each and the rows left through shared memory (630). M o D and N o D enter D5 and D6 as two terms like all
// that is computed, so that the rows' gradients have their rounding's error alone (0.0017; one term: 0.0021, and 18 us less).
template <int DKP>
struct GradTc {
    // a slice: U's two terms, [W; dY], [W's rests; 0], S's and dS's two terms, all in units of 8 value columns
    static constexpr int kUnit = DKP * 16, kTerm = 4 * kUnit, kStates = 2 * kTerm;
    static constexpr int U = 0, WY = 8192, S = WY + 16384, dS = S + kStates, stage = dS + kStates;
    static constexpr int kKQ = 2 * kC * DKP * 2;             // [K; Q], two of them: tiles of 128 rows for 64 columns
    // [-(M o D); N o D] in two terms (as an operand of 128 columns its transpose is read 16 KB beyond either), the slices, the terms of dg
    static constexpr int XN = 2 * kKQ, slices = XN + 2 * 16384, Z = slices + 2 * stage, bytes = Z + 16 * (17 + 33 + 49 + 65) * 4;
    static_assert(2 * stage >= 16384, "the operand's end");
    static constexpr int threads = 512;
    // The place of row i of dg's terms: rows of block b of 16 have the 16 b + 16 columns up to their diagonal block's end
    __device__ static __forceinline__ int row(int i) {
        const int b = i >> 4;
        return 128 * b * (b + 1) + 16 * b + (i & 15) * (16 * b + 17);
    }
};

template <int DKP>
__global__ void __launch_bounds__(512, 1) gdr_grad_tc_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using W = GradTc<DKP>;
    constexpr int QC = DKP / 4;   // columns of dk of a thread
    struct Unit {
        int64_t id, b;   // id: block x head; its rows are [b, b + n)
        int h, kh, n;
    };
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(128) float vecs[2][kVecs * kC];
    __shared__ float sums[3][4][kC];   // scale-free q . (S dY), k . (S W), k . (dS' u) by quarters of dk
    __shared__ float diag[kC];         // W . U
    __shared__ float share[2][kC];     // a and e
    __shared__ float inner[W::threads / 32];
    __shared__ __align__(16) float far[4][68], near[kC];   // decays: e^(gam_16b - gam_j) before block b of 16 rows, e^(gam_i - gam_16b) within
    __shared__ Unit ring[4];           // the units that are loaded, by their number
    __shared__ __align__(8) uint64_t bars[7];   // a stage's products each, and the last ones; a stage's copies each, and [K; Q]'s
    __shared__ uint32_t tmem;
    start_dependent();
    const int tid = threadIdx.x, w = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_of(smem), bar = smem_of(bars);
    const int groups = (a.dv + 15) / 16, nslices = (groups + 1) / 2;
    const int64_t units = (a.rows / kC + a.P) * a.Hv;

    auto find = [&](int64_t id) {   // the first one from id on, in steps of the grid, that has rows: by one warp
        Unit u;
        u.n = u.h = u.kh = 0;
        u.b = 0;
        for (u.id = id; u.id < units; u.id += gridDim.x) {
            const int blk = static_cast<int>(u.id) / a.Hv;
            u.h = static_cast<int>(u.id) - blk * a.Hv;
            u.kh = u.h / (a.Hv / a.Hk);
            block_rows(a, blk, u.b, u.n);
            if (u.n > 0) break;
        }
        return u;
    };
    Unit lu;   // what is loaded next
    int ls = 0, lkq = 0;
    int64_t issued = 0, found = 0;   // slices on their way or there; units that follow the first
    auto load = [&]() {              // behind a barrier that stands behind the last one
        if (ls == 0) lu = ring[found & 3];
        if (lu.id < units) {
            const int sg = static_cast<int>(issued & 1);
            const uint32_t st = base + W::slices + sg * W::stage;
            const int g0 = 2 * ls, have = min(2, groups - g0), c0 = 32 * ls, cols = min(32, a.dv - c0), kh = lu.kh;
            const bool box = maps.boxes && lu.n == kC;
            // a copy takes its thread 80 cycles, so five warps share them
            if (w >= 1 && w < 5 + (ls == 0) && tensor::elect()) {
                const int64_t first = lu.id * 2 * (2 * groups) + 2 * g0, rest = first + 2 * groups;   // the slice's first unit of 8 value columns, by terms
                const uint32_t full = bar + 24 + 8 * sg, sb = have * 2 * W::kUnit, rb = have * 2048;
                if (w == 1) {
                    tensor::barrier_expect(full, 4 * (sb + rb));
                    tensor::copy_bulk(st + W::S, a.states + first * (DKP * 8), sb, full);
                    tensor::copy_bulk(st + W::S + W::kTerm, a.states + rest * (DKP * 8), sb, full);
                } else if (w == 2) {
                    tensor::copy_bulk(st + W::dS, a.dstates + first * (DKP * 8), sb, full);
                    tensor::copy_bulk(st + W::dS + W::kTerm, a.dstates + rest * (DKP * 8), sb, full);
                    tensor::copy_bulk(st + W::U, a.writes + first * (kC * 8), rb, full);
                    tensor::copy_bulk(st + W::U + 4096, a.writes + rest * (kC * 8), rb, full);
                } else if (w == 3) {
                    for (int x = 0; x < 2 * have; ++x) tensor::copy_bulk(st + W::WY + x * 2048, a.du + (first + x) * (kC * 8), 1024, full);
                } else if (w == 4) {
                    for (int x = 0; x < 2 * have; ++x) tensor::copy_bulk(st + W::WY + 8192 + x * 2048, a.du + (rest + x) * (kC * 8), 1024, full);
                } else {
                    const uint32_t to = base + lkq * W::kKQ, kqfull = bar + 40 + 8 * lkq;
                    tensor::barrier_expect(kqfull, kVecs * kC * 4 + (box ? W::kKQ : 0));
                    tensor::copy_bulk(smem_of(vecs[lkq]), a.vec + lu.id * kVecs * kC, kVecs * kC * 4, kqfull);
                    if (box) {
#pragma unroll
                        for (int x = 0; x < DKP / 64; ++x) {
                            tensor::copy_box(to + x * 16384, &maps.k, kh * DKP + x * 64, static_cast<int>(lu.b), kqfull);
                            tensor::copy_box(to + x * 16384 + 8192, &maps.q, kh * DKP + x * 64, static_cast<int>(lu.b), kqfull);
                        }
                    }
                }
            }
            if (tid >= 256) {   // dY: a warp takes eight rows of four units
                const int r = (tid & 7) + (tid >> 5 & 7) * 8, u = tid >> 3 & 3;
                const bool there = r < lu.n && u * 8 < cols;
                copy16(st + W::WY + u * 2048 + 1024 + r * 16, there ? a.dy.p + (lu.b + r) * a.dy.ld + lu.h * a.dv + c0 + u * 8 : a.dy.p, there);
            }
            if (ls == 0 && !box) {
                for (int x = tid; x < 2 * kC * (DKP / 8); x += W::threads) {
                    const int r = x / (DKP / 8), u = x % (DKP / 8), t = r & 63;
                    const Planes& p = r < kC ? a.k : a.q;
                    const bool there = t < lu.n && u * 8 < a.dk;
                    copy16(base + lkq * W::kKQ + (u >> 3) * 16384 + swizzled_at(r, u & 7),
                           there ? p.p + (lu.b + t) * p.ld + kh * a.dk + u * 8 : p.p, there);
                }
            }
            if (++ls == nslices) {
                ls = 0;
                lkq ^= 1;
                ++found;
                if (w == 6) {
                    const Unit next = find(lu.id + gridDim.x);
                    if (lane == 0) ring[found & 3] = next;
                }
            }
        }
        copies_commit();
        ++issued;
    };
    // zeros under dY's rests stay; what no copy reaches is a number
    for (int i = tid; i < W::bytes / 16; i += W::threads) *reinterpret_cast<uint4*>(smem + i * 16) = make_uint4(0, 0, 0, 0);
    if (w == 0) tensor::allocate<512>(smem_of(&tmem));
    if (tid == 0) {
        for (int i = 0; i < 7; ++i) tensor::barrier_init(bar + 8 * i, 1);
        tensor::barrier_fence();
    }
    if (w == 1) {
        const Unit first = find(blockIdx.x);
        if (lane == 0) ring[0] = first;
    }
    async_fence();
    tensor::fence_before();
    __syncthreads();
    tensor::fence_after();
    load();
    Unit u = lu;
    const uint32_t D1 = tmem, D2 = D1 + 128, D3 = D1 + 256, D4 = D1 + 320, D5 = D1 + 384, D6 = D1 + 256;
    const uint32_t mine = static_cast<uint32_t>(w & 3) << 21;   // this warp's 32 rows
    const int r = 32 * (w & 3) + lane, quarter = w >> 2, i = r & 63;
    const bool key = r < kC;                                    // the key's side
    uint32_t phase[2] = {};
    int64_t waited[2] = {}, step = 0, number = 0;   // steps whose products were waited for, by stage; slices and units that are through
    bool bad = false;
    int kq = 0;
    auto wait_stage = [&](int s, int64_t before) {   // the products of the stage's steps before step `before`
        while (waited[s] < (before - s + 1) / 2) {
            bad |= !tensor::barrier_wait(bar + 8 * s, phase[s]);
            phase[s] ^= 1;
            ++waited[s];
        }
    };
    while (u.id < units) {
        const uint32_t KQ = base + kq * W::kKQ;
        const float* const vec = vecs[kq];
        uint64_t ss = 0;
        bool out = false;
        for (int s = 0; s < nslices; ++s, ++step) {
            // the last slice's products are done and its states read, so the next one's copies follow this one's products
            const int sg = static_cast<int>(step & 1), so = W::slices + sg * W::stage;
            wait_stage(sg ^ 1, step);
            if (s == 0) bad |= !tensor::barrier_wait(bar + 40 + 8 * kq, static_cast<uint32_t>(number >> 1) & 1);
            copies_wait<0>();
            async_fence();
            out = __syncthreads_or(bad);
            if (out) break;
            bad |= !tensor::barrier_wait(bar + 24 + 8 * sg, static_cast<uint32_t>(step >> 1) & 1);
            __syncwarp();
            const int have = min(2, groups - 2 * s);
            if (w == 0 && tensor::elect()) {
                tensor::fence_after();
                const uint32_t st = base + so;
                if (s == 0) {
#pragma unroll
                    for (int ks = 0; ks < DKP / 16; ++ks) {
                        const uint64_t x = tensor::swizzled(KQ + (ks >> 2) * 16384 + (ks & 3) * 32, 0);
                        tensor::mma(D4, x, x, tensor::shape(128, 64, false, false), ks > 0);
                    }
                }
                for (int gr = 0; gr < have; ++gr) {
                    const uint64_t wy = tensor::operand(st + W::WY + gr * 4096, 2048, 128), w0 = wy + 8192 / 16;
                    const uint64_t uh = tensor::operand(st + W::U + gr * 2048, 1024, 128), ul = uh + 4096 / 16;
                    const uint64_t sh = tensor::operand(st + W::S + gr * 2 * W::kUnit, W::kUnit, 128), sl = sh + W::kTerm / 16;
                    const uint64_t dh = tensor::operand(st + W::dS + gr * 2 * W::kUnit, W::kUnit, 128), dl = dh + W::kTerm / 16;
                    constexpr uint32_t wide = tensor::shape(128, DKP, false, false), square = tensor::shape(128, 64, false, false);
                    const bool add = s + gr > 0;
                    tensor::mma(D3, wy, uh, square, add);
                    tensor::mma(D3, wy, ul, square, true);
                    tensor::mma(D3, w0, uh, square, true);
                    tensor::mma(D3, w0, ul, square, true);   // W . U, which dbeta takes, to 2^-17
                    tensor::mma(D1, wy, sh, wide, add);
                    tensor::mma(D1, wy, sl, wide, true);
                    tensor::mma(D1, w0, sh, wide, true);
                    tensor::mma(D2, uh, dh, wide, add);
                    tensor::mma(D2, uh, dl, wide, true);
                    tensor::mma(D2, ul, dh, wide, true);
                }
                tensor::commit(bar + 8 * sg);
            }
            if (issued == step + 1) load();
            if (s == 0) {
                auto gap = [&](int i, int j) { return decay<1>((vec[3 * kC + i] - vec[3 * kC + j]) + (vec[4 * kC + i] - vec[4 * kC + j])); };
                const int x = tid & 63, y = tid >> 6;
                if (y < 4) {
                    if (x < 16 * y) far[y][x] = gap(16 * y, x);
                } else if (y == 4) {
                    near[x] = gap(x, x & ~15);
                }
            }
            if (vec[kC - 1] != 0.f) {   // <dS', S>, both in the same tiles
                for (int x = tid; x < have * 2 * DKP; x += W::threads) {
                    const int o = x * 16;
                    uint64_t p[4], q[4];
#pragma unroll
                    for (int t = 1; t >= 0; --t) {
                        const uint4 y = *reinterpret_cast<const uint4*>(smem + so + W::S + o + t * W::kTerm);
                        const uint4 z = *reinterpret_cast<const uint4*>(smem + so + W::dS + o + t * W::kTerm);
                        const uint32_t yw[4] = {y.x, y.y, y.z, y.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = t ? widen2(yw[e]) : add2(p[e], widen2(yw[e]));
                            q[e] = t ? widen2(zw[e]) : add2(q[e], widen2(zw[e]));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss = fma2(p[e], q[e], ss);
                }
            }
            __syncwarp();
        }
        if (out) break;
        wait_stage(0, step);
        wait_stage(1, step);
        __syncthreads();   // the last stage's states have been read
        if (ls != 0 || lkq != kq) load();   // not yet queries and keys in these ones' place
        tensor::fence_after();
        // N o D and - M o D, and the terms of dg that both give
        float* const Z = reinterpret_cast<float*>(smem + W::Z);
        {
            float x[16], y[16];
            const int own = i >> 4;   // the row's block of 16
            tensor::fetch16(D3 + mine + 16 * quarter, x);
            tensor::fetch16(D4 + mine + 16 * quarter, y);
            tensor::arrived(x);
            tensor::arrived(y);
            const float mul = key ? -vec[kC + i] : a.scale;
            if (quarter < own) {
                const float f = mul * near[i];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    x[c] *= f * far[own][16 * quarter + c];
                    y[c] *= x[c];
                }
            } else if (quarter == own) {
                const float gh = vec[3 * kC + i], gl = vec[4 * kC + i];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const int j = 16 * quarter + c;
                    if (key && j == i) diag[i] = x[c];
                    const float d = decay<1>((gh - vec[3 * kC + j]) + (gl - vec[4 * kC + j]));
                    x[c] = j < i || (!key && j == i) ? d * (mul * x[c]) : 0.f;
                    y[c] = j < i ? x[c] * y[c] : 0.f;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = y[c] = 0.f;
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) terms2(pack2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1]), hi[e], lo[e]);
                unsigned char* const to = smem + W::XN + stacked_at(r, 2 * quarter + q);
                *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(to + 16384) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            async_fence();
            tensor::fence_before();
            float* const mine_z = Z + W::row(i) + 16 * quarter;
            if (key && quarter <= own) {
#pragma unroll
                for (int c = 0; c < 16; ++c) mine_z[c] = y[c];
            }
            __syncthreads();
            if (w == 0 && tensor::elect()) {
                tensor::fence_after();
                constexpr uint32_t out5 = tensor::shape(128, DKP, false, true), out6 = tensor::shape(128, DKP, true, true);
                const uint64_t k = tensor::swizzled(KQ, 16384), q = k + 8192 / 16, X = tensor::operand(base + W::XN, 2048, 128);
                const uint64_t Xt = tensor::operand(base + W::XN, 128, 2048);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        tensor::mma(D5, X + t * 1024 + ks * 256, k + ks * 128, out5, t + ks > 0);
                        tensor::mma(D6, Xt + t * 1024 + 64 + ks * 16, q + ks * 128, out6, t + ks > 0);
                        tensor::mma(D6, Xt + t * 1024 + ks * 16, k + ks * 128, out6, true);
                    }
                tensor::commit(bar + 16);
            }
            if (!key && quarter <= own) {
#pragma unroll
                for (int c = 0; c < 16; ++c) mine_z[c] += y[c];
            }
        }
        // the rows' products with their own queries and keys
        {
            float s1 = 0.f, s3 = 0.f;
#pragma unroll
            for (int p = 0; p < QC / 16; ++p) {
                const int c0 = QC * quarter + 16 * p;
                float v[16], t[16];
                tensor::fetch16(D1 + mine + c0, v);
                tensor::fetch16(D2 + mine + c0, t);
                tensor::arrived(v);
                tensor::arrived(t);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int un = c0 / 8 + q;
                    const uint4 x = *reinterpret_cast<const uint4*>(smem + kq * W::kKQ + (un >> 3) * 16384 + swizzled_at(r, un & 7));
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float k = __uint_as_float(e & 1 ? xw[e >> 1] & 0xFFFF0000u : xw[e >> 1] << 16);
                        s1 = fmaf(k, v[8 * q + e], s1);
                        s3 = fmaf(k, t[8 * q + e], s3);
                    }
                }
            }
            sums[key ? 1 : 0][quarter][i] = s1;
            if (key) sums[2][quarter][i] = s3;
        }
        {
            float s, t;
            unpack2(ss, s, t);
            s += t;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(kFull, s, o);
            if (lane == 0) inner[w] = s;
        }
        __syncthreads();
        // Half of the warps write dg and dbeta, the others meanwhile the rows' gradients.
        if (quarter >= 2) {
            const int g = tid - 256;
            auto sync = [&]() {
                __syncwarp();
                asm volatile("bar.sync 1, 256;" ::: "memory");
            };
            if (g < kC) {
                const float eg = vec[g];
                auto four = [&](int x) { return (sums[x][0][g] + sums[x][1][g]) + (sums[x][2][g] + sums[x][3][g]); };
                share[0][g] = eg * (a.scale * four(0) - vec[kC + g] * four(1));
                share[1][g] = vec[2 * kC + g] * four(2);
            }
            // Column by column sums from the bottom (16 rows a thread, then what lies below them), then row by row up to the diagonal.
            const int j = g & 63, part = g >> 6;
            float* const column = Z + W::row(16 * part) + j;
            const int pitch = 16 * part + 17;
            float (*const parts)[68] = far;   // whose decays have been taken
            float run = 0.f, z[16];
            if (j >> 4 <= part) {
#pragma unroll
                for (int x = 15; x >= 0; --x) {
                    run += column[x * pitch];
                    z[x] = run;
                }
            }
            parts[part][j] = run;
            sync();
            if (j >> 4 <= part) {
                float below = 0.f;
                for (int q = 3; q > part; --q) below += parts[q][j];
#pragma unroll
                for (int x = 0; x < 16; ++x) column[x * pitch] = z[x] + below;
            }
            sync();
            const int t = g >> 2, fourth = g & 3;
            const float* const row = Z + W::row(t);
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int c = 4 * e + fourth;   // a column before row t, its end's share, and a row from t on
                x += c < t ? row[c] + share[1][c] : share[0][c];
            }
            x += __shfl_xor_sync(kFull, x, 1);
            x += __shfl_xor_sync(kFull, x, 2);
            if (fourth == 0 && t < u.n) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < W::threads / 32; ++e) s += inner[e];
                x = fmaf(vec[kC - 1], s, x);
                const float db = diag[t] / vec[kC + t];
                const int64_t gi = (u.b + t) * a.dg_ld + u.h, bi = (u.b + t) * a.db_ld + u.h;
                if (a.g_bf16) {
                    static_cast<__nv_bfloat16*>(a.dg)[gi] = __float2bfloat16_rn(x);
                    static_cast<__nv_bfloat16*>(a.dbeta)[bi] = __float2bfloat16_rn(db);
                } else {
                    static_cast<float*>(a.dg)[gi] = x;
                    static_cast<float*>(a.dbeta)[bi] = db;
                }
            }
            __syncwarp();
        } else {
            // of a head's own queries and keys, or a value head's share of them in float32
            bad |= !tensor::barrier_wait(bar + 16, static_cast<uint32_t>(number) & 1);
            tensor::fence_after();
            const float f1 = key ? -vec[i] * vec[kC + i] : a.scale * vec[i], f2 = vec[2 * kC + i];
#pragma unroll
            for (int p = 0; p < DKP / 32; ++p) {
                const int c0 = DKP / 2 * quarter + 16 * p;
                float v[16], t[16];
                tensor::fetch16(D1 + mine + c0, v);
                tensor::fetch16(D5 + mine + c0, t);
                if (key) {   // whole warps
                    float x[16], y[16];
                    tensor::fetch16(D2 + mine + c0, x);
                    tensor::fetch16(D6 + mine + c0, y);
                    tensor::arrived(x);
                    tensor::arrived(y);
                    tensor::arrived(v);
                    tensor::arrived(t);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = fmaf(f2, x[c], fmaf(f1, v[c], t[c])) + y[c];
                } else {
                    tensor::arrived(v);
                    tensor::arrived(t);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = fmaf(f1, v[c], t[c]);
                }
                if (a.part != nullptr) {
                    float* const to = a.part + ((key ? a.rows : 0) + u.b + i) * a.Hv * a.dk + u.h * a.dk + c0;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (i < u.n && c0 + 4 * q < a.dk)
                            *reinterpret_cast<float4*>(to + 4 * q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else {   // over K and Q, which nobody needs any more, to leave in whole rows
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int un = c0 / 8 + q;
                        *reinterpret_cast<uint4*>(smem + kq * W::kKQ + (un >> 3) * 16384 + swizzled_at(r, un & 7)) =
                            make_uint4(round2(v[8 * q], v[8 * q + 1]), round2(v[8 * q + 2], v[8 * q + 3]), round2(v[8 * q + 4], v[8 * q + 5]),
                                       round2(v[8 * q + 6], v[8 * q + 7]));
                    }
                }
            }
            if (a.part == nullptr) {
                asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll
                for (int x = tid; x < 2 * kC * (DKP / 8); x += 256) {
                    const int row = x / (DKP / 8), un = x % (DKP / 8), t = row & 63;
                    if (t < u.n && un * 8 < a.dk) {
                        const uint4 v = *reinterpret_cast<const uint4*>(smem + kq * W::kKQ + (un >> 3) * 16384 + swizzled_at(row, un & 7));
                        const int64_t at = row < kC ? (u.b + t) * a.dk_ld : (u.b + t) * a.dq_ld;
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row < kC ? a.dk_out : a.dq) + at + u.h * a.dk + un * 8) = v;
                    }
                }
            }
            __syncwarp();
        }
        tensor::fence_before();
        ++number;
        u = ring[number & 3];
        kq ^= 1;
    }
    copies_wait<0>();
    if (__syncthreads_or(bad)) {   // a wait ran out: what has been written so far is not to be trusted
        if (tid == 0 && a.status != nullptr) atomicOr(a.status, SDM_DEV_STALLED);
        tensor::drain(bar, 7);
        __syncthreads();
    }
    tensor::fence_after();
    if (w == 0) tensor::release<512>(tmem);
}

// The gradients of queries and keys that several value heads share: their heads' shares in order, 4 columns a thread. Rows
// of no sequence stay as they are.
template <typename X>
__global__ void __launch_bounds__(256) gdr_join_kernel(const __grid_constant__ Args a) {
    start_dependent();
    const int R = a.Hv / a.Hk, units = a.Hk * a.dk / 4;
    const int64_t first = a.offsets == nullptr ? 0 : min(max(a.offsets[0], int64_t(0)), a.rows);
    const int64_t last = a.offsets == nullptr ? a.rows : max(min(a.offsets[a.P], a.rows), first);
    const int64_t count = (last - first) * units * 2;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < count; i += gridDim.x * int64_t(256)) {
        const bool k = i >= (last - first) * units;
        const int64_t at = k ? i - (last - first) * units : i, r = first + at / units;
        const int c = static_cast<int>(at % units) * 4, kh = c / a.dk, d = c - kh * a.dk;
        const float* src = a.part + ((k ? a.rows : 0) + r) * a.Hv * a.dk + static_cast<int64_t>(kh) * R * a.dk + d;
        float s[4] = {};
        for (int q = 0; q < R; ++q) {
            float x[4];
            load4(src + static_cast<int64_t>(q) * a.dk).get(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += x[e];
        }
        st4(static_cast<X*>(k ? a.dk_out : a.dq) + r * (k ? a.dk_ld : a.dq_ld) + c, s);
    }
}

// ---- host side ------------------------------------------------------------------------------------------------------
template <typename K>
cudaError_t big_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DKP>
cudaError_t back(const Args& a, cudaStream_t cs) {
    using W = Back<DKP>;
    auto* const k = gdr_back_kernel<DKP>;
    const cudaError_t e = big_smem(k, W::bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(a.P) * a.Hv * ((a.dv + W::BV - 1) / W::BV);
    return launch_dependent(k, dim3(static_cast<unsigned>(grid)), dim3(W::threads), W::bytes, cs, a);
}

template <int DKP>
cudaError_t grad_tc(const Args& a, int64_t blocks, cudaStream_t cs) {
    using W = GradTc<DKP>;
    auto* const k = gdr_grad_tc_kernel<DKP>;
    const cudaError_t e = big_smem(k, W::bytes);
    if (e != cudaSuccess) return e;
    Maps m;
    const cudaError_t f = make_maps(&m, a, a.dy, 64);
    if (f != cudaSuccess) return f;
    return launch_dependent(k, dim3(static_cast<unsigned>(std::min<int64_t>(blocks * a.Hv, 152))), dim3(W::threads), W::bytes, cs, a, m);
}

template <int DKP>
cudaError_t grad(const Args& a, int64_t blocks, cudaStream_t cs) {
    using W = Grad<DKP>;
    auto* const k = gdr_grad_kernel<DKP>;
    const cudaError_t e = big_smem(k, W::bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(k, dim3(static_cast<unsigned>(blocks * a.Hv)), dim3(W::threads), W::bytes, cs, a);
}

template <int DKP, int BV>
cudaError_t back_tc(const Args& a, cudaStream_t cs) {
    using W = WalkTc<DKP, BV>;
    auto* const k = gdr_back_tc_kernel<DKP, BV>;
    const cudaError_t e = big_smem(k, W::bytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(a.P) * a.Hv * ((a.dv + BV - 1) / BV);
    Maps m;
    const cudaError_t f = make_maps(&m, a, a.dy, BV);
    if (f != cudaSuccess) return f;
    return launch_dependent(k, dim3(static_cast<unsigned>(grid)), dim3(W::threads), W::bytes, cs, a, m);
}

template <int DKP>
cudaError_t back_bf16(const Args& a, cudaStream_t cs) {
    switch (columns(static_cast<int64_t>(a.P) * a.Hv, a.dv)) {
        case 32: return back_tc<DKP, 32>(a, cs);
        case 64: return back_tc<DKP, 64>(a, cs);
        default: return back_tc<DKP, 128>(a, cs);
    }
}

}  // namespace
}  // namespace gdr
}  // namespace sdm

using namespace sdm;
using namespace sdm::gdr;

extern "C" sdm_status sdm_gdr_backward(const sdm_gdr_shape* shape, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                       const void* v, int64_t v_ld, const void* g, int64_t g_ld, const void* beta,
                                       int64_t beta_ld, const void* dy, int64_t dy_ld, const int64_t* offsets,
                                       const void* states, const float* dhT, void* dq, int64_t dq_ld, void* dk, int64_t dk_ld,
                                       void* dv, int64_t dv_ld, void* dg, int64_t dg_ld, void* dbeta, int64_t dbeta_ld,
                                       float* dh0, void* ws, size_t ws_bytes, uint32_t* status, sdm_stream_t stream) {
    Args a;
    sdm_status st = check_inputs(shape, q, q_ld, k, k_ld, v, v_ld, g, g_ld, beta, beta_ld, offsets, ws, ws_bytes, true, status, &a);
    if (st != SDM_OK) return st;
    const int xe = shape->x_dtype == SDM_BF16 ? 2 : 4, ge = shape->g_dtype == SDM_BF16 ? 2 : 4;
    const int64_t kn = static_cast<int64_t>(shape->k_heads) * shape->dk, vn = static_cast<int64_t>(shape->v_heads) * shape->dv;
    if (shape->rows > 0) {
        if ((st = check_array(dy, dy_ld, vn, xe, 16, false)) != SDM_OK) return st;
        if ((st = check_array(dq, dq_ld, kn, xe, 16, true)) != SDM_OK) return st;
        if ((st = check_array(dk, dk_ld, kn, xe, 16, true)) != SDM_OK) return st;
        if ((st = check_array(dv, dv_ld, vn, xe, 16, true)) != SDM_OK) return st;
        if ((st = check_array(dg, dg_ld, shape->v_heads, ge, ge, true)) != SDM_OK) return st;
        if ((st = check_array(dbeta, dbeta_ld, shape->v_heads, ge, ge, true)) != SDM_OK) return st;
        if (states == nullptr) return SDM_ERR_ARG;
    }
    if (!checks::aligned_all(16, {states, dhT, dh0})) return SDM_ERR_ALIGN;
    a.dq = dq; a.dq_ld = dq_ld; a.dk_out = dk; a.dk_ld = dk_ld; a.dv_out = dv; a.dv_ld = dv_ld;
    a.dg = dg; a.dg_ld = dg_ld; a.dbeta = dbeta; a.db_ld = dbeta_ld; a.dhT = dhT; a.dh0 = dh0;
    set_states(shape, const_cast<void*>(states), &a);
    const Layout l = layout(shape, true);
    unsigned char* const w = static_cast<unsigned char*>(ws);
    a.dstates = reinterpret_cast<__nv_bfloat16*>(w + l.dstates);
    a.du = reinterpret_cast<__nv_bfloat16*>(w + l.du);
    a.part = shape->v_heads == shape->k_heads ? nullptr : reinterpret_cast<float*>(w + l.part);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (shape->rows > 0) {
        e = launch_planes(shape, q, q_ld, k, k_ld, v, v_ld, ws, true, &a, cs);
        if (shape->x_dtype == SDM_BF16) {
            a.dy = {static_cast<const __nv_bfloat16*>(dy), dy_ld, 0};
        } else {
            __nv_bfloat16* const to = reinterpret_cast<__nv_bfloat16*>(w + l.dy);
            a.dy = {to, vn, shape->rows * vn};
            if (e == cudaSuccess) e = launch_split(dy, dy_ld, shape->rows, static_cast<int>(vn), to, cs);
        }
    }
    const bool narrow = padded(shape->dk) == 64, bf16 = shape->x_dtype == SDM_BF16;
    if (e == cudaSuccess)
        e = bf16 ? (narrow ? back_bf16<64>(a, cs) : back_bf16<128>(a, cs)) : (narrow ? back<64>(a, cs) : back<128>(a, cs));
    const int64_t blocks = blocks_of(shape);
    if (e == cudaSuccess && shape->rows > 0)
        e = bf16 ? (narrow ? grad_tc<64>(a, blocks, cs) : grad_tc<128>(a, blocks, cs))
                 : (narrow ? grad<64>(a, blocks, cs) : grad<128>(a, blocks, cs));
    if (e == cudaSuccess && shape->rows > 0 && a.part != nullptr) {
        const int64_t grid = std::min<int64_t>((shape->rows * (kn / 4) * 2 + 255) / 256, 152 * 16);
        e = launch_dependent(bf16 ? gdr_join_kernel<__nv_bfloat16> : gdr_join_kernel<float>, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
                             cs, a);
    }
    return e == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}
