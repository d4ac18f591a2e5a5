// Routed (mixture) LoRA side path: a token carries up to K adapters with weights,
//   y_t = bf16( base_t + sum_j w_tj s_{e_tj} B'_{e_tj} (A'_{e_tj} x_t) ),
// the products of the experts a gate chose (router.cuh), or of LoRASpace's dynamically
// composed pool (the arXiv listing's abstract), at their retained ranks and with one
// rounding.  Gradients for frozen adapters, with u = B'^T dy per direction:
//   dx_t   = bf16( dx_base_t + sum_j w_tj s_j A'^T u ),   dw_tj = s_j < u , A'_j x_t >.
#pragma once
#include <cooperative_groups.h>

#include "apply_common.cuh"

namespace lf {

constexpr int kMixMaxK = 16;
constexpr int kMixMaxRows = kMixMaxK * kMaxRank;   // directions of one token
constexpr int kMixThreads = 512;
constexpr int kMixSeg = 1024;      // elements of one shrink unit: four 16-byte loads per lane
constexpr int kMixMaxSeg = 32;     // units per direction at most (longer rows use longer units)

struct MixProj {
    const __nv_bfloat16* x;      // rows of x_ld
    const __nv_bfloat16* in2;    // forward: base (nullable: zeros), rows of out_ld; gradient: dy, rows of dy_ld
    const __nv_bfloat16* base;   // gradient: dx_base (nullable: zeros)
    __nv_bfloat16* out;          // forward: y; gradient: dx (nullable)
    int64_t x_ld, dy_ld, out_ld, y_off;
    int32_t d_in, d_out, max_rank, pad;
    const int32_t* ranks;
    const int64_t* off_A;
    const int64_t* off_Bt;
    const __nv_bfloat16* A_pool;
    const __nv_bfloat16* Bt_pool;
    int64_t pool_A, pool_Bt;
};
struct MixArgs {
    int32_t T, K, n_adapters, n_proj;
    const int32_t* ids;          // T x K
    const float* weights;        // T x K (nullable: 1)
    float scale;
    const float* scales;         // per adapter (nullable)
    float* gw;                   // gradient: n_proj x T x K partial (or, for one projection, final) weight gradients
    MixProj p[kMaxProj];
};

struct MixSmem {
    int64_t oa[kMixMaxRows], ob[kMixMaxRows];   // row offsets in the pools
    float coef[kMixMaxRows];                    // w_j s_j of the row's slot
    float t[kMixMaxRows];                       // A' x, summed over the cluster
    float u[kMixMaxRows];                       // gradient: B'^T dy
    float part[2][kMixMaxRows];                 // this CTA's share of t and u (read by the cluster)
    int32_t k[kMixMaxK], first[kMixMaxK + 1];
    int64_t soa[kMixMaxK], sob[kMixMaxK];
    float sc[kMixMaxK], w[kMixMaxK];
    union {
        float seg[kMixThreads / 32][8];
        float red[kMixThreads * 8];             // expand partial sums of the row groups
    };
};

// part[r] = sum over [d0, d1) of v[d] * pool[off[r] + d], for r in [0, R): every warp takes
// whole (direction) rows over this CTA's range; when there are fewer rows than warps, a
// row's range is cut into equal pieces whose sums are added in order.  d0, d1 multiples of 8.
__device__ __forceinline__ void mix_shrink(const __nv_bfloat16* v, const __nv_bfloat16* pool, const int64_t* off, int R,
                                           int d0, int d1, float* red, float* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int W = kMixThreads / 32;
    const int len = d1 - d0;
    int S = 1;   // pieces per row
    while (S < kMixMaxSeg && (len + S - 1) / S > kMixSeg) ++S;
    while (S > 1 && R * S > kMixThreads * 8) --S;
    const int piece = ((len + S - 1) / S + 7) & ~7;
    for (int un = warp; un < R * S; un += W) {
        const int r = un / S, q = un - r * S;
        const int b = d0 + q * piece, e = min(d1, b + piece);
        const __nv_bfloat16* row = pool + off[r];
        float acc = 0.f;
        for (int d = b + lane * 8; d < e; d += 4 * 256) {
            uint4 xv[4], av[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (d + 256 * i < e) {
                    av[i] = __ldg(reinterpret_cast<const uint4*>(row + d + 256 * i));
                    xv[i] = __ldg(reinterpret_cast<const uint4*>(v + d + 256 * i));
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (d + 256 * i < e) {
                    float xf[8], af[8];
                    bf16x8_to_f32(xv[i], xf);
                    bf16x8_to_f32(av[i], af);
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc = fmaf(af[c], xf[c], acc);
                }
        }
        acc = warp_sum(acc);
        if (lane == 0) red[un] = acc;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += kMixThreads) {
        float s = 0.f;
        for (int q = 0; q < S; ++q) s += red[r * S + q];
        part[r] = s;
    }
    __syncthreads();
}

// out[c0 .. c1) = bf16(base + sum_r tc[r] pool[off[r] + c]); tc = t * coef formed here.
// Threads cover 8-column vectors; a narrow range is covered by several groups of threads
// that share the rows, summed through shared memory in group order.
__device__ __forceinline__ void mix_expand(const float* t, const float* coef, const __nv_bfloat16* pool,
                                           const int64_t* off, int R, const __nv_bfloat16* base, __nv_bfloat16* out,
                                           int c0, int c1, float* red) {
    const int tid = threadIdx.x;
    const int nvec = (c1 - c0) >> 3;
    int RG = 1, nv = kMixThreads;   // row groups, threads per group
    while (RG < 8 && nv / 2 >= nvec && 2 * RG <= R) {
        RG *= 2;
        nv /= 2;
    }
    const int rg = tid / nv, vt = tid - rg * nv;
    for (int v0 = 0; v0 < nvec; v0 += nv) {
        const int v = v0 + vt;
        const int c = c0 + 8 * v;
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        uint4 bv = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            if (rg == 0 && base) bv = *reinterpret_cast<const uint4*>(base + c);
            int r = rg;
            for (; r + 3 * RG < R; r += 4 * RG) {
                uint4 pv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pv[i] = __ldg(reinterpret_cast<const uint4*>(pool + off[r + i * RG] + c));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[8];
                    bf16x8_to_f32(pv[i], f);
                    const float tv = t[r + i * RG] * coef[r + i * RG];
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(tv, f[e], acc[e]);
                }
            }
            for (; r < R; r += RG) {
                float f[8];
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(pool + off[r] + c)), f);
                const float tv = t[r] * coef[r];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = fmaf(tv, f[e], acc[e]);
            }
        }
        if (RG > 1) {   // uniform
#pragma unroll
            for (int e = 0; e < 8; ++e) red[e * kMixThreads + tid] = acc[e];
            __syncthreads();
            if (rg == 0)
                for (int q = 1; q < RG; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] += red[e * kMixThreads + q * nv + vt];
            __syncthreads();
        }
        if (rg == 0 && v < nvec) {
            float bf[8];
            bf16x8_to_f32(bv, bf);
            uint4 o;
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(bf[2 * i] + acc[2 * i], bf[2 * i + 1] + acc[2 * i + 1]);
            *reinterpret_cast<uint4*>(out + c) = o;
        }
    }
}

__device__ __forceinline__ int mix_cut(int d, int part, int parts) {   // multiples of 8
    return (int)((int64_t)(d >> 3) * part / parts) * 8;
}

// Token-parallel form.  Cluster of CS CTAs per (token, projection): each takes a piece of
// d_in for the shrink, the pieces' sums are added over distributed shared memory in rank
// order, and each then writes its piece of the output columns.  CS grows as the batch
// shrinks, so that one token of one projection still spreads over 8 SMs; large batches use
// single CTAs.
template <bool GRAD>
__global__ void __launch_bounds__(kMixThreads, 2) mixture_token_kernel(const __grid_constant__ MixArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char mix_raw[];
    MixSmem& s = *reinterpret_cast<MixSmem*>(mix_raw);
    cg::cluster_group cl = cg::this_cluster();
    const int CS = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tok = blockIdx.x / CS, pi = blockIdx.y;
    const MixProj& P = a.p[pi];
    const int tid = threadIdx.x;
    if (tid < a.K) {
        const int ad = a.ids[(int64_t)tok * a.K + tid];
        const bool lead = rank == 0;
        int k = 0;
        int64_t oa = 0, ob = 0;
        if (ad < -1 || ad >= a.n_adapters) {
            if (lead && pi == 0) latch_error(LF_ERR_BAD_INDEX);
        } else if (ad >= 0) {
            factor_lookup(P.ranks, P.off_A, P.off_Bt, 0, P.max_rank, P.d_in, P.d_out, P.pool_A, P.pool_Bt, ad, lead, k,
                          oa, ob);
        }
        s.k[tid] = k;
        s.soa[tid] = oa;
        s.sob[tid] = ob;
        s.sc[tid] = k > 0 ? (a.scales ? a.scales[ad] : a.scale) : 0.f;
        s.w[tid] = k > 0 && a.weights ? a.weights[(int64_t)tok * a.K + tid] : 1.f;
    }
    __syncthreads();
    if (tid == 0) {
        int n = 0;
        for (int j = 0; j < a.K; ++j) {
            s.first[j] = n;
            n += s.k[j];
        }
        s.first[a.K] = n;
    }
    __syncthreads();
    const int R = s.first[a.K];
    for (int i = tid; i < a.K * kMaxRank; i += kMixThreads) {
        const int j = i / kMaxRank, q = i % kMaxRank;
        if (q < s.k[j]) {
            const int r = s.first[j] + q;
            s.oa[r] = s.soa[j] + (int64_t)q * P.d_in;
            s.ob[r] = s.sob[j] + (int64_t)q * P.d_out;
            s.coef[r] = s.w[j] * s.sc[j];
        }
    }
    __syncthreads();
    const __nv_bfloat16* x = P.x + (int64_t)tok * P.x_ld;
    const __nv_bfloat16* dy = GRAD ? P.in2 + (int64_t)tok * P.dy_ld + P.y_off : nullptr;
    mix_shrink(x, P.A_pool, s.oa, R, mix_cut(P.d_in, rank, CS), mix_cut(P.d_in, rank + 1, CS), s.red, s.part[0]);
    if (GRAD)
        mix_shrink(dy, P.Bt_pool, s.ob, R, mix_cut(P.d_out, rank, CS), mix_cut(P.d_out, rank + 1, CS), s.red, s.part[1]);
    if (CS > 1) cl.sync();
    for (int i = tid; i < (GRAD ? 2 : 1) * R; i += kMixThreads) {
        const int h = i >= R ? 1 : 0, r = i - h * R;
        float v = 0.f;
        for (int c = 0; c < CS; ++c) v += CS > 1 ? cl.map_shared_rank(&s.part[h][r], c)[0] : s.part[h][r];
        (h ? s.u : s.t)[r] = v;
    }
    __syncthreads();
    if (GRAD) {
        if (rank == 0 && a.gw) {
            for (int j = tid >> 5; j < a.K; j += kMixThreads / 32) {
                float d = 0.f;
                for (int r = s.first[j] + (tid & 31); r < s.first[j + 1]; r += 32) d = fmaf(s.t[r], s.u[r], d);
                d = warp_sum(d);
                if ((tid & 31) == 0) a.gw[((int64_t)pi * a.T + tok) * a.K + j] = s.sc[j] * d;
            }
        }
        if (P.out) {
            const __nv_bfloat16* base = P.base ? P.base + (int64_t)tok * P.out_ld : nullptr;
            __nv_bfloat16* out = P.out + (int64_t)tok * P.out_ld;
            if (R > 0 || base != out)
                mix_expand(s.u, s.coef, P.A_pool, s.oa, R, base, out, mix_cut(P.d_in, rank, CS),
                           mix_cut(P.d_in, rank + 1, CS), s.red);
        }
    } else {
        const int64_t at = (int64_t)tok * P.out_ld + P.y_off;
        const __nv_bfloat16* base = P.in2 ? P.in2 + at : nullptr;
        if (R > 0 || base != P.out + at)
            mix_expand(s.t, s.coef, P.Bt_pool, s.ob, R, base, P.out + at, mix_cut(P.d_out, rank, CS),
                       mix_cut(P.d_out, rank + 1, CS), s.red);
    }
    if (CS > 1) cl.sync();   // the sums above are read by the whole cluster
}

// grad_weights[t][j] = sum over the projections, in their order.
__global__ void mixture_gw_sum_kernel(const float* part, int n_proj, int64_t n, float* out) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int p = 0; p < n_proj; ++p) v += part[(int64_t)p * n + i];
    out[i] = v;
}

}  // namespace lf
