// Routed (mixture) LoRA side path: a token carries up to K adapters with weights,
//   y_t = bf16( base_t + sum_j w_tj s_{e_tj} B'_{e_tj} (A'_{e_tj} x_t) ),
// the products of the experts a gate chose (router.cuh), or of LoRASpace's dynamically
// composed pool (the arXiv listing's abstract), at their retained ranks and with one
// rounding.  Gradients for frozen adapters, with u = B'^T dy per direction:
//   dx_t   = bf16( dx_base_t + sum_j w_tj s_j A'^T u ),   dw_tj = s_j < u , A'_j x_t >.
#pragma once
#include <cooperative_groups.h>

#include "apply_common.cuh"
#include "mma.cuh"

namespace lf {

constexpr int kMixMaxK = 16;
constexpr int kMixMaxRows = kMixMaxK * kMaxRank;   // directions of one token
constexpr int kMixThreads = 256;
constexpr int kMixWarps = kMixThreads / 32;
constexpr int kMixTile = 16;       // directions of one shrink tile (the rows of a matrix instruction)

struct MixProj {
    const __nv_bfloat16* x;      // rows of x_ld
    const __nv_bfloat16* in2;    // forward: base (nullable: zeros), rows of out_ld; gradient: dy, rows of dy_ld
    const __nv_bfloat16* base;   // gradient: dx_base (nullable: zeros)
    __nv_bfloat16* out;          // forward: y; gradient: dx (nullable)
    int64_t x_ld, dy_ld, out_ld, y_off;
    int32_t d_in, d_out, max_rank;
    int32_t slot;                // gradient: which partial weight gradient is the projection's
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
    float t[kMixMaxRows];                       // forward: coef * A' x; gradient: A' x
    float u[kMixMaxRows];                       // gradient: B'^T dy
    float tc[kMixMaxRows];                      // gradient: coef * B'^T dy
    float part[2][kMixMaxRows];                 // this CTA's share of t and u (read by the cluster)
    int32_t k[kMixMaxK], first[kMixMaxK + 1];
    int64_t soa[kMixMaxK], sob[kMixMaxK];
    float sc[kMixMaxK], w[kMixMaxK];
    float red[kMixThreads * 8];                 // shrink pieces; expand partial sums of the row groups
};

// part[r] = sum over [d0, d1) of v[d] * pool[off[r] + d], for r in [0, R): tiles of 16 rows on
// mma.sync m16n8k16 (rows = the 16-row operand, the vector in all eight columns), so that no
// value is converted: an fp32 multiply-add per element took 2.5 instructions each, and their
// issue bound the kernel.  Lane t of a row's four takes 16 bytes (8 elements) of each 32; the
// order of k inside a step is that of the loads on both sides.  Warps share the tiles' ranges
// in S pieces, added in order.  d0, d1 multiples of 8.
__device__ __forceinline__ void mix_shrink(const __nv_bfloat16* v, const __nv_bfloat16* pool, const int64_t* off, int R,
                                           int d0, int d1, float* red, float* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tiles = (R + kMixTile - 1) / kMixTile;
    const int units = (d1 - d0 + 31) >> 5;
    const int S = tiles >= kMixWarps ? 1 : (tiles > 1 ? kMixWarps / tiles : kMixWarps);   // pieces per tile
    const int per = S == 1 ? units : (units + S - 1) / S;
    for (int un = warp; un < tiles * S; un += kMixWarps) {
        const int tile = S == 1 ? un : un / S, q = un - tile * S;
        const __nv_bfloat16* ra = pool + off[min(tile * kMixTile + g, R - 1)] + d0 + 8 * t;
        const __nv_bfloat16* rb = pool + off[min(tile * kMixTile + 8 + g, R - 1)] + d0 + 8 * t;
        const __nv_bfloat16* rv = v + d0 + 8 * t;
        const int e = min(units, (q + 1) * per), len = d1 - d0 - 8 * t;   // this lane's elements end at len
        // the tensor core's running sum drops what falls below it, so four units are summed there
        // and added in registers, whose additions round
        float s0 = 0.f, s1 = 0.f;
        for (int u = q * per; u < e; u += 4) {
            uint4 a[4], b[4], x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = b[i] = x[i] = make_uint4(0, 0, 0, 0);
                if (u + i < e && (u + i) * 32 < len) {
                    a[i] = __ldg(reinterpret_cast<const uint4*>(ra + (u + i) * 32));
                    b[i] = __ldg(reinterpret_cast<const uint4*>(rb + (u + i) * 32));
                    x[i] = __ldg(reinterpret_cast<const uint4*>(rv + (u + i) * 32));
                }
            }
            float acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo[4] = {a[i].x, b[i].x, a[i].y, b[i].y}, hi[4] = {a[i].z, b[i].z, a[i].w, b[i].w};
                if (i == 0) mma_16816_0(acc, lo, x[i].x, x[i].y);
                else mma_16816(acc, lo, x[i].x, x[i].y);
                mma_16816(acc, hi, x[i].z, x[i].w);
            }
            s0 += acc[0];
            s1 += acc[2];
        }
        if (t == 0) {
            red[un * kMixTile + g] = s0;
            red[un * kMixTile + 8 + g] = s1;
        }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += kMixThreads) {
        const int tile = r / kMixTile;
        float s = 0.f;
        for (int q = 0; q < S; ++q) s += red[(tile * S + q) * kMixTile + r % kMixTile];
        part[r] = s;
    }
    __syncthreads();
}

// out[c0 .. c1) = bf16(base + sum_r tc[r] pool[off[r] + c]).  Threads cover 8-column vectors; a
// narrow range is covered by several groups of threads that share the rows, summed through
// shared memory in group order.
__device__ __forceinline__ void mix_expand(const float* tc, const __nv_bfloat16* pool, const int64_t* off, int R,
                                           const __nv_bfloat16* base, __nv_bfloat16* out, int c0, int c1, float* red) {
    const int tid = threadIdx.x;
    const int nvec = (c1 - c0) >> 3;
    int RG = 1, nv = kMixThreads;   // row groups, threads per group
    while (RG < 16 && nv / 2 >= nvec && 2 * RG <= R) {
        RG *= 2;
        nv /= 2;
    }
    const int rg = tid / nv, vt = tid - rg * nv;
    for (int v0 = 0; v0 < nvec; v0 += nv) {
        const bool on = v0 + vt < nvec;
        const int c = c0 + 8 * (on ? v0 + vt : 0);
        float2 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
        uint4 bv = make_uint4(0, 0, 0, 0);
        if (rg == 0 && base && on) bv = *reinterpret_cast<const uint4*>(base + c);
        if (on) {
#pragma unroll 8
            for (int r = rg; r < R; r += RG) {
                const uint4 pv = __ldg(reinterpret_cast<const uint4*>(pool + off[r] + c));
                const uint32_t w[4] = {pv.x, pv.y, pv.z, pv.w};
                const float2 tv = make_float2(tc[r], tc[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] = ffma2(tv, make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), acc[i]);
            }
        }
        if (RG > 1) {   // uniform
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                red[2 * i * kMixThreads + tid] = acc[i].x;
                red[(2 * i + 1) * kMixThreads + tid] = acc[i].y;
            }
            __syncthreads();
            if (rg == 0)
                for (int q = 1; q < RG; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i].x += red[2 * i * kMixThreads + q * nv + vt];
                        acc[i].y += red[(2 * i + 1) * kMixThreads + q * nv + vt];
                    }
            __syncthreads();
        }
        if (rg == 0 && on) {
            float bf[8];
            bf16x8_to_f32(bv, bf);
            uint4 o;
            __nv_bfloat162* y = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __floats2bfloat162_rn(bf[2 * i] + acc[i].x, bf[2 * i + 1] + acc[i].y);
            *reinterpret_cast<uint4*>(out + c) = o;
        }
    }
}

__device__ __forceinline__ int mix_cut(int d, int part, int parts) {   // multiples of 8
    if (parts == 1) return part * d;
    return (int)((uint32_t)(d >> 3) * (uint32_t)part / (uint32_t)parts) * 8;   // d / 8 * 8 fits
}

// Token-parallel form.  Cluster of CS CTAs per (token, projection): each takes a piece of
// d_in for the shrink, the pieces' sums are added over distributed shared memory in rank
// order, and each then writes its piece of the output columns.  CS grows as the batch
// shrinks, so that one token of one projection still spreads over 8 SMs; large batches use
// single CTAs.
template <bool GRAD>
__global__ void __launch_bounds__(kMixThreads, 3) mixture_token_kernel(const __grid_constant__ MixArgs a) {
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
        if (CS == 1) {
            v = s.part[h][r];
        } else {
            for (int c = 0; c < CS; ++c) v += cl.map_shared_rank(&s.part[h][r], c)[0];
        }
        if (GRAD) {
            (h ? s.u : s.t)[r] = v;
            if (h) s.tc[r] = s.coef[r] * v;
        } else {
            s.t[r] = s.coef[r] * v;
        }
    }
    __syncthreads();
    if (GRAD) {
        if (rank == 0 && a.gw) {
            for (int j = tid >> 5; j < a.K; j += kMixWarps) {
                float d = 0.f;
                for (int r = s.first[j] + (tid & 31); r < s.first[j + 1]; r += 32) d = fmaf(s.t[r], s.u[r], d);
                d = warp_sum(d);
                if ((tid & 31) == 0) a.gw[((int64_t)P.slot * a.T + tok) * a.K + j] = s.sc[j] * d;
            }
        }
        if (P.out) {
            const __nv_bfloat16* base = P.base ? P.base + (int64_t)tok * P.out_ld : nullptr;
            __nv_bfloat16* out = P.out + (int64_t)tok * P.out_ld;
            if (R > 0 || base != out)
                mix_expand(s.tc, P.A_pool, s.oa, R, base, out, mix_cut(P.d_in, rank, CS),
                           mix_cut(P.d_in, rank + 1, CS), s.red);
        }
    } else {
        const int64_t at = (int64_t)tok * P.out_ld + P.y_off;
        const __nv_bfloat16* base = P.in2 ? P.in2 + at : nullptr;
        if (R > 0 || base != P.out + at)
            mix_expand(s.t, P.Bt_pool, s.ob, R, base, P.out + at, mix_cut(P.d_out, rank, CS),
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
