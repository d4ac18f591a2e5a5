// Routed LoRA side path of a long batch over a small pool, as two dense tcgen05 products.
//
// With all experts' rows stacked, A (R x d_in) and B^T (R x d_out), R = sum of the retained
// ranks, a token's weighted update is y = base + (W o (A x)) B^T, where W[t][r] = sum_j
// [e_tj = expert of row r] w_tj s_j is zero outside the token's experts.  Taking all R rows
// costs R / (K k) times the operations the token needs, but they run on the tensor cores and
// every factor row is read once per 128 tokens; the token-parallel form reads K k rows per
// token from L2, which bounds it (16 experts of rank 16, 2 per token, 8192 tokens of 3584 x
// 3584: 386 us token by token).
//
//   pack    the experts' rows into one matrix each (pools may hold them anywhere), so that TMA
//           fetches tiles of them; rows past R are zero
//   shrink  S = X A^T: 128 tokens x up to 256 rows per CTA, d_in shared by a cluster; the sum
//           over the cluster (rank order) is weighted and split into two bf16 values
//           (P_hi + P_lo, 16 significant bits), and / or stored raw
//   expand  Y = base + P_hi B^T + P_lo B^T: 128 tokens x 256 columns per tile, persistent
// The gradient for x is the same pair with the factors exchanged (U = dY B, dX = (W o U) A), and
// the weights' gradient is s_j <S, U> over the expert's rows (raw S and U).
#pragma once
#include <cooperative_groups.h>
#include <cuda.h>   // CUtensorMap (type only)

#include "mixture.cuh"
#include "tc.cuh"

namespace lf {

constexpr int kMtRows = 1024;      // most stacked rows (a multiple of 256)
constexpr int kMtM = 128;          // tokens per tile
constexpr int kMtN = 256;          // stacked rows (shrink) or output columns (expand) per tile
constexpr int kMtKB = 64;          // columns or rows per stage

// Tables of one projection's stacked rows, in the workspace.
struct MixPlan {
    int32_t R;                     // stacked rows
    int32_t pad[15];
    int32_t first[kMtRows + 1];    // per adapter (at most kMtRows of them with any rank): first stacked row
    int32_t rank[kMtRows];         // retained rank, 0 for one that fails the checks
    int32_t err[kMtRows];          // its error (latched by the tokens that use it)
    int32_t bad[2][kMtRows];       // per stacked row: its A, its B^T row holds a value that is not finite
};

struct MixPackArgs {
    int32_t n_adapters, max_rank, d_in, d_out, Rp;   // Rp: rows of the packed matrices (zeros past R)
    const int32_t* ranks;
    const int64_t* off_A;
    const int64_t* off_Bt;
    const __nv_bfloat16* A_pool;
    const __nv_bfloat16* Bt_pool;
    int64_t pool_A, pool_Bt;
    MixPlan* plan;
    __nv_bfloat16* A;              // Rp x d_in
    __nv_bfloat16* Bt;             // Rp x d_out
};

// CTA (stacked row, grid.y = 0: A, 1: B^T).  Each CTA finds its row's adapter by a block-wide
// scan of the ranks (at most kMtRows), so that one launch plans and copies.
__global__ void __launch_bounds__(256) mixture_pack_kernel(MixPackArgs a) {
    __shared__ int32_t first[kMtRows + 1];
    __shared__ int32_t wsum[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int e0 = 0; e0 < a.n_adapters; e0 += 256) {
        const int e = e0 + tid;
        int k = 0, err = 0;
        if (e < a.n_adapters) {
            k = a.ranks[e];
            const int64_t oa = a.off_A[e], ob = a.off_Bt[e];
            if (k > kMaxRank || (a.max_rank > 0 && k > a.max_rank)) err = LF_ERR_SHAPE;
            else if (k > 0 && ((oa & 7) || (ob & 7))) err = LF_ERR_ALIGNMENT;
            else if (k > 0 && (oa < 0 || ob < 0 || oa > a.pool_A - (int64_t)k * a.d_in || ob > a.pool_Bt - (int64_t)k * a.d_out))
                err = LF_ERR_WORKSPACE;
            if (err || k < 0) k = 0;
        }
        int x = k;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        int base = carry, tot = 0;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) base += wsum[w];
            tot += wsum[w];
        }
        if (e < a.n_adapters) {
            first[e] = base + x - k;
            if (blockIdx.x == 0 && blockIdx.y == 0) {
                a.plan->first[e] = base + x - k;
                a.plan->rank[e] = k;
                a.plan->err[e] = err;
            }
        }
        carry += tot;
        __syncthreads();
    }
    const int R = carry, r = blockIdx.x;
    if (tid == 0) {
        first[a.n_adapters] = R;
        if (r == 0 && blockIdx.y == 0) {
            a.plan->R = R;
            a.plan->first[a.n_adapters] = R;
        }
    }
    __syncthreads();
    const bool is_a = blockIdx.y == 0;
    const int d = is_a ? a.d_in : a.d_out;
    uint4* dst = reinterpret_cast<uint4*>((is_a ? a.A : a.Bt) + (int64_t)r * d);
    if (r >= R) {
        if (tid == 0) a.plan->bad[blockIdx.y][r] = 0;
        for (int c = tid; c < d / 8; c += 256) dst[c] = make_uint4(0, 0, 0, 0);
        return;
    }
    int lo = 0, hi = a.n_adapters;   // first[lo] <= r < first[hi], lo the last such (empty ones share a start)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid;
        else hi = mid;
    }
    const int q = r - first[lo];
    const uint4* src = reinterpret_cast<const uint4*>(is_a ? a.A_pool + a.off_A[lo] + (int64_t)q * d
                                                           : a.Bt_pool + a.off_Bt[lo] + (int64_t)q * d);
    // Products of the other tokens with this row are 0 times its values: what is not finite is
    // packed as 0 and flagged, and the tokens that do use the row get NaN.
    bool bad = false;
    for (int c = tid; c < d / 8; c += 256) {
        uint4 u = __ldg(src + c);
        uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool b0 = (w[i] & 0x00007F80u) == 0x00007F80u, b1 = (w[i] & 0x7F800000u) == 0x7F800000u;
            if (b0) w[i] &= 0xFFFF0000u;
            if (b1) w[i] &= 0x0000FFFFu;
            bad = bad || b0 || b1;
        }
        dst[c] = u;
    }
    const int any = __syncthreads_or(bad ? 1 : 0);
    if (tid == 0) a.plan->bad[blockIdx.y][r] = any ? 1 : 0;
}

struct MixShrinkArgs {
    int32_t T, K, n_adapters, d;   // d: columns contracted
    int32_t Rp;                    // row stride of the outputs
    int32_t report;                // latch bad ids and bad factors here
    const MixPlan* plan;
    const int32_t* ids;
    const float* weights;          // nullable: 1
    float scale;
    const float* scales;
    float* raw;                    // nullable: T x Rp
    __nv_bfloat16* hi;             // nullable: T x Rp, then lo
    __nv_bfloat16* lo;
};

constexpr int mt_shrink_stages(int nch) { return nch == 128 ? 6 : 4; }
constexpr int kMtABox = 32;        // stacked rows per copy: a chunk loads what it has, rounded up to this
template <int NCH>
struct MixShrinkSmem {
    static constexpr int kMtShrinkStages = mt_shrink_stages(NCH);
    union {
        struct {
            unsigned char x[kMtShrinkStages][kMtM * 128];
            unsigned char a[kMtShrinkStages][NCH * 128];
        };
        float part[kMtM][NCH + 4];
    };
    int32_t bad[NCH];
    // the tokens' slots: first stacked row of the expert less r0, its rank (0: nothing), weight
    // times scale; an expert named twice has one slot with the sum of its weights
    int16_t col[kMtM][kMixMaxK], rank[kMtM][kMixMaxK];
    float w[kMtM][kMixMaxK];
    uint64_t full[kMtShrinkStages], empty[kMtShrinkStages], dfull[2], dempty[2];
    uint32_t tmem;
    int32_t failed;
};
constexpr int kMtShrinkThreads = 320;   // warps 0-7 sums, 8 copies, 9 products
// The tensor core's running fp32 sum drops what falls below it, so an error grows with the number
// of products added up in one: after kMtSeg stages (16 products) the sum moves to registers, whose
// additions round (the weights' gradient of 8192 tokens of 3584 columns: 3.4e-6 off in norm with
// sums of 1792 columns, 4e-7 with 256, in the same time).
constexpr int kMtSeg = 4;

// xmap: T rows of d columns, box 64 x 128; amap: Rp rows of d columns, box 64 x 32; 128-byte
// swizzle both.  Grid: clusters of CS along x (shares of d), token tiles, y = chunks of NCH rows.
// NCH 256: x is read
// once for 256 rows; 128: twice the CTAs, where 256 leave most SMs idle.
template <int NCH>
__global__ void __launch_bounds__(kMtShrinkThreads, 1) mixture_shrink_kernel(const __grid_constant__ MixShrinkArgs a,
                                                                const __grid_constant__ CUtensorMap xmap,
                                                                const __grid_constant__ CUtensorMap amap) {
    namespace cg = cooperative_groups;
    constexpr int kMtShrinkStages = mt_shrink_stages(NCH);
    extern __shared__ __align__(1024) unsigned char mt_raw[];
    auto& s = *reinterpret_cast<MixShrinkSmem<NCH>*>(mt_raw);
    cg::cluster_group cl = cg::this_cluster();
    const int CS = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tok0 = ((int)blockIdx.x / CS) * kMtM, r0 = blockIdx.y * NCH;
    const int R = a.plan->R;
    if (r0 >= ((R + kMtKB - 1) & ~(kMtKB - 1)) && r0 > 0) return;   // uniform over the cluster: no rows here
    const int n = min(NCH, (max(R - r0, 1) + 15) & ~15);     // rows of this chunk, for the products
    const int nbox = (n + kMtABox - 1) / kMtABox;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int steps = (a.d + kMtKB - 1) / kMtKB;
    const int k0 = (int)((int64_t)steps * rank / CS), nk = (int)((int64_t)steps * (rank + 1) / CS) - k0;
    if (warp == 0) tc::tmem_alloc(&s.tmem, 2 * NCH);
    if (tid == 0) {
        for (int i = 0; i < kMtShrinkStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.dfull[i], 1);
            mbar_init(&s.dempty[i], 8);
        }
        s.failed = 0;
        fence_barrier_init();
    }
    if (tid < NCH) {
        const int r = min(r0 + tid, a.Rp - 1);
        s.bad[tid] = a.plan->bad[0][r] | a.plan->bad[1][r];
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s.tmem;
    bool ok = true;
    if (warp >= 4 && warp < 8) {   // a thread per token: its slots, while the products run
        const int m = tid - 128, t = tok0 + m;
        const bool lead = a.report && r0 == 0 && rank == 0;
        if ((a.hi || lead) && t < a.T) {
            int id[kMixMaxK];
#pragma unroll
            for (int j = 0; j < kMixMaxK; ++j) {
                id[j] = j < a.K ? a.ids[(int64_t)t * a.K + j] : -1;
                if (id[j] < -1 || id[j] >= a.n_adapters) {
                    if (lead) latch_error(LF_ERR_BAD_INDEX);
                    id[j] = -1;
                }
            }
#pragma unroll
            for (int j = 0; j < kMixMaxK; ++j) {
                if (j >= a.K) break;
                int k = 0, c = 0;
                float w = 0.f;
                if (id[j] >= 0) {
                    k = a.plan->rank[id[j]];
                    c = a.plan->first[id[j]] - r0;
                    if (k == 0 && lead && a.plan->err[id[j]]) latch_error(a.plan->err[id[j]]);
                    w = (a.weights ? a.weights[(int64_t)t * a.K + j] : 1.f) * (a.scales ? a.scales[id[j]] : a.scale);
#pragma unroll
                    for (int q = 0; q < kMixMaxK; ++q)   // into the expert's first slot
                        if (q < j && id[q] == id[j] && k > 0) {
                            s.w[m][q] += w;
                            k = 0;
                        }
                }
                s.col[m][j] = (int16_t)c;
                s.rank[m][j] = (int16_t)k;
                s.w[m][j] = w;
            }
        }
    }
    const int nseg = (nk + kMtSeg - 1) / kMtSeg;
    float acc[NCH / 2];   // columns NCH / 2 * (warp / 4) .. of row 32 (warp % 4) + lane
#pragma unroll
    for (int i = 0; i < NCH / 2; ++i) acc[i] = 0.f;
    if (warp == 8) {
        if (lane == 0) {
            int i = 0;
            for (; i < nk; ++i) {
                const int st = i % kMtShrinkStages;
                if (i >= kMtShrinkStages) ok = mbar_wait(&s.empty[st], (uint32_t)(i / kMtShrinkStages - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.full[st], (kMtM + nbox * kMtABox) * 128);
                tc::tma_load_2d(s.x[st], &xmap, (k0 + i) * kMtKB, tok0, &s.full[st]);
                for (int q = 0; q < nbox; ++q)
                    tc::tma_load_2d(s.a[st] + q * kMtABox * 128, &amap, (k0 + i) * kMtKB, r0 + q * kMtABox, &s.full[st]);
            }
            // nothing is in flight when the buffers are reused or the CTA leaves
            for (int j = max(0, i - kMtShrinkStages); j < i; ++j)
                ok = mbar_wait(&s.full[j % kMtShrinkStages], (uint32_t)(j / kMtShrinkStages) & 1) && ok;
        }
    } else if (warp == 9) {
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t idesc = tc::idesc_bf16(kMtM, n, 0, 0);
        const uint64_t xd0 = tc::smem_desc_sw128(s.x[0]), ad0 = tc::smem_desc_sw128(s.a[0]);
        for (int i = 0; i < nk; ++i) {
            const int st = i % kMtShrinkStages, g = i / kMtSeg;
            ok = mbar_wait(&s.full[st], (uint32_t)(i / kMtShrinkStages) & 1);
            if (i % kMtSeg == 0 && g >= 2) ok = ok && mbar_wait(&s.dempty[g & 1], (uint32_t)(g / 2 - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t xd = xd0 + (uint64_t)(st * (kMtM * 128 / 16)), ad = ad0 + (uint64_t)(st * (NCH * 128 / 16));
            const uint32_t d = tm + (uint32_t)((g & 1) * NCH);
#pragma unroll
            for (int k = 0; k < kMtKB / 16; ++k) tc::mma_bf16_warp(d, xd + 2 * k, ad + 2 * k, idesc, i % kMtSeg > 0 || k > 0);
            tc::commit_warp(&s.empty[st]);
            if (i % kMtSeg == kMtSeg - 1 || i == nk - 1) tc::commit_warp(&s.dfull[g & 1]);
        }
        if (ok && nseg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&s.dfull[(nseg - 1) & 1], (uint32_t)((nseg - 1) / 2) & 1));
    } else {
        const int c0 = (warp >> 2) * (NCH / 2);
        for (int g = 0; g < nseg; ++g) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s.dfull[g & 1], (uint32_t)(g / 2) & 1));
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < NCH / 2; c += 16) {
                if (c0 + c < n) {   // uniform
                    float v[16];
                    tc::tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)((g & 1) * NCH + c0 + c), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive1(&s.dempty[g & 1]);
        }
    }
    if (!ok) s.failed = 1;
    tc::fence_before_sync();
    __syncthreads();   // all products complete, all copies landed: the stages become the partial sums
    tc::fence_after_sync();
    if (warp < 8) {
        const int m = 32 * (warp & 3) + lane, c0 = (warp >> 2) * (NCH / 2);
#pragma unroll
        for (int c = 0; c < NCH / 2; c += 4)
            if (c0 + c < n) *reinterpret_cast<float4*>(&s.part[m][c0 + c]) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 2 * NCH);
    if (CS > 1) cl.sync();
    bool all_ok = s.failed == 0;
    for (int c = 0; c < CS && CS > 1; ++c) all_ok = all_ok && *cl.map_shared_rank(&s.failed, c) == 0;
    if (all_ok) {   // uniform over the cluster; a timeout is latched
        // this CTA's rows of the tile.  Raw sums and the zeros of P first, whole rows at a time;
        // the loads of a batch of pieces (remote shared memory among them) go out together
        const int rows = kMtM / CS, m0 = rank * rows;
        constexpr int V = NCH / 4, kBatch = 2;   // four-column pieces per row
        for (int i0 = tid; i0 < rows * V; i0 += kMtShrinkThreads * kBatch) {
            float4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q0 = 0; q0 < CS && a.raw; q0 += 4) {
                float4 p[4][kBatch];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const int i = i0 + kMtShrinkThreads * u, m = m0 + i / V, c = i % V * 4;
                        p[q][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (q0 + q < CS && i < rows * V && c < n && tok0 + m < a.T)
                            p[q][u] = *reinterpret_cast<const float4*>(CS > 1 ? cl.map_shared_rank(&s.part[m][c], q0 + q)
                                                                             : &s.part[m][c]);
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        v[u].x += p[q][u].x, v[u].y += p[q][u].y, v[u].z += p[q][u].z, v[u].w += p[q][u].w;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + kMtShrinkThreads * u, m = m0 + i / V, c = i % V * 4;
                if (i >= rows * V || r0 + c >= a.Rp || tok0 + m >= a.T) continue;
                const int64_t at = (int64_t)(tok0 + m) * a.Rp + r0 + c;
                if (a.raw) *reinterpret_cast<float4*>(a.raw + at) = v[u];
                if (a.hi) {
                    *reinterpret_cast<uint2*>(a.hi + at) = make_uint2(0u, 0u);
                    *reinterpret_cast<uint2*>(a.lo + at) = make_uint2(0u, 0u);
                }
            }
        }
        if (a.hi) {   // then the entries of the tokens' experts: eight lanes per slot
            __syncthreads();
            for (int i = tid >> 3; i < rows * a.K; i += kMtShrinkThreads / 8) {
                const int m = m0 + i / a.K, j = i % a.K;
                if (tok0 + m >= a.T) break;
                const int k = s.rank[m][j], cb = s.col[m][j];
                const float w = s.w[m][j];
                for (int c = max(cb, 0) + (tid & 7); c < min(cb + k, NCH); c += 8) {
                    float part[8], v = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        part[q] = q >= CS ? 0.f : (CS > 1 ? *cl.map_shared_rank(&s.part[m][c], q) : s.part[m][c]);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v += part[q];
                    const float p = s.bad[c] ? NAN : w * v;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(p);
                    const float h = __bfloat162float(hi);
                    const int64_t at = (int64_t)(tok0 + m) * a.Rp + r0 + c;
                    a.hi[at] = hi;
                    a.lo[at] = __float2bfloat16_rn(fabsf(h) < INFINITY ? p - h : 0.f);
                }
            }
        }
    }
    if (CS > 1) cl.sync();   // the parts are read by the whole cluster
}

struct MixExpandArgs {
    int32_t T, d;              // d: output columns
    int32_t has_base, pad;
    const MixPlan* plan;
};
constexpr int kMtExpandStages = 2;
struct MixExpandSmem {
    unsigned char p[kMtExpandStages][2][kMtM * 128];        // hi, lo: 128 tokens x 64 rows
    unsigned char b[kMtExpandStages][4][kMtKB * 128];       // 64 rows x 256 columns, four pieces of 64 columns
    unsigned char y[4][kMtM * 128];                         // 128 tokens x 256 columns, four pieces of 64 columns
    uint64_t full[kMtExpandStages], empty[kMtExpandStages], dfull[2], dempty[2], ybase[4];
    uint32_t tmem;
};
constexpr int kMtExpandThreads = 320;   // warps 0-7 epilogue, 8 copies, 9 products

// Persistent: CTA c takes tiles c, c + gridDim.x, .. (column tiles fastest, so that neighbours
// share P).  himap, lomap: T rows of Rp, box 64 x 128; bmap: Rp rows of d columns, box 64 x 64;
// basemap, ymap: T rows of d columns (the slice), box 64 x 128; 128-byte swizzle all.
__global__ void __launch_bounds__(kMtExpandThreads, 1)
    mixture_expand_kernel(const __grid_constant__ MixExpandArgs a, const __grid_constant__ CUtensorMap himap,
                          const __grid_constant__ CUtensorMap lomap, const __grid_constant__ CUtensorMap bmap,
                          const __grid_constant__ CUtensorMap basemap, const __grid_constant__ CUtensorMap ymap) {
    extern __shared__ __align__(1024) unsigned char mt_raw[];
    auto& s = *reinterpret_cast<MixExpandSmem*>(mt_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nkb = max(1, (a.plan->R + kMtKB - 1) / kMtKB);    // stages per tile (rows past R are zero)
    const int nct = (a.d + kMtN - 1) / kMtN, ntiles = nct * ((a.T + kMtM - 1) / kMtM);
    const int mine = ntiles > (int)blockIdx.x ? (ntiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
    if (warp == 0) tc::tmem_alloc(&s.tmem, 2 * kMtN);
    if (tid == 0) {
        for (int i = 0; i < kMtExpandStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.dfull[i], 1);
            mbar_init(&s.dempty[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&s.ybase[i], 1);
        fence_barrier_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s.tmem;
    bool ok = true;
    if (warp == 8) {   // ---- copies of P and B
        if (lane == 0) {
            int it = 0;
            for (int j = 0; j < mine && ok; ++j) {
                const int tile = (int)blockIdx.x + j * (int)gridDim.x;
                const int t0 = tile / nct * kMtM, c0 = tile % nct * kMtN;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int st = it % kMtExpandStages;
                    if (it >= kMtExpandStages) ok = mbar_wait(&s.empty[st], (uint32_t)(it / kMtExpandStages - 1) & 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s.full[st], 2 * kMtM * 128 + 4 * kMtKB * 128);
                    tc::tma_load_2d(s.p[st][0], &himap, kb * kMtKB, t0, &s.full[st]);
                    tc::tma_load_2d(s.p[st][1], &lomap, kb * kMtKB, t0, &s.full[st]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc::tma_load_2d(s.b[st][q], &bmap, c0 + 64 * q, kb * kMtKB, &s.full[st]);
                }
            }
            for (int i = max(0, it - kMtExpandStages); i < it; ++i)
                ok = mbar_wait(&s.full[i % kMtExpandStages], (uint32_t)(i / kMtExpandStages) & 1) && ok;
        }
    } else if (warp == 9) {   // ---- products
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t idesc = tc::idesc_bf16(kMtM, kMtN, 0, 1);
        const uint64_t pd0 = tc::smem_desc_sw128(s.p[0][0]), bd0 = tc::smem_desc_sw128_mn(s.b[0][0], kMtKB * 128);
        int it = 0;
        for (int j = 0; j < mine && ok; ++j) {
            if (j >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&s.dempty[j & 1], (uint32_t)(j / 2 - 1) & 1));
            for (int kb = 0; kb < nkb && ok; ++kb, ++it) {
                const int st = it % kMtExpandStages;
                ok = __all_sync(0xffffffffu, mbar_wait(&s.full[st], (uint32_t)(it / kMtExpandStages) & 1));
                if (!ok) break;
                tc::fence_after_sync();
                const uint64_t pd = pd0 + (uint64_t)(st * (2 * kMtM * 128 / 16)), bd = bd0 + (uint64_t)(st * (4 * kMtKB * 128 / 16));
#pragma unroll
                for (int k = 0; k < kMtKB / 16; ++k) {   // 16 rows of B: two groups of 8, 1 KB each
                    tc::mma_bf16_warp(tm + (uint32_t)((j & 1) * kMtN), pd + 2 * k, bd + 128 * k, idesc, kb > 0 || k > 0);
                    tc::mma_bf16_warp(tm + (uint32_t)((j & 1) * kMtN), pd + kMtM * 128 / 16 + 2 * k, bd + 128 * k, idesc, true);
                }
                tc::commit_warp(&s.empty[st]);
            }
            if (ok) tc::commit_warp(&s.dfull[j & 1]);
        }
        if (ok && mine > 0) ok = __all_sync(0xffffffffu, mbar_wait(&s.dfull[(mine - 1) & 1], (uint32_t)((mine - 1) / 2) & 1));
    } else {   // ---- epilogue: y = base + D by way of shared memory, 64 columns at a time in a ring of
               // four buffers, so that bases arrive and tiles leave while others are worked on
        const int m = 32 * (warp & 3) + lane, half = warp >> 2;
        const int nq = 4 * mine;   // quarters of tiles
        auto load_base = [&](int i) {   // thread 0
            const int tile = (int)blockIdx.x + (i >> 2) * (int)gridDim.x;
            mbar_arrive_expect_tx(&s.ybase[i & 3], kMtM * 128);
            tc::tma_load_2d(s.y[i & 3], &basemap, tile % nct * kMtN + 64 * (i & 3), tile / nct * kMtM, &s.ybase[i & 3]);
        };
        int loaded = 0;
        if (tid == 0 && a.has_base)
            for (; loaded < min(3, nq); ++loaded) load_base(loaded);
        for (int i = 0; i < nq; ++i) {
            const int j = i >> 2, tile = (int)blockIdx.x + j * (int)gridDim.x;
            if ((i & 3) == 0) ok = mbar_wait(&s.dfull[j & 1], (uint32_t)(j / 2) & 1);
            if (a.has_base) ok = ok && mbar_wait(&s.ybase[i & 3], (uint32_t)j & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc::fence_after_sync();
#pragma unroll
                for (int c16 = 0; c16 < 2; ++c16) {
                    const int c = 32 * half + 16 * c16;   // column of the quarter
                    float v[16];
                    tc::tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)((j & 1) * kMtN + 64 * (i & 3) + c), v);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4* p = reinterpret_cast<uint4*>(s.y[i & 3] + m * 128 + ((((c >> 3) + h) ^ (m & 7)) << 4));
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (a.has_base) u = *p;
                        __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float2 f = __bfloat1622float2(q[x]);
                            q[x] = __floats2bfloat162_rn(f.x + v[8 * h + 2 * x], f.y + v[8 * h + 2 * x + 1]);
                        }
                        *p = u;
                    }
                }
                if ((i & 3) == 3) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(&s.dempty[j & 1]);
                }
                tc::fence_proxy_async();
            }
            ok = tc::named_sync_and(1, 256, ok);
            if (!ok) break;   // the other warps' waits run out as well
            if (tid == 0) {
                tc::tma_store_2d(&ymap, tile % nct * kMtN + 64 * (i & 3), tile / nct * kMtM, s.y[i & 3]);
                tc::bulk_commit();
                tc::bulk_wait_read1();   // the store before has read its buffer, that of quarter i + 3
                if (a.has_base && i + 3 < nq) {
                    load_base(i + 3);
                    loaded = i + 4;
                }
            }
        }
        if (tid == 0) {   // nothing is in flight when the CTA leaves
            tc::bulk_wait0();
            for (int i = max(0, loaded - 4); i < loaded; ++i) mbar_wait(&s.ybase[i & 3], (uint32_t)(i >> 2) & 1);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 2 * kMtN);
}

// grad_weights[t][j] = s_j <S, U> over the stacked rows of the slot's expert; one warp per token.
struct MixDotArgs {
    int32_t T, K, n_adapters, Rp;
    const MixPlan* plan;
    const int32_t* ids;
    float scale;
    const float* scales;
    const float* S;
    const float* U;
    float* gw;
};
__global__ void __launch_bounds__(256) mixture_dot_kernel(MixDotArgs a) {
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.T) return;
    const int mine = lane < a.K ? a.ids[(int64_t)t * a.K + lane] : -1;
    for (int j = 0; j < a.K; ++j) {
        const int id = __shfl_sync(0xffffffffu, mine, j);
        float d = 0.f;
        if (id >= 0 && id < a.n_adapters) {
            const int64_t at = (int64_t)t * a.Rp + a.plan->first[id];
            const int k = a.plan->rank[id];
            for (int r = lane; r < k; r += 32) {
                const int row = a.plan->first[id] + r;
                d = a.plan->bad[0][row] | a.plan->bad[1][row] ? NAN : fmaf(a.S[at + r], a.U[at + r], d);
            }
            d *= a.scales ? a.scales[id] : a.scale;
        }
        d = warp_sum(d);
        if (lane == 0) a.gw[(int64_t)t * a.K + j] = d;
    }
}

}  // namespace lf
