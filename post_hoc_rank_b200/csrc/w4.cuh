// Base weights in 4 bits with group scales: quantisation, its inverse, and the product
//   y = bf16( bias + sum_g s_g sum_{i in g} (q_i - z_g) x_i )
// of a token batch with them: the W0 x of "Compress then Serve" (academ.us/article/
// 2407.00066), section 3, that the LoRA side path adds to, at a quarter of the bytes.
//
// Format: q holds d_out rows of d_in / 2 bytes, column 2 c in the low nibble of byte c;
// scales (bf16) and zero points (one byte each, 0 .. 15; absent = 8) are d_out x ng,
// ng = ceil(d_in / group) (the last group may be short).  A weight is (q - z) * s.
#pragma once
#include <cuda.h>   // CUtensorMap (type only)
#include <cuda_fp16.h>

#include "apply_common.cuh"
#include "router.cuh"
#include "tc.cuh"

namespace lf {

// ---- quantisation ------------------------------------------------------------------------
// Symmetric: s = bf16(max|w| / 7), z = 8.  With zero points: lo = min(w, 0), hi = max(w, 0),
// s = bf16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15).  q = clamp(rint(w / s) + z, 0, 15)
// with the rounded s; every rint is of the exact quotient, halves to even.
// G / 8 lanes per group, 8 weights each: one 16- or 32-byte read and one 4-byte write per
// lane, the group's extremes by shuffles.  Bound by the read of W (a bf16 18944 x 3584
// matrix: 136 MB in, 36 MB out, 26 us).

// rint(w / s) for s >= 2^-100 and |w / s| < 2^6, inv = 1 / s: w * inv is within 2^-22 |w / s| of
// the quotient, so only a product next to a half can round the wrong way; the sign of
// w - (q +- 1/2) s settles that exactly (one fma: the product is exact inside it).
__device__ __forceinline__ float rint_quotient(float w, float s, float inv) {
    const float t = w * inv;
    float q = rintf(t);
    if (fabsf(fabsf(t - q) - 0.5f) < 0x1p-12f) {
        const float up = fmaf(-(q + 0.5f), s, w), dn = fmaf(-(q - 0.5f), s, w);
        const bool odd = ((int)q & 1) != 0;
        if (up > 0.f || (up == 0.f && odd)) q += 1.f;
        else if (dn < 0.f || (dn == 0.f && odd)) q -= 1.f;
    }
    return q;
}

// bf16(num / den) of the exact quotient (num exact in fp64): fp32 division unless that
// lands next to the middle of two bf16 values.
__device__ __forceinline__ float bf16_quotient(float hi, float lo, float den) {
    float f = (hi - lo) / den;
    const uint32_t low = __float_as_uint(f) & 0xffffu;
    if (!(f < 1e38f) || f < 1e-37f || (low >= 0x7ff0u && low <= 0x8010u))
        f = (float)(((double)hi - (double)lo) / (double)den);
    return __bfloat162float(__float2bfloat16_rn(f));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(p)), v);
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

struct W4QuantArgs {
    const void* W;          // d_out x d_in
    int32_t d_out, d_in, ng;
    uint8_t* q;             // d_out x d_in / 2
    __nv_bfloat16* scales;  // d_out x ng
    uint8_t* zeros;         // nullable (symmetric)
};

// CTA per row, blockDim a multiple of 32.
template <typename T, int G>
__global__ void __launch_bounds__(256) w4_quantize_kernel(W4QuantArgs a) {
    constexpr int L = G / 8;   // lanes per group
    const int64_t row = blockIdx.x;
    const T* src = reinterpret_cast<const T*>(a.W) + row * a.d_in;
    uint8_t* dst = a.q + row * (a.d_in >> 1);
    const int sub = threadIdx.x % L;
    const int n8 = a.d_in >> 3;
    const int n8r = (n8 + 31) & ~31;   // whole warps walk the row: the shuffles below see every lane
    for (int p = threadIdx.x; p < n8r; p += blockDim.x) {
        float v[8];
        const bool in = p < n8;
        if (in) {
            load8<T>(src + 8 * p, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
        float lo = 0.f, hi = 0.f, chk = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            chk = fmaf(v[i], 0.f, chk);   // NaN once a value is not finite
        }
        if (chk != 0.f) {
            latch_error(LF_ERR_NUMERIC);
            lo = hi = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!(fabsf(v[i]) < INFINITY)) v[i] = 0.f;
                lo = fminf(lo, v[i]);
                hi = fmaxf(hi, v[i]);
            }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        float s, z;
        if (a.zeros) s = bf16_quotient(hi, lo, 15.f);
        else s = bf16_quotient(fmaxf(hi, -lo), 0.f, 7.f);
        uint32_t w;
        if (s >= 0x1p-100f) {
            const float inv = 1.f / s;
            z = a.zeros ? fminf(fmaxf(rint_quotient(-lo, s, inv), 0.f), 15.f) : 8.f;
            w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = fminf(fmaxf(rint_quotient(v[i], s, inv) + z, 0.f), 15.f);
                w |= __float_as_uint(q + 8388608.f) << (4 * i);   // 2^23 + q: the integer in the low bits
                if (i < 7) w &= (1u << (4 * i + 4)) - 1u;
            }
        } else {   // 1 / s may overflow, and s may be 0
            z = a.zeros ? (s > 0.f ? (float)fmin(fmax(rint(-(double)lo / (double)s), 0.0), 15.0) : 0.f) : 8.f;
            w = 0;
            for (int i = 0; i < 8; ++i) {
                const double q = s > 0.f ? rint((double)v[i] / (double)s) : 0.0;
                w |= (uint32_t)fmin(fmax(q + (double)z, 0.0), 15.0) << (4 * i);
            }
        }
        if (in) {
            *reinterpret_cast<uint32_t*>(dst + 4 * p) = w;
            if (sub == 0) {
                const int64_t gi = row * a.ng + p / L;
                a.scales[gi] = __float2bfloat16_rn(s);   // exact: s is a bf16 value
                if (a.zeros) a.zeros[gi] = (uint8_t)z;
            }
        }
    }
}

// W = (q - z) * s, one rounding to the output type (none for fp32: 13 significant bits).
struct W4DequantArgs {
    const uint8_t* q;
    const __nv_bfloat16* scales;
    const uint8_t* zeros;
    int32_t d_out, d_in, ng, log_g;
    void* W;
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&v)[8]) {
    uint4 u;
    __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
}

template <typename T>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(W4DequantArgs a) {
    const int64_t row = blockIdx.x;   // CTA per row
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + row * (a.d_in >> 1));
    T* dst = reinterpret_cast<T*>(a.W) + row * a.d_in;
    const int n8 = a.d_in >> 3;
#pragma unroll 2
    for (int p = threadIdx.x; p < n8; p += blockDim.x) {
        const int64_t gi = row * a.ng + (p >> (a.log_g - 3));
        const uint32_t w = __ldg(src + p);
        const float s = __bfloat162float(a.scales[gi]);
        const float z = 8388608.f + (float)(a.zeros ? (a.zeros[gi] & 15) : 8);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (__uint_as_float(((w >> (4 * j)) & 15u) | 0x4B000000u) - z) * s;
        store8<T>(dst + 8 * p, v);
    }
}

// ---- product, few tokens -----------------------------------------------------------------
// CTA (32 rows of one projection, 8 NT tokens): eight warps take the 256-column blocks of d_in
// in turn and add up through shared memory in warp order.  Each warp streams its blocks
// through a private ring of TMA stages (one box of 32 rows x 128 bytes each, 128-byte
// swizzle, no block barriers), unpacks to bf16 and multiplies with mma.sync m16n8k16
// (weights = the 16-row operand, tokens = the 8 columns): one product feeds up to 8 tokens.
// The reads bound it; what competes is the instructions of unpacking, about 60 per 512
// bytes and warp, so the kernel spends none on anything else it can leave out:
//  - a lane's 32-bit word gives nibbles i and i + 4 as a bf16 pair 128 + q by one mask (the
//    columns of the product are permuted alike for x), and the 128 + z to subtract is taken
//    out of the group's sum, sum (128 + q) x - (128 + z) sum x, instead of 4 subtractions per
//    word; sum x comes from a product with ones, in the same accumulator layout.  Products
//    and both sums are fp32; the difference loses at most the 5 bits that 128 + q is larger
//    than q - z, far below the output's rounding (2^-19 of sum |w| |x|).
//  - with groups of 128 or more columns, lane t of a row takes the 16 bytes of unit t (32
//    weights) of four, one 16-byte load for 4 words (WIDE); smaller groups, which end inside
//    that, take word t of every unit.
constexpr int kW4Warps = 8;
constexpr int kW4Rows = 32;            // rows per CTA
constexpr int kW4Depth = 3;            // stages of 4 KB per warp
constexpr int kW4MaxProj = 8;
constexpr uint32_t kW4StageBytes = kW4Rows * 128;

struct W4Proj {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const __nv_bfloat16* scales;
    const uint8_t* zeros;          // nullable: 8
    const __nv_bfloat16* bias;     // nullable
    int64_t x_ld, y_ld;
    int32_t d_in, d_out, ng, log_u;   // log_u: log2(units per group)
    int32_t tile0, pad;               // first row tile of the projection in the grid
};
struct W4Args {
    int32_t T, n_proj;
    W4Proj p[kW4MaxProj];
};
struct alignas(64) W4Maps {
    CUtensorMap q[kW4MaxProj];     // d_out rows of d_in / 2 bytes, box 128 bytes x 32 rows, 128-byte swizzle
};

// bf16x2 of (128 + nibble i, 128 + nibble i + 4)
template <int I>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)), "r"(0x000F000Fu), "r"(0x43004300u));
    return r;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int NT>
struct W4Smem {
    union {
        unsigned char ring[kW4Warps][kW4Depth][kW4StageBytes];   // 1024-byte aligned stages
        float part[kW4Warps][kW4Rows][8 * NT + 1];
    };
    uint64_t full[kW4Warps][kW4Depth];
};

// State of one warp's sums over its columns: two 16-row tiles, NT token tiles.
template <int NT>
struct W4Acc {
    float acc[2][NT][4], part[2][NT][4], xs[NT][4];
    float sc[2][2], zf[2][2];   // scale and 128 + z of rows 16 m + 8 h + (this lane's row)
    int grp;

    __device__ __forceinline__ void clear() {
        grp = -1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xs[n][i] = 0.f;
                acc[0][n][i] = acc[1][n][i] = part[0][n][i] = part[1][n][i] = 0.f;
            }
    }
    // end of a group: acc += s (sum (128 + q) x - (128 + z) sum x)
    __device__ __forceinline__ void flush() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[m][n][i] = fmaf(sc[m][i >> 1], fmaf(-zf[m][i >> 1], xs[n][i], part[m][n][i]), acc[m][n][i]);
                    part[m][n][i] = 0.f;
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) xs[n][i] = 0.f;
        }
    }
    // one word of each of the lane's four rows against 8 columns of x
    __device__ __forceinline__ void product(const uint32_t (&w)[2][2], const uint4 (&xv)[NT]) {
        const uint32_t one[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            b[n][0] = __byte_perm(xv[n].x, xv[n].z, 0x5410);   // (x0, x4)
            b[n][1] = __byte_perm(xv[n].x, xv[n].z, 0x7632);   // (x1, x5)
            b[n][2] = __byte_perm(xv[n].y, xv[n].w, 0x5410);   // (x2, x6)
            b[n][3] = __byte_perm(xv[n].y, xv[n].w, 0x7632);   // (x3, x7)
            mma_16816(xs[n], one, b[n][0], b[n][1]);
            mma_16816(xs[n], one, b[n][2], b[n][3]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t lo[4] = {nibble_pair<0>(w[m][0]), nibble_pair<0>(w[m][1]), nibble_pair<1>(w[m][0]),
                                    nibble_pair<1>(w[m][1])};
            const uint32_t hi[4] = {nibble_pair<2>(w[m][0]), nibble_pair<2>(w[m][1]), nibble_pair<3>(w[m][0]),
                                    nibble_pair<3>(w[m][1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16816(part[m][n], lo, b[n][0], b[n][1]);
                mma_16816(part[m][n], hi, b[n][2], b[n][3]);
            }
        }
    }
};

template <int NT, bool WIDE>
__global__ void __launch_bounds__(32 * kW4Warps, 2) w4_gemv_kernel(const __grid_constant__ W4Args a,
                                                                   const __grid_constant__ W4Maps maps) {
    extern __shared__ __align__(1024) unsigned char w4_raw[];
    auto& sm = *reinterpret_cast<W4Smem<NT>*>(w4_raw);
    int pi = 0;
#pragma unroll
    for (int i = 1; i < kW4MaxProj; ++i)
        if (i < a.n_proj && (int)blockIdx.x >= a.p[i].tile0) pi = i;
    const W4Proj& P = a.p[pi];
    const int row0 = ((int)blockIdx.x - P.tile0) * kW4Rows;
    const int tok0 = blockIdx.y * 8 * NT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int units = P.d_in >> 5;
    const int nblk = (units + 7) >> 3;                               // blocks of 8 units
    const int n_st = nblk > warp ? (nblk - warp + kW4Warps - 1) / kW4Warps : 0;
    uint64_t* full = sm.full[warp];
    if (lane == 0) {
        for (int i = 0; i < kW4Depth; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    auto issue = [&](int st) {   // lane 0: block warp + 8 st of the rows into its ring slot
        if (st < n_st) {
            uint64_t* bar = &full[st % kW4Depth];
            mbar_arrive_expect_tx(bar, kW4StageBytes);
            tc::tma_load_2d(sm.ring[warp][st % kW4Depth], &maps.q[pi], (warp + kW4Warps * st) * 128, row0, bar);
        }
    };
    if (lane == 0)
        for (int st = 0; st < kW4Depth; ++st) issue(st);
    __syncwarp();

    // lane's row of a tile: rows of neighbouring g differ in bit 2, so that the 16-byte loads of
    // 8 lanes (two rows) fall on distinct banks of the swizzled stage
    const int rg = (g >> 1) | ((g & 1) << 2);
    W4Acc<NT> A;
    A.clear();
    const __nv_bfloat16* xr[NT];
    bool live[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        live[n] = tok0 + 8 * n + g < a.T;
        xr[n] = P.x + (int64_t)(live[n] ? tok0 + 8 * n + g : 0) * P.x_ld;
    }
    // scale and zero point of row row0 + lane in group `grp` (rows past the last: any)
    const int64_t srow = (int64_t)min(row0 + lane, P.d_out - 1) * P.ng;
    auto enter_group = [&](int grp) {
        if (A.grp >= 0) A.flush();
        A.grp = grp;
        const uint32_t s16 = __bfloat16_as_ushort(P.scales[srow + grp]);
        const uint32_t z = P.zeros ? (P.zeros[srow + grp] & 15u) : 8u;
        const uint32_t sz = (s16 << 16) | z;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t v = __shfl_sync(0xffffffffu, sz, 16 * m + 8 * h + rg);
                A.sc[m][h] = __uint_as_float(v & 0xffff0000u);
                A.zf[m][h] = 128.f + (float)(v & 15u);
            }
    };
    bool ok = true;
    for (int st = 0; st < n_st; ++st) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[st % kW4Depth], (uint32_t)((st / kW4Depth) & 1)));
        if (!ok) break;   // uniform; the timeout is latched
        const unsigned char* src = sm.ring[warp][st % kW4Depth];
        const int u0 = (warp + kW4Warps * st) * 8;
        if (WIDE) {
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                if (u0 + 4 * sb >= units) break;   // uniform
                const int grp = (u0 + 4 * sb) >> P.log_u;
                if (grp != A.grp) enter_group(grp);
                uint4 q[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        q[m][h] = *reinterpret_cast<const uint4*>(src + (16 * m + 8 * h + rg) * 128 +
                                                                  (((4 * sb + t) ^ rg) << 4));
                const bool in = u0 + 4 * sb + t < units;
                const int k = (u0 + 4 * sb + t) * 32;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 xv[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        xv[n] = make_uint4(0, 0, 0, 0);
                        if (live[n] && in) xv[n] = __ldg(reinterpret_cast<const uint4*>(xr[n] + k + 8 * i));
                    }
                    uint32_t w[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            w[m][h] = i == 0 ? q[m][h].x : i == 1 ? q[m][h].y : i == 2 ? q[m][h].z : q[m][h].w;
                    A.product(w, xv);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (u0 + k >= units) break;   // uniform
                const int grp = (u0 + k) >> P.log_u;
                if (grp != A.grp) enter_group(grp);
                uint4 xv[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    xv[n] = make_uint4(0, 0, 0, 0);
                    if (live[n]) xv[n] = __ldg(reinterpret_cast<const uint4*>(xr[n] + (u0 + k) * 32 + t * 8));
                }
                uint32_t w[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[m][h] = *reinterpret_cast<const uint32_t*>(src + (16 * m + 8 * h + rg) * 128 + ((k ^ rg) << 4) +
                                                                     4 * t);
                A.product(w, xv);
            }
        }
        __syncwarp();   // the stage has been read
        if (lane == 0) issue(st + kW4Depth);
    }
    if (A.grp >= 0) A.flush();
    if (!ok && lane == 0)   // no copy of this warp is in flight when the ring is reused or the CTA leaves
        for (int st = 0; st < n_st; ++st) mbar_wait(&full[st % kW4Depth], (uint32_t)((st / kW4Depth) & 1));
    if (!__syncthreads_and(ok)) return;   // the ring becomes the partial sums
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sm.part[warp][16 * m + 8 * (i >> 1) + rg][8 * n + 2 * t + (i & 1)] = A.acc[m][n][i];
    __syncthreads();
    for (int o = tid; o < kW4Rows * 8 * NT; o += 32 * kW4Warps) {
        const int r = o % kW4Rows, n = o / kW4Rows;
        if (row0 + r >= P.d_out || tok0 + n >= a.T) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) v += sm.part[w][r][n];
        if (P.bias) v += __bfloat162float(P.bias[row0 + r]);
        P.y[(int64_t)(tok0 + n) * P.y_ld + row0 + r] = __float2bfloat16_rn(v);
    }
}

}  // namespace lf
