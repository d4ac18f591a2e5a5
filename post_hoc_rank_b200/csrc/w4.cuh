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
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "apply_common.cuh"
#include "mma.cuh"
#include "router.cuh"
#include "tc.cuh"

namespace lf {

// ---- quantisation ------------------------------------------------------------------------
// Symmetric: s = bf16(max|w| / 7), z = 8.  With zero points: lo = min(w, 0), hi = max(w, 0),
// s = bf16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15).  q = clamp(rint(w / s) + z, 0, 15)
// with the rounded s; every rint is of the exact quotient, halves to even.  A scale is the bf16
// value of the fp32 quotient: rounded twice, as fp32 code that fits scales rounds it.
// G / 16 lanes per group, 16 weights each, the group's extremes by shuffles.  The read of W
// bounds it (a bf16 18944 x 3584 matrix: 136 MB in, 36 MB out, 26 us) if the instructions
// stay below it: scales by a product with a constant and quotients by a product with an
// approximate reciprocal, two columns per packed fp32 instruction, each followed by one test
// (per 16 weights) that sends what lies next to a border the exact way.

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
    return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kRintMagic = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, halves to even

// rint(w / s) for s >= 2^-100 and |w / s| < 2^6 from an integer q off by at most one: the
// residual w - q s is exact in one fma, and is compared with s / 2; halves go to even.
__device__ __forceinline__ float rint_quotient(float w, float s, float q) {
    const float e = fmaf(-q, s, w), a = fabsf(e), h = 0.5f * s;
    const bool odd = (__float_as_uint(q + kRintMagic) & 1u) != 0;
    return a > h || (a == h && odd) ? q + copysignf(1.f, e) : q;
}

// bf16(fp32((hi - lo) / den)): a product with 1 / den unless that lands next to the middle of two
// bf16 values (or near the ends of the range), where the quotient is formed in fp64 and rounded
// to fp32, then to bf16.
__device__ __forceinline__ float bf16_quotient(float hi, float lo, float den) {
    float f = (hi - lo) * (1.f / den);
    const uint32_t low = __float_as_uint(f) & 0xffffu;
    if (!(f < 1e38f) || f < 1e-37f || (low >= 0x7ff0u && low <= 0x8010u))
        f = (float)(((double)hi - (double)lo) / (double)den);
    return __bfloat162float(__float2bfloat16_rn(f));
}

// 16 consecutive weights as fp32 pairs, with their smallest and largest value (0 included);
// false when one is not finite.
__device__ __forceinline__ bool load16(const float* p, float2 (&v)[8], float& lo, float& hi) {
    float chk = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
        v[2 * i] = make_float2(a.x, a.y);
        v[2 * i + 1] = make_float2(a.z, a.w);
        lo = fminf(fminf(lo, fminf(a.x, a.y)), fminf(a.z, a.w));
        hi = fmaxf(fmaxf(hi, fmaxf(a.x, a.y)), fmaxf(a.z, a.w));
        chk = fmaf(a.x, 0.f, fmaf(a.y, 0.f, fmaf(a.z, 0.f, fmaf(a.w, 0.f, chk))));   // NaN once one is not finite
    }
    return chk == 0.f;
}
template <typename H2>   // __nv_bfloat162 or __half2
__device__ __forceinline__ bool load16_half(const void* p, float2 (&v)[8], float& lo, float& hi) {
    uint4 u[2] = {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1)};
    const H2* h = reinterpret_cast<const H2*>(u);
    H2 mn = h[0], mx = h[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn = __hmin2_nan(mn, h[i]);
        mx = __hmax2_nan(mx, h[i]);
    }
    float2 a, b;
    if constexpr (sizeof(H2) == 4 && std::is_same<H2, __nv_bfloat162>::value) {
        a = __bfloat1622float2(mn), b = __bfloat1622float2(mx);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __bfloat1622float2(h[i]);
    } else {
        a = __half22float2(mn), b = __half22float2(mx);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __half22float2(h[i]);
    }
    const float low = a.x + a.y, high = b.x + b.y;   // NaN or infinite once one is not finite (or their sum overflows)
    lo = fminf(lo, fminf(a.x, a.y));
    hi = fmaxf(hi, fmaxf(b.x, b.y));
    return fabsf(low) < INFINITY && fabsf(high) < INFINITY;
}
__device__ __forceinline__ bool load16(const __nv_bfloat16* p, float2 (&v)[8], float& lo, float& hi) {
    return load16_half<__nv_bfloat162>(p, v, lo, hi);
}
__device__ __forceinline__ bool load16(const __half* p, float2 (&v)[8], float& lo, float& hi) {
    return load16_half<__half2>(p, v, lo, hi);
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
    constexpr int L = G / 16;   // lanes per group
    const int64_t row = blockIdx.x;
    const T* src = reinterpret_cast<const T*>(a.W) + row * a.d_in;
    uint8_t* dst = a.q + row * (a.d_in >> 1);
    const int sub = threadIdx.x % L;
    const int np = a.d_in >> 4;        // pieces of 16 columns (d_in is a multiple of 32)
    const int npr = (np + 31) & ~31;   // whole warps walk the row: the shuffles below see every lane
    for (int p = threadIdx.x; p < npr; p += blockDim.x) {
        float2 v[8];
        const bool in = p < np;
        float lo = 0.f, hi = 0.f;
        if (in) {
            if (!load16(src + 16 * p, v, lo, hi)) {   // (or, rarely, two huge values whose sum overflows)
                bool bad = false;
                lo = hi = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (!(fabsf(v[i].x) < INFINITY)) bad = true, v[i].x = 0.f;
                    if (!(fabsf(v[i].y) < INFINITY)) bad = true, v[i].y = 0.f;
                    lo = fminf(lo, fminf(v[i].x, v[i].y));
                    hi = fmaxf(hi, fmaxf(v[i].x, v[i].y));
                }
                if (bad) latch_error(LF_ERR_NUMERIC);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const float s = a.zeros ? bf16_quotient(hi, lo, 15.f) : bf16_quotient(fmaxf(hi, -lo), 0.f, 7.f);
        float z = 8.f;
        uint32_t w[2];
        if (s >= 0x1p-100f) {
            const float inv = rcp_approx(s);
            if (a.zeros) {
                z = rint_quotient(-lo, s, (fmaf(-lo, inv, kRintMagic)) - kRintMagic);
                z = fminf(fmaxf(z, 0.f), 15.f);
            }
            // code = rint(w / s) + z in the low bits of u = 1.5 2^23 + z + w * inv: |w / s| <= 15.1, so
            // w * inv is within 2^-18 of the quotient; what lies that close to a half is settled exactly
            const float2 inv2 = make_float2(inv, inv), ninv2 = make_float2(-inv, -inv);
            const float2 up = make_float2(kRintMagic + z, kRintMagic + z), dn = make_float2(-kRintMagic - z, -kRintMagic - z);
            float2 u[8];
            float far = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                u[i] = ffma2(v[i], inv2, up);
                const float2 d = ffma2(v[i], ninv2, fadd2(u[i], dn));
                far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
            }
            if (far > 0.5f - 0x1p-17f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i].x = rint_quotient(v[i].x, s, u[i].x + dn.x) + up.x;
                    u[i].y = rint_quotient(v[i].y, s, u[i].y + dn.y) + up.y;
                }
            }
            // codes are 0 or more (rint is odd), and 15 or less without zero points
            if (a.zeros) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i].x = fminf(u[i].x, kRintMagic + 15.f);
                    u[i].y = fminf(u[i].y, kRintMagic + 15.f);
                }
            }
            w[0] = w[1] = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t c = __float_as_uint(i & 1 ? u[i >> 1].y : u[i >> 1].x) << (4 * (i & 7));
                w[i >> 3] = (w[i >> 3] & ~(15u << (4 * (i & 7)))) | (c & (15u << (4 * (i & 7))));
            }
        } else {   // 1 / s may overflow, and s may be 0
            if (a.zeros) z = s > 0.f ? (float)fmin(fmax(rint(-(double)lo / (double)s), 0.0), 15.0) : 0.f;
            w[0] = w[1] = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = i & 1 ? v[i >> 1].y : v[i >> 1].x;
                const double q = s > 0.f ? rint((double)x / (double)s) : 0.0;
                w[i >> 3] |= (uint32_t)fmin(fmax(q + (double)z, 0.0), 15.0) << (4 * (i & 7));
            }
        }
        if (in) {
            *reinterpret_cast<uint2*>(dst + 8 * p) = make_uint2(w[0], w[1]);
            if (sub == 0) {
                const int64_t gi = row * a.ng + p / L;
                a.scales[gi] = __float2bfloat16_rn(s);   // exact: s is a bf16 value
                if (a.zeros) a.zeros[gi] = (uint8_t)z;
            }
        }
    }
}

// W = (q - z) * s, one rounding to the output type (none for fp32: 13 significant bits).
// Bound by the write of W.
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

// CTA per kW4DeqRows rows: a thread has that many reads in flight.
constexpr int kW4DeqRows = 4;
template <typename T>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(W4DequantArgs a) {
    const int row0 = (int)blockIdx.x * kW4DeqRows;
    const int n8 = a.d_in >> 3;
    for (int p = threadIdx.x; p < n8; p += blockDim.x) {
        uint32_t w[kW4DeqRows];
        float s[kW4DeqRows], z[kW4DeqRows];
#pragma unroll
        for (int r = 0; r < kW4DeqRows; ++r) {
            const int64_t row = min(row0 + r, a.d_out - 1);
            const int64_t gi = row * a.ng + (p >> (a.log_g - 3));
            w[r] = __ldg(reinterpret_cast<const uint32_t*>(a.q + row * (a.d_in >> 1)) + p);
            s[r] = __bfloat162float(a.scales[gi]);
            z[r] = 8388608.f + (float)(a.zeros ? (a.zeros[gi] & 15) : 8);
        }
#pragma unroll
        for (int r = 0; r < kW4DeqRows; ++r) {
            if (row0 + r >= a.d_out) break;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (__uint_as_float(((w[r] >> (4 * j)) & 15u) | 0x4B000000u) - z[r]) * s[r];
            store8<T>(reinterpret_cast<T*>(a.W) + (int64_t)(row0 + r) * a.d_in + 8 * p, v);
        }
    }
}

// ---- product, few tokens -----------------------------------------------------------------
// CTA (32 rows of one projection, 8 NT tokens): eight warps take the 256-column blocks of d_in
// in turn and add up through shared memory in warp order.  Each warp streams its blocks
// through a private ring of TMA stages (one box of 32 rows x 128 bytes each, 128-byte
// swizzle, no block barriers), unpacks to bf16 and multiplies with mma.sync m16n8k16
// (weights = the 16-row operand, tokens = the 8 columns): one product feeds up to 8 tokens.
// The reads bound it from below (a layer's 122 MB: 19 us); what competes is the instructions,
// about 80 per 512 bytes and warp, and the waits that 16 warps per SM leave open (one token
// through 7 projections: 37 us, issue slots 51 %, DRAM 39 % busy), so the kernel spends none on
// anything it can leave out:
//  - a lane's 32-bit word gives nibbles i and i + 4 as a bf16 pair 128 + q by one mask (the
//    columns of the product are permuted alike for x), and one packed subtraction makes q - z of
//    it, exactly.  (Taking 128 + z out of the group's sum instead saves the subtractions, but
//    leaves the rounding of 128 sum x where codes are near the zero point, and an x above 2^120
//    overflows.)
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

// bf16x2 of (nibble i, nibble i + 4) - z, exact; z2: 128 + z twice
template <int I>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, uint32_t z2) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)), "r"(0x000F000Fu), "r"(0x43004300u));
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&r), *reinterpret_cast<__nv_bfloat162*>(&z2));
    return *reinterpret_cast<const uint32_t*>(&d);
}
template <int NT>
struct W4Smem {
    union {
        unsigned char ring[kW4Warps][kW4Depth][kW4StageBytes];   // 1024-byte aligned stages
        float part[kW4Warps][kW4Rows][8 * NT + 1];
    };
    uint64_t full[kW4Warps][kW4Depth];
};

// Sums of one warp over its columns: two 16-row tiles, NT token tiles; acc over all groups, part
// over the current one.
template <int NT>
struct W4Acc {
    float acc[2][NT][4], part[2][NT][4];
    float sc[2][2];             // scale of rows 16 m + 8 h + (this lane's row)
    uint32_t z2[2][2];          // 128 + z of the same rows, twice (bf16)

    // end of a group: acc += s sum (q - z) x
    __device__ __forceinline__ void flush() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 r = ffma2(make_float2(sc[m][h], sc[m][h]),
                                           make_float2(part[m][n][2 * h], part[m][n][2 * h + 1]),
                                           make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]));
                    acc[m][n][2 * h] = r.x;
                    acc[m][n][2 * h + 1] = r.y;
                }
    }
    // scale and zero point of every row of the tile, one row per lane in sz: the scale's bf16 bits
    // above those of 128 + z
    __device__ __forceinline__ void scales(uint32_t sz, int rg) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t v = __shfl_sync(0xffffffffu, sz, 16 * m + 8 * h + rg);
                sc[m][h] = __uint_as_float(v & 0xffff0000u);
                z2[m][h] = __byte_perm(v, v, 0x1010);
            }
    }
    // one word of each of the lane's four rows against 8 columns of x; a group begins with FIRST
    template <bool FIRST>
    __device__ __forceinline__ void product(const uint32_t (&w)[2][2], const uint4 (&xv)[NT]) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            b[n][0] = __byte_perm(xv[n].x, xv[n].z, 0x5410);   // (x0, x4)
            b[n][1] = __byte_perm(xv[n].x, xv[n].z, 0x7632);   // (x1, x5)
            b[n][2] = __byte_perm(xv[n].y, xv[n].w, 0x5410);   // (x2, x6)
            b[n][3] = __byte_perm(xv[n].y, xv[n].w, 0x7632);   // (x3, x7)
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t lo[4] = {nibble_pair<0>(w[m][0], z2[m][0]), nibble_pair<0>(w[m][1], z2[m][1]),
                                    nibble_pair<1>(w[m][0], z2[m][0]), nibble_pair<1>(w[m][1], z2[m][1])};
            const uint32_t hi[4] = {nibble_pair<2>(w[m][0], z2[m][0]), nibble_pair<2>(w[m][1], z2[m][1]),
                                    nibble_pair<3>(w[m][0], z2[m][0]), nibble_pair<3>(w[m][1], z2[m][1])};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (FIRST) mma_16816_0(part[m][n], lo, b[n][0], b[n][1]);
                else mma_16816(part[m][n], lo, b[n][0], b[n][1]);
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
    auto issue = [&](int st, int slot) {   // lane 0: block warp + 8 st of the rows into a ring slot
        if (st < n_st) {
            uint64_t* bar = &full[slot];
            mbar_arrive_expect_tx(bar, kW4StageBytes);
            tc::tma_load_2d(sm.ring[warp][slot], &maps.q[pi], (warp + kW4Warps * st) * 128, row0, bar);
        }
    };
    if (lane == 0)
        for (int st = 0; st < kW4Depth; ++st) issue(st, st);
    __syncwarp();

    // lane's row of a tile: rows of neighbouring g differ in bit 2, so that the 16-byte loads of
    // 8 lanes (two rows) fall on distinct banks of the swizzled stage
    const int rg = (g >> 1) | ((g & 1) << 2);
    W4Acc<NT> A;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) A.acc[0][n][i] = A.acc[1][n][i] = 0.f;
    // columns of the product past the last token take some token's x; they are not stored
    const __nv_bfloat16* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xr[n] = P.x + (int64_t)min(tok0 + 8 * n + g, a.T - 1) * P.x_ld + (WIDE ? t * 32 : t * 8);
    // A step is what one 16-byte load per row covers: four units (WIDE; a whole group or half of
    // one) or one unit.  Its x, scale and zero point (of row row0 + lane; rows past the last: any)
    // are fetched a step ahead, so that their latency passes while the step before is multiplied
    // (x of two token tiles would not fit the registers: fetched as its step begins).
    constexpr int kUnits = WIDE ? 4 : 1, kSteps = 8 / kUnits;
    const __nv_bfloat16* srow = P.scales + (int64_t)min(row0 + lane, P.d_out - 1) * P.ng;
    const uint8_t* zrow = P.zeros ? P.zeros + (int64_t)min(row0 + lane, P.d_out - 1) * P.ng : nullptr;
    const int log_u = P.log_u;
    uint4 xb[2][kUnits][NT];   // this step's, the next one's
    __nv_bfloat16 sn = __float2bfloat16_rn(0.f);
    uint32_t zn = 8u;
    auto fetch_s = [&](int u) {
        sn = srow[u >> log_u];
        if (zrow) zn = zrow[u >> log_u];
    };
    auto fetch_x = [&](int u, uint4 (&xn)[kUnits][NT]) {
        if (!WIDE || u + 4 <= units) {   // uniform
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kUnits; ++i) xn[i][n] = __ldg(reinterpret_cast<const uint4*>(xr[n] + u * 32 + 8 * i));
        } else {   // the row ends inside the step
            const bool in = u + t < units;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    xn[i][n] = make_uint4(0, 0, 0, 0);
                    if (in) xn[i][n] = __ldg(reinterpret_cast<const uint4*>(xr[n] + u * 32 + 8 * i));
                }
        }
    };
    bool ok = true;
    if (n_st > 0) {
        fetch_s(warp * 8);
        if (NT == 1) fetch_x(warp * 8, xb[0]);
    }
    int slot = 0;
    uint32_t parity = 0;
    for (int st = 0; st < n_st; ++st) {
        const unsigned char* src = sm.ring[warp][slot] + rg * 128;
        const int u0 = (warp + kW4Warps * st) * 8;
#pragma unroll
        for (int sb = 0; sb < kSteps; ++sb) {
            const int u = u0 + kUnits * sb;
            if (u >= units) break;   // uniform
            uint4 (&xc)[kUnits][NT] = xb[NT > 1 ? 0 : sb & 1];
            if (NT > 1) fetch_x(u, xc);
            const uint32_t sz = ((uint32_t)__bfloat16_as_ushort(sn) << 16) | (zn & 15u) | 0x4300u;
            int un = u + kUnits;     // the next step, in this block or the warp's next
            if (sb == kSteps - 1 || un >= units) un = u0 + 8 * kW4Warps;
            if (un < units) {
                fetch_s(un);
                if (NT == 1) fetch_x(un, xb[(sb + 1) & 1]);
            }
            if (sb == 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], parity));
                if (!ok) break;   // uniform; the timeout is latched
            }
            if (WIDE) {
                A.scales(sz, rg);
                uint4 q[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        q[m][h] = *reinterpret_cast<const uint4*>(src + (16 * m + 8 * h) * 128 + (((4 * sb + t) ^ rg) << 4));
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    uint32_t w[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            w[m][h] = i == 0 ? q[m][h].x : i == 1 ? q[m][h].y : i == 2 ? q[m][h].z : q[m][h].w;
                    if (i == 0) A.template product<true>(w, xc[i]);
                    else A.template product<false>(w, xc[i]);
                }
                A.flush();
            } else {
                uint32_t w[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[m][h] = *reinterpret_cast<const uint32_t*>(src + (16 * m + 8 * h) * 128 + ((sb ^ rg) << 4) + 4 * t);
                // groups of one or two units begin at every unit, at every even unit
                if (log_u == 0 || (sb & 1) == 0) {
                    A.scales(sz, rg);
                    A.template product<true>(w, xc[0]);
                } else {
                    A.template product<false>(w, xc[0]);
                }
                if (log_u == 0 || (sb & 1) != 0 || u + 1 >= units) A.flush();
            }
        }
        if (!ok) break;
        __syncwarp();   // the stage has been read
        if (lane == 0) issue(st + kW4Depth, slot);
        if (++slot == kW4Depth) {
            slot = 0;
            parity ^= 1;
        }
    }
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

// ---- product, many tokens ------------------------------------------------------------------
// CTA (128 rows of one projection, N tokens, a share of d_in): D = W x^T on tcgen05 with the
// weights as the 128-row operand A.  A comes from tensor memory: a thread unpacks its row's
// codes (lane = row there) and stores q - z as bf16 pairs, so the unpacked weights never
// touch shared memory, whose bandwidth would bound the product (128 columns of 128 rows:
// 32 KB written and 32 KB read against 512 cycles of products at N = 128).  Blocks of 256
// columns: one code stage, four x boxes, one A buffer.
//   warps 0-7, unpack: two warpgroups take the blocks in turn; codes by TMA (boxes of 128 rows
//     x 128 bytes), exact q - z, tcgen05.st (9 integer instructions per 8 weights, 576 cycles of an
//     SM per block against 712 in which HBM delivers its codes);
//   warps 8-15, sums: each group's product leaves tensor memory and is added to fp32 registers
//     times the row's scale (A stays exact, and a group's scale multiplies once, in fp32);
//     two product buffers, so that the next group runs meanwhile;
//   warps 16, 17: TMA of the codes, of x;  warp 18: issues the products, converged, so that
//     the descriptors stay in uniform registers (issued from a branch of one lane, each
//     product took 100 to 270 cycles of that lane's own instructions).
// CS CTAs of a cluster share d_in when there are few tiles; they add up over distributed
// shared memory in rank order.
constexpr int kW4mThreads = 19 * 32;
constexpr int kW4mRows = 128;
constexpr int kW4mX = 2;      // x stages: N tokens x 256 columns
// code stages (128 rows x 256 columns, 16 KB): with few tokens the reads of the codes bound
// the kernel, and what x leaves of shared memory keeps them in flight
constexpr int w4m_q(int N) { return N == 128 ? 5 : 8; }

struct alignas(64) W4mMaps {
    CUtensorMap q[kW4MaxProj];   // box 128 bytes x 128 rows, 128-byte swizzle
    CUtensorMap x[kW4MaxProj];   // box 64 columns x N rows, 128-byte swizzle
};

template <int N>
struct W4mSmem {
    static constexpr int kW4mQ = w4m_q(N);
    union {
        struct {
            unsigned char q[kW4mQ][kW4mRows * 128];
            unsigned char x[kW4mX][4][N * 128];       // four pieces of 64 columns
        };
        float part[N][kW4mRows];                      // this CTA's sums, for the cluster
    };
    uint64_t qfull[kW4mQ], qempty[kW4mQ], xfull[kW4mX], xempty[kW4mX], afull[2], aempty[2], dfull[2], dempty[2];
    uint32_t tmem;
    int32_t failed;
};

// 8 columns (one word) as four bf16 pairs of q - z in column order
__device__ __forceinline__ void unpack_word(uint32_t w, __nv_bfloat162 z, uint32_t* out) {
    const uint32_t odd = w >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // byte i of both, their low nibbles
        uint32_t p = __byte_perm(w, odd, (uint32_t)(i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12)));
        p = (p & 0x000F000Fu) | 0x43004300u;   // 128 + q
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&p), z);
        out[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

constexpr uint32_t kW4mAcol = 256;   // two product buffers of N <= 128 columns, then two A buffers of 128

// The products of a CTA's nb blocks, 2^LOGD groups in each: one converged warp.
template <int N, int LOGD>
__device__ __forceinline__ bool w4m_products(W4mSmem<N>& s, uint32_t tmem_any, int nb) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    const uint32_t idesc = tc::idesc_bf16(kW4mRows, N, 0, 0);
    const uint64_t xdesc = tc::smem_desc_sw128(s.x[0][0]);
    constexpr int per = 16 >> LOGD;   // K = 16 steps of a group's piece
    int d = 0;
    for (int b = 0; b < nb; ++b) {
        const uint64_t xd = xdesc + (uint64_t)((b % kW4mX) * (4 * N * 128 / 16));
        const uint32_t ad = tmem + kW4mAcol + 128 * (b & 1);
        bool ok = mbar_wait(&s.xfull[b % kW4mX], (uint32_t)(b / kW4mX) & 1) && mbar_wait(&s.afull[b & 1], (uint32_t)(b >> 1) & 1);
#pragma unroll
        for (int g = 0; g < (1 << LOGD); ++g, ++d) {
            if (d >= 2) ok = ok && mbar_wait(&s.dempty[d & 1], (uint32_t)((d >> 1) - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc::fence_after_sync();
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const int k = g * per + i;
                tc::mma_bf16_ta_warp(tmem + (uint32_t)((d & 1) * N), ad + 8 * k,
                                     xd + (uint64_t)((k >> 2) * (N * 128 / 16) + 2 * (k & 3)), idesc, i > 0);
            }
            tc::commit_warp(&s.dfull[d & 1]);
        }
        tc::commit_warp(&s.xempty[b % kW4mX]);
        tc::commit_warp(&s.aempty[b & 1]);
    }
    // every product has completed before the buffers are reused or the CTA leaves
    bool ok = nb == 0 || mbar_wait(&s.aempty[(nb - 1) & 1], (uint32_t)((nb - 1) >> 1) & 1);
    return __all_sync(0xffffffffu, ok);
}

template <int N>
__global__ void __launch_bounds__(kW4mThreads, 1) w4_gemm_kernel(const __grid_constant__ W4Args a,
                                                                 const __grid_constant__ W4mMaps maps, int n_tok_tiles) {
    namespace cg = cooperative_groups;
    constexpr uint32_t kTmemCols = 512;
    constexpr int NH = N / 2;              // tokens per sum thread
    constexpr int kW4mQ = w4m_q(N);
    extern __shared__ __align__(1024) unsigned char w4_raw[];
    auto& s = *reinterpret_cast<W4mSmem<N>*>(w4_raw);
    cg::cluster_group cl = cg::this_cluster();
    const int CS = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tile = (int)blockIdx.x / CS / n_tok_tiles;
    const int tok0 = ((int)blockIdx.x / CS % n_tok_tiles) * N;
    int pi = 0;
#pragma unroll
    for (int i = 1; i < kW4MaxProj; ++i)
        if (i < a.n_proj && tile >= a.p[i].tile0) pi = i;
    const W4Proj& P = a.p[pi];
    const int row0 = (tile - P.tile0) * kW4mRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (P.d_in + 255) >> 8;
    const int b0 = (int)((int64_t)blocks * rank / CS);                        // this CTA's blocks: b0 ..
    const int nb = (int)((int64_t)blocks * (rank + 1) / CS) - b0;
    const int log_u = P.log_u, log_d = 3 - log_u;                             // log2 of groups per block
    if (warp == 0) tc::tmem_alloc(&s.tmem, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kW4mQ; ++i) {
            mbar_init(&s.qfull[i], 1);
            mbar_init(&s.qempty[i], 4);
        }
        for (int i = 0; i < kW4mX; ++i) {
            mbar_init(&s.xfull[i], 1);
            mbar_init(&s.xempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.afull[i], 4);
            mbar_init(&s.aempty[i], 1);
            mbar_init(&s.dfull[i], 1);
            mbar_init(&s.dempty[i], 8);
        }
        s.failed = 0;
        fence_barrier_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s.tmem;
    const int row = row0 + 32 * (warp & 3) + lane;                 // unpack and sum threads
    const int64_t grow = (int64_t)min(row, P.d_out - 1) * P.ng;    // rows past the last: any
    bool ok = true;
    if (warp < 8) {   // ---- unpack: blocks b = warpgroup, warpgroup + 2, ..
        const int r = 32 * (warp & 3) + lane, wg = warp >> 2;
        const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kW4mAcol + 128 * wg;
        const uint8_t* zrow = P.zeros ? P.zeros + grow : nullptr;
        for (int b = wg; b < nb && ok; b += 2) {
            const int qs = b % kW4mQ;
            uint32_t z[8];   // 0x4300 + zero point of each 32-column unit (a group covers 1, 2, 4 or 8)
            if (zrow) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    z[u] = (u & ((1 << log_u) - 1)) == 0 ? zrow[min(((b0 + b) * 8 + u) >> log_u, P.ng - 1)] : z[u > 0 ? u - 1 : 0];
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) z[u] = 8u;
            }
            ok = mbar_wait(&s.qfull[qs], (uint32_t)(b / kW4mQ) & 1);
            if (b >= 2) ok = ok && mbar_wait(&s.aempty[wg], (uint32_t)((b >> 1) - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after_sync();   // the products that read this buffer are complete (aempty)
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // 64 columns: 32 columns of tensor memory
                uint32_t o[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = 2 * q + h;   // 16-byte piece of the row
                    const uint4 w = *reinterpret_cast<const uint4*>(s.q[qs] + r * 128 + ((c ^ (r & 7)) << 4));
                    const uint32_t zz = (0x4300u + (z[c] & 15u)) * 0x10001u;
                    const __nv_bfloat162 zp = *reinterpret_cast<const __nv_bfloat162*>(&zz);
                    unpack_word(w.x, zp, o + 16 * h);
                    unpack_word(w.y, zp, o + 16 * h + 4);
                    unpack_word(w.z, zp, o + 16 * h + 8);
                    unpack_word(w.w, zp, o + 16 * h + 12);
                }
                tc::tmem_st32(at + 32 * q, o);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive1(&s.afull[wg]);
                mbar_arrive1(&s.qempty[qs]);
            }
        }
    } else if (warp < 16) {   // ---- sums: NH of the tokens, every group's product
        const int half = (warp - 8) >> 2;
        const int nd = nb << log_d;
        const __nv_bfloat16* srow = P.scales + grow;
        const int g0 = b0 << log_d;
        const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(half * NH);
        float2 acc[NH / 2];
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) acc[i] = make_float2(0.f, 0.f);
        const int last = P.ng - 1;
        __nv_bfloat16 next = srow[min(g0, last)];   // kept as loaded: a conversion would wait for it
        for (int d = 0; d < nd && ok; ++d) {
            const __nv_bfloat16 cur = next;
            next = srow[min(g0 + d + 1, last)];     // arrives while this one is waited for
            ok = __all_sync(0xffffffffu, mbar_wait(&s.dfull[d & 1], (uint32_t)(d >> 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
            const float2 sc = make_float2(__bfloat162float(cur), __bfloat162float(cur));
#pragma unroll
            for (int c = 0; c < NH / 16; ++c) {
                float v[16];
                tc::tmem_ld16(at + (uint32_t)((d & 1) * N + 16 * c), v);
                if (c == NH / 16 - 1) {   // all read: the buffer is free for the group after next
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive1(&s.dempty[d & 1]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[8 * c + i] = ffma2(sc, make_float2(v[2 * i], v[2 * i + 1]), acc[8 * c + i]);
            }
        }
        if (ok && CS == 1) {
            const int t0 = tok0 + half * NH;
            const float bias = P.bias ? __bfloat162float(P.bias[min(row, P.d_out - 1)]) : 0.f;
#pragma unroll
            for (int i = 0; i < NH; ++i)
                if (row < P.d_out && t0 + i < a.T)
                    P.y[(int64_t)(t0 + i) * P.y_ld + row] = __float2bfloat16_rn((i & 1 ? acc[i / 2].y : acc[i / 2].x) + bias);
        } else if (ok) {   // the last product has read the last stage: the stages become this CTA's sums
#pragma unroll
            for (int i = 0; i < NH; ++i)
                s.part[half * NH + i][32 * (warp & 3) + lane] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
        }
    } else if (warp == 16) {   // ---- TMA of the codes
        if (lane == 0) {
            int i = 0;   // stages issued
            for (; i < nb; ++i) {
                const int st = i % kW4mQ;
                if (i >= kW4mQ) ok = mbar_wait(&s.qempty[st], (uint32_t)(i / kW4mQ - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.qfull[st], kW4mRows * 128);
                tc::tma_load_2d(s.q[st], &maps.q[pi], (b0 + i) * 128, row0, &s.qfull[st]);
            }
            // nothing is in flight when the buffers are reused or the CTA leaves
            for (int j = max(0, i - kW4mQ); j < i; ++j) ok = mbar_wait(&s.qfull[j % kW4mQ], (uint32_t)(j / kW4mQ) & 1) && ok;
        }
    } else if (warp == 17) {   // ---- TMA of x
        if (lane == 0) {
            int i = 0;
            for (; i < nb; ++i) {
                const int st = i % kW4mX;
                if (i >= kW4mX) ok = mbar_wait(&s.xempty[st], (uint32_t)(i / kW4mX - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.xfull[st], 4 * N * 128);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    tc::tma_load_2d(s.x[st][q], &maps.x[pi], (b0 + i) * 256 + 64 * q, tok0, &s.xfull[st]);
            }
            for (int j = max(0, i - kW4mX); j < i; ++j) ok = mbar_wait(&s.xfull[j % kW4mX], (uint32_t)(j / kW4mX) & 1) && ok;
        }
    } else {   // ---- products
        ok = log_d == 0   ? w4m_products<N, 0>(s, tmem, nb)
             : log_d == 1 ? w4m_products<N, 1>(s, tmem, nb)
             : log_d == 2 ? w4m_products<N, 2>(s, tmem, nb)
                          : w4m_products<N, 3>(s, tmem, nb);
    }
    if (!ok) s.failed = 1;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
    if (CS == 1) return;
    cl.sync();
    bool all_ok = true;
    for (int c = 0; c < CS; ++c) all_ok = all_ok && *cl.map_shared_rank(&s.failed, c) == 0;
    // this CTA's share of the tokens, summed over the cluster in rank order
    const int nt = min(N, a.T - tok0);
    const int n0 = nt * rank / CS, n1 = all_ok ? nt * (rank + 1) / CS : n0;   // a timeout is latched
    for (int o = tid; o < (n1 - n0) * kW4mRows; o += kW4mThreads) {
        const int n = n0 + o / kW4mRows, r = o % kW4mRows;
        if (row0 + r >= P.d_out) continue;
        float v = 0.f;
        for (int c = 0; c < CS; ++c) v += cl.map_shared_rank(&s.part[n][r], c)[0];
        if (P.bias) v += __bfloat162float(P.bias[row0 + r]);
        P.y[(int64_t)(tok0 + n) * P.y_ld + row0 + r] = __float2bfloat16_rn(v);
    }
    cl.sync();   // the parts are read by the whole cluster
}

}  // namespace lf
