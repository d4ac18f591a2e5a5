// Base weights in 4 bits with group scales: quantisation, its inverse, and the product
//   y = bf16( bias + sum_g s_g sum_{i in g} (q_i - z_g) x_i )
// of a token batch with them: the W0 x of "Compress then Serve" (academ.us/article/
// 2407.00066), section 3, that the LoRA side path adds to, at a quarter of the bytes.
//
// Format: q holds d_out rows of d_in / 2 bytes, column 2 c in the low nibble of byte c;
// scales (bf16) and zero points (one byte each, 0 .. 15; absent = 8) are d_out x ng,
// ng = ceil(d_in / group) (the last group may be short).  A weight is (q - z) * s.
#pragma once
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

// rint(w / s) for s > 0 and |w / s| < 2^20: an estimate off by at most one, corrected by
// the exact sign of w - (q +- 1/2) s (one fma: the product is exact inside it).
__device__ __forceinline__ float rint_quotient(float w, float s, float inv) {
    if (s < 0x1p-100f) return (float)rint((double)w / (double)s);   // 1 / s may overflow
    const float q = rintf(w * inv);
    const float up = fmaf(-(q + 0.5f), s, w), dn = fmaf(-(q - 0.5f), s, w);
    const bool odd = ((int)q & 1) != 0;
    if (up > 0.f || (up == 0.f && odd)) return q + 1.f;
    if (dn < 0.f || (dn == 0.f && odd)) return q - 1.f;
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

template <typename T, int G>
__global__ void __launch_bounds__(256) w4_quantize_kernel(W4QuantArgs a) {
    constexpr int L = G / 8;   // lanes per group
    const int64_t gid = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;   // (row, group)
    const int sub = threadIdx.x % L;
    const bool live = gid < (int64_t)a.d_out * a.ng;
    const int64_t row = live ? gid / a.ng : 0;
    const int g = live ? (int)(gid - row * a.ng) : 0;
    const int c0 = g * G + sub * 8;
    float v[8];
    const bool in = live && c0 < a.d_in;   // d_in is a multiple of 32
    if (in) {
        load8<T>(reinterpret_cast<const T*>(a.W) + row * a.d_in + c0, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    float lo = 0.f, hi = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!(fabsf(v[i]) < INFINITY)) {
            bad = true;
            v[i] = 0.f;
        }
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    if (bad) latch_error(LF_ERR_NUMERIC);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    float s, z;
    if (a.zeros) s = bf16_quotient(hi, lo, 15.f);
    else s = bf16_quotient(fmaxf(hi, -lo), 0.f, 7.f);
    const float inv = s > 0.f ? 1.f / s : 0.f;
    if (a.zeros) z = s > 0.f ? fminf(fmaxf(rint_quotient(-lo, s, inv), 0.f), 15.f) : 0.f;
    else z = 8.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = s > 0.f ? rint_quotient(v[i], s, inv) : 0.f;
        w |= (uint32_t)fminf(fmaxf(q + z, 0.f), 15.f) << (4 * i);
    }
    if (in) *reinterpret_cast<uint32_t*>(a.q + row * (a.d_in >> 1) + (c0 >> 1)) = w;
    if (live && sub == 0) {
        a.scales[gid] = __float2bfloat16_rn(s);   // exact: s is a bf16 value
        if (a.zeros) a.zeros[gid] = (uint8_t)z;
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
    const int per = a.d_in >> 3;   // 8-weight pieces per row
    const int64_t n = (int64_t)a.d_out * per;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t row = i / per;
    const int c0 = (int)(i - row * per) * 8;
    const int64_t gi = row * a.ng + (c0 >> a.log_g);
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(a.q + row * (a.d_in >> 1) + (c0 >> 1)));
    const float s = __bfloat162float(a.scales[gi]);
    const int z = a.zeros ? (a.zeros[gi] & 15) : 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((int)((w >> (4 * j)) & 15u) - z) * s;
    store8<T>(reinterpret_cast<T*>(a.W) + row * a.d_in + c0, v);
}

// ---- product, few tokens -----------------------------------------------------------------
// CTA (16 MT rows of one projection, 8 NT tokens): eight warps split d_in evenly in units of
// 32 weights (16 bytes of a row) and add up through shared memory in warp order.  Each warp
// streams its part of the rows through a private ring of cp.async stages (no block
// barriers), unpacks to bf16 and multiplies with mma.sync m16n8k16 (weights = the 16-row
// operand, tokens = the 8 columns): one product feeds up to 8 tokens, and the arithmetic
// stays far below the reads it hides behind.
//
// Exactness: q - z is a small integer, exact in bf16 (128 + q by bits, minus 128 + z), so a
// group's sum is the fp32 accumulation of exact products; s_g multiplies it in fp32.
//
// Inside a unit, lane t of a row's four lanes takes the 32-bit word t, whose nibbles i and
// i + 4 come out of one mask as a pair: the columns of the product are permuted alike for
// x (pairs (x_i, x_{i+4}) of the lane's 8 values), which costs four byte permutes per unit.
// Any group of 32 or more weights covers whole units, so one layout serves every group size.
constexpr int kW4Warps = 8;
constexpr int kW4Units = 4;                        // units per stage: 64 bytes of each row
constexpr int kW4RowBytes = kW4Units * 16 + 16;    // padded: 8 rows x 4 words hit 32 distinct banks
constexpr int kW4MaxProj = 8;

struct W4Proj {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const uint8_t* q;
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

// bf16x2 of (128 + nibble i, 128 + nibble i + 4)
template <int I>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)), "r"(0x000F000Fu), "r"(0x43004300u));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int MT, int NT, int DEPTH>
struct W4Smem {
    union {
        unsigned char ring[kW4Warps][DEPTH][16 * MT * kW4RowBytes];
        float part[kW4Warps][16 * MT][8 * NT + 1];
    };
};

template <int MT, int NT, int DEPTH>
__global__ void __launch_bounds__(32 * kW4Warps) w4_gemv_kernel(const __grid_constant__ W4Args a) {
    extern __shared__ __align__(16) unsigned char w4_raw[];
    auto& sm = *reinterpret_cast<W4Smem<MT, NT, DEPTH>*>(w4_raw);
    int pi = 0;
    for (int i = 1; i < a.n_proj; ++i)
        if ((int)blockIdx.x >= a.p[i].tile0) pi = i;
    const W4Proj& P = a.p[pi];
    const int row0 = ((int)blockIdx.x - P.tile0) * 16 * MT;
    const int tok0 = blockIdx.y * 8 * NT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int units = P.d_in >> 5;
    const int u0 = (int)((int64_t)units * warp / kW4Warps), u1 = (int)((int64_t)units * (warp + 1) / kW4Warps);
    const int n_st = (u1 - u0 + kW4Units - 1) / kW4Units;
    const int64_t row_bytes = P.d_in >> 1;

    // stage st of this warp: 16 MT rows x kW4Units units
    auto issue = [&](int st) {
        if (st < n_st) {
            unsigned char* dst = sm.ring[warp][st % DEPTH];
            const int u = u0 + st * kW4Units;
#pragma unroll
            for (int c = lane; c < 16 * MT * kW4Units; c += 32) {
                const int r = c / kW4Units, k = c % kW4Units;
                const bool ok = row0 + r < P.d_out && u + k < u1;
                cp_async16_zfill(dst + r * kW4RowBytes + k * 16,
                                 ok ? P.q + (int64_t)(row0 + r) * row_bytes + (int64_t)(u + k) * 16 : P.q, ok);
            }
        }
        tc::cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < DEPTH - 1; ++st) issue(st);

    float acc[MT][NT][4], part[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = part[m][n][i] = 0.f;
    uint32_t zp[MT][2];      // bf16x2 of 128 + z for rows g and g + 8
    float sc[MT][2];
    int grp = -1;
    auto flush = [&]() {     // acc += s_g * part
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[m][n][i] = fmaf(sc[m][i >> 1], part[m][n][i], acc[m][n][i]);
                    part[m][n][i] = 0.f;
                }
    };
    for (int st = 0; st < n_st; ++st) {
        tc::cp_async_wait<DEPTH - 2>();
        __syncwarp();
        issue(st + DEPTH - 1);
        const unsigned char* src = sm.ring[warp][st % DEPTH];
        const int nu = min(kW4Units, u1 - u0 - st * kW4Units);
#pragma unroll
        for (int k = 0; k < kW4Units; ++k) {
            if (k >= nu) break;
            const int u = u0 + st * kW4Units + k;
            if ((u >> P.log_u) != grp) {
                if (grp >= 0) flush();
                grp = u >> P.log_u;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = min(row0 + 16 * m + 8 * h + g, P.d_out - 1);
                        sc[m][h] = __bfloat162float(P.scales[(int64_t)r * P.ng + grp]);
                        const uint32_t z = P.zeros ? (P.zeros[(int64_t)r * P.ng + grp] & 15u) : 8u;
                        zp[m][h] = (0x4300u + z) * 0x10001u;
                    }
            }
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int tok = tok0 + 8 * n + g;
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (tok < a.T) xv = __ldg(reinterpret_cast<const uint4*>(P.x + (int64_t)tok * P.x_ld + u * 32 + t * 8));
                b[n][0] = __byte_perm(xv.x, xv.z, 0x5410);   // (x0, x4)
                b[n][1] = __byte_perm(xv.x, xv.z, 0x7632);   // (x1, x5)
                b[n][2] = __byte_perm(xv.y, xv.w, 0x5410);   // (x2, x6)
                b[n][3] = __byte_perm(xv.y, xv.w, 0x7632);   // (x3, x7)
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t w0 = *reinterpret_cast<const uint32_t*>(src + (16 * m + g) * kW4RowBytes + k * 16 + t * 4);
                const uint32_t w1 = *reinterpret_cast<const uint32_t*>(src + (16 * m + 8 + g) * kW4RowBytes + k * 16 + t * 4);
                const uint32_t z0 = zp[m][0], z1 = zp[m][1];
                const uint32_t lo[4] = {bf16x2_sub(nibble_pair<0>(w0), z0), bf16x2_sub(nibble_pair<0>(w1), z1),
                                        bf16x2_sub(nibble_pair<1>(w0), z0), bf16x2_sub(nibble_pair<1>(w1), z1)};
                const uint32_t hi[4] = {bf16x2_sub(nibble_pair<2>(w0), z0), bf16x2_sub(nibble_pair<2>(w1), z1),
                                        bf16x2_sub(nibble_pair<3>(w0), z0), bf16x2_sub(nibble_pair<3>(w1), z1)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_16816(part[m][n], lo, b[n][0], b[n][1]);
                    mma_16816(part[m][n], hi, b[n][2], b[n][3]);
                }
            }
        }
        __syncwarp();   // the stage's reads are done before it is refilled
    }
    if (grp >= 0) flush();
    tc::cp_async_wait<0>();
    __syncthreads();    // the ring becomes the partial sums
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sm.part[warp][16 * m + g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = acc[m][n][i];
    __syncthreads();
    for (int o = tid; o < 16 * MT * 8 * NT; o += 32 * kW4Warps) {
        const int r = o % (16 * MT), n = o / (16 * MT);
        if (row0 + r >= P.d_out || tok0 + n >= a.T) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kW4Warps; ++w) v += sm.part[w][r][n];
        if (P.bias) v += __bfloat162float(P.bias[row0 + r]);
        P.y[(int64_t)(tok0 + n) * P.y_ld + row0 + r] = __float2bfloat16_rn(v);
    }
}

}  // namespace lf
