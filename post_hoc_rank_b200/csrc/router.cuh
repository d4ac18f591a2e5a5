// Routing of tokens to experts (adapters): scores from a gate's logits, an optional bias
// that only steers the choice, groups of experts, top-k, renormalised weights; and the
// gradient of the weights for the logits.
//
// Choosing adapters per token is the dynamic side of a pool of LoRAs (LoRASpace, the arXiv
// listing's abstract: "static and dynamic multi-LoRA composition"); the weights feed the
// routed side path (mixture.cuh).
//
// One warp per token, expert e = 32 i + lane in register i of its lane, so a row is read
// once with whole-line loads and stays in registers; top-k is k rounds of a warp-wide
// maximum (redux.sync on an order-preserving integer image of the key), which ends on the
// lowest index among equals.  The floor is the row's read (a T = 16384, E = 256 fp32 batch:
// 16.8 MB, 2.6 us); the instructions of the scores
// and the rounds bound it.
//
// The chosen indices are those of fp64 scores: without a bias the key is the logit itself (both
// scores are increasing), and a sum with a bias, formed in fp32, is trusted only where neighbours
// in the order are further apart than a bound of its rounding that holds for every expert of the
// row (so that none that was not drawn can belong above); a row with a closer pair is decided
// again from fp64 scores.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace lf {

constexpr int kRouterWarps = 8;   // tokens per CTA

struct RouterArgs {
    const void* logits;     // T rows of ld
    int64_t ld;
    const float* bias;      // nullable, E
    int32_t T, E, K, G, top_groups, group_top;
    int32_t group_mul;      // e / (E / G) = e * group_mul >> 20 for e < 1024
    int32_t sigmoid, renorm;
    float weight_scale;
    int32_t* ids;           // T x K
    float* weights;         // T x K
    int32_t* counts;        // nullable, E (zeroed before the launch)
};

struct RouterGradArgs {
    const void* logits;
    int64_t ld;
    int32_t T, E, K, sigmoid, renorm;
    float weight_scale;
    const int32_t* ids;     // T x K
    const float* gw;        // T x K
    void* dlogits;          // T rows of ld_out, the logits' type
    int64_t ld_out;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename TL> __device__ __forceinline__ TL from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Order-preserving image of a float (no NaN; -0 taken as +0); 0 is below every float and
// marks an expert that cannot be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// For the choice alone (its rounding is allowed for): hardware exponential and reciprocal.
__device__ __forceinline__ float fast_sigmoid(float l) {
    const float e = __expf(-fabsf(l));
    return __fdividef(l >= 0.f ? 1.f : e, 1.f + e);
}

__device__ __forceinline__ float sigmoid_f32(float l) {   // no overflow on either side
    const float e = expf(-fabsf(l));
    return (l >= 0.f ? 1.f : e) / (1.f + e);
}

constexpr float kNoScore = -INFINITY;

// The row's choice from fp64 scores (see the file comment); `c` holds E doubles of this
// warp's shared memory.  Lane j < K returns the j-th chosen expert, -1 where none is left.
template <typename TL>
__device__ __noinline__ int route_row_f64(const RouterArgs& a, const TL* row, double* c) {
    const int lane = threadIdx.x & 31;
    double m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmax(m, (double)to_f32(row[e]));
    m = warp_max(m);   // a bias shuts an expert out of the choice, not of the scores
    double inv = 1.0;
    if (!a.sigmoid) {
        double s = 0.0;
        for (int e = lane; e < a.E; e += 32) {
            const double p = m == -INFINITY ? 0.0 : exp((double)to_f32(row[e]) - m);
            c[e] = p;
            s += p;
        }
        inv = warp_sum(s);
    }
    for (int e = lane; e < a.E; e += 32) {
        const float l = to_f32(row[e]);
        const float b = a.bias ? a.bias[e] : 0.f;
        const double ex = exp(-fabs((double)l));   // no overflow on either side
        const double s = a.sigmoid ? (l >= 0.f ? 1.0 : ex) / (1.0 + ex) : c[e] / inv;
        c[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : s + (double)b;
    }
    __syncwarp();
    if (a.G > 1) {
        const int n = a.E / a.G;
        double mine = -INFINITY;   // group `lane`
        for (int g = 0; g < a.G; ++g) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int e = g * n + lane; e < (g + 1) * n; e += 32) {
                b2 = fmax(b2, fmin(b1, c[e]));
                b1 = fmax(b1, c[e]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double p1 = __shfl_xor_sync(0xffffffffu, b1, o), p2 = __shfl_xor_sync(0xffffffffu, b2, o);
                b2 = fmax(fmin(b1, p1), fmax(b2, p2));
                b1 = fmax(b1, p1);
            }
            if (lane == g) mine = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        }
        int rank = 0;
        for (int g = 0; g < a.G; ++g) {
            const double o = __shfl_sync(0xffffffffu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.G && mine > -INFINITY && rank < a.top_groups);
        for (int g = 0; g < a.G; ++g)
            if (!((kept >> g) & 1u))
                for (int e = g * n + lane; e < (g + 1) * n; e += 32) c[e] = -INFINITY;
        __syncwarp();
    }
    if (!a.bias) {   // the logit decides among those that are left
        for (int e = lane; e < a.E; e += 32)
            if (c[e] > -INFINITY) c[e] = to_f32(row[e]);
        __syncwarp();
    }
    int chosen = -1, last = -1;
    double best = -INFINITY;
    int at = INT_MAX;
    for (int j = 0; j < a.K; ++j) {
        if (last < 0 || (last & 31) == lane) {   // this lane's best has changed
            best = -INFINITY;
            at = INT_MAX;
            for (int e = lane; e < a.E; e += 32)
                if (c[e] > best) {
                    best = c[e];
                    at = e;
                }
        }
        double tv = best;
        int te = at;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, tv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, te, o);
            if (ov > tv || (ov == tv && oe < te)) {
                tv = ov;
                te = oe;
            }
        }
        if (te == INT_MAX) break;   // uniform
        last = te;
        if ((te & 31) == lane) c[te] = -INFINITY;
        if (lane == j) chosen = te;
    }
    return chosen;
}

// Sum of the warp's best (and second best, with group_top 2) keys from every lane's two best;
// no score where nothing can be chosen.
__device__ __forceinline__ float group_score(uint32_t b1, uint32_t b2, int group_top, int lane) {
    const uint32_t w1 = __reduce_max_sync(0xffffffffu, b1);
    float g = w1 ? key_value(w1) : kNoScore;
    if (group_top == 2) {
        const uint32_t has = __ballot_sync(0xffffffffu, b1 == w1);
        const bool first = lane == __ffs(has) - 1;   // this lane's best is the one counted
        const uint32_t w2 = __reduce_max_sync(0xffffffffu, first ? b2 : b1);
        if (w1 && w2) g += key_value(w2);
    }
    return g;
}

// EPL: registers per lane (E <= 32 EPL).  Dynamic shared memory: kRouterWarps * E doubles
// when rows may need fp64 (a bias, or group scores of two), else none.
template <typename TL, int EPL>
__global__ void __launch_bounds__(32 * kRouterWarps) route_experts_kernel(RouterArgs a) {
    extern __shared__ double router_c64[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouterWarps + warp;
    if (t >= a.T) return;   // whole warps; no block barriers below
    const TL* row = reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.ld;
    const int E = a.E, n = E / a.G;
    float l[EPL];
    bool bad = false;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = 32 * i + lane;
        l[i] = e < E ? to_f32(row[e]) : -INFINITY;
        bad = bad || !(l[i] < INFINITY);
        m = fmaxf(m, l[i]);
    }
    float bmax = 0.f;
    uint32_t key[EPL];   // order image of what chooses; 0 = not to be chosen
    const bool scores = a.bias != nullptr || (a.G > 1 && a.group_top == 2);
    m = warp_max(m);
    float c[EPL];        // selection score (only with `scores`)
    float rden = 1.f;    // 1 / softmax denominator, for the choice
    if (scores && !a.sigmoid) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = l[i] == -INFINITY ? 0.f : __expf(l[i] - m);
            s += c[i];
        }
        s = warp_sum(s);
        rden = s > 0.f ? __fdividef(1.f, s) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = 32 * i + lane;
        float b = 0.f;
        if (scores) {
            if (a.bias && e < E) {
                b = a.bias[e];
                bad = bad || !(b < INFINITY);
                if (b != -INFINITY) bmax = fmaxf(bmax, fabsf(b));
            }
            c[i] = (a.sigmoid ? fast_sigmoid(l[i]) : c[i] * rden) + b;
        } else {
            c[i] = 0.f;
        }
        const bool open = l[i] != -INFINITY && b != -INFINITY;
        key[i] = open && !bad ? order_key(a.bias ? c[i] : l[i]) : 0u;
    }
    if (__any_sync(0xffffffffu, bad)) {   // NaN or +inf: the row is left without experts
        if (lane == 0) latch_error(LF_ERR_NUMERIC);
        if (lane < a.K) {
            a.ids[(int64_t)t * a.K + lane] = -1;
            a.weights[(int64_t)t * a.K + lane] = 0.f;
        }
        return;
    }
    if (a.bias) bmax = warp_max(bmax);
    // Error of a score, u = 2^-23, smax the row's largest score.  CUDA's bound for the hardware
    // exponential is 2 + 1.173 |x| ulp, d = |x| (rounded before, for softmax: d / 2 ulp more), for
    // __fdividef 2 ulp.
    //   sigmoid: where l < 0, s (2 + 1.173 d + 1/2 + 2) u, and s d <= smax max(-m, 1), m the largest
    //     logit; where l >= 0 (smax >= 1/2) only e / (1 + e) of the exponential's error: less.
    //   softmax: s d <= 0.37 smax, so the numerator's is 2.62 u smax; the denominator's, weighted by
    //     the scores, (2 + 1.673 ln E) u and (EPL + 5) / 2 u for its sum; its reciprocal and the
    //     product 2.5 u.
    // A sum s + b adds u / 2 of itself, the rounds below leave out EPL - 1 ulp of it.  So every
    // expert's key is within err + rel |key| of its score and bias, the further down the lower
    // still: two neighbours in the order that are further apart than both bounds order all that
    // is above them and all that is below.  2^-120: scores that fp32 flushes or holds in few bits.
    const float smax = a.sigmoid ? fast_sigmoid(m) : rden;
    const float err = smax * (a.sigmoid ? 6.f + 1.25f * fminf(fmaxf(-m, 0.f), 104.f) : 22.f + 0.5f * (float)EPL) * 0x1p-23f +
                      0x1p-120f;
    const float rel = (float)(EPL + 1) * 0x1p-23f;
    bool close = false;
    if (a.G > 1) {
        float mine = kNoScore;   // score of group `lane`
        if ((n & 31) == 0) {     // a group is whole registers: n / 32 of them
            const int per = n >> 5;
            uint32_t b1 = 0, b2 = 0;
            int left = per, g = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (32 * i < E) {
                    const uint32_t kq = a.bias || a.group_top == 1 ? key[i] : (key[i] ? order_key(c[i]) : 0u);
                    b2 = max(b2, min(b1, kq));
                    b1 = max(b1, kq);
                    if (--left == 0) {
                        const float gs = group_score(b1, b2, a.group_top, lane);
                        if (lane == g) mine = gs;
                        b1 = b2 = 0;
                        left = per;
                        ++g;
                    }
                }
            }
        } else {
            for (int g = 0; g < a.G; ++g) {
                uint32_t b1 = 0, b2 = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = 32 * i + lane;
                    if (e >= g * n && e < (g + 1) * n) {
                        const uint32_t kq = a.bias || a.group_top == 1 ? key[i] : (key[i] ? order_key(c[i]) : 0u);
                        b2 = max(b2, min(b1, kq));
                        b1 = max(b1, kq);
                    }
                }
                const float gs = group_score(b1, b2, a.group_top, lane);
                if (lane == g) mine = gs;
            }
        }
        int rank = 0;
        for (int g = 0; g < a.G; ++g) {
            const float o = __shfl_sync(0xffffffffu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const bool live = lane < a.G && mine > kNoScore;
        const uint32_t kept = __ballot_sync(0xffffffffu, live && rank < a.top_groups);
        if (scores) {   // the last group kept and the first left out
            const float lo = -warp_max(live && rank < a.top_groups ? -mine : -INFINITY);
            const float hi = warp_max(live && rank >= a.top_groups ? mine : -INFINITY);
            // one or two sums each, of at most smax + bmax, and their sum
            close = hi > -INFINITY && lo - hi <= 4.f * err + 0x1p-22f * (smax + bmax) + 0x1p-23f * (fabsf(lo) + fabsf(hi));
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = 32 * i + lane;
            if (!((kept >> (((e * a.group_mul) >> 20) & 31)) & 1u)) key[i] = 0u;   // past E: 0 already
        }
    }
    int chosen = -1;     // lane j: the j-th
    uint32_t ckey = 0;   // lane j: its key
    if (a.bias) {
        // K + 1 rounds (one more, to see how close the first one left out is) over keys that carry
        // the register's index in their last bits, sorted within each lane: a round is one
        // warp-wide maximum, and its winner moves up by one.  What the cut bits decide is close
        // anyway, and so are equal keys of two lanes.
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i]) key[i] = (key[i] & ~(uint32_t)(EPL - 1)) | (uint32_t)(EPL - 1 - i);
#pragma unroll
        for (int k = 2; k <= EPL; k *= 2)   // bitonic, descending
#pragma unroll
            for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if ((i ^ j) > i) {
                        const uint32_t hi = max(key[i], key[i ^ j]), lo = min(key[i], key[i ^ j]);
                        key[i] = (i & k) == 0 ? hi : lo;
                        key[i ^ j] = (i & k) == 0 ? lo : hi;
                    }
        for (int j = 0; j <= a.K; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
            if (top == 0) break;   // uniform: nothing left
            const uint32_t has = __ballot_sync(0xffffffffu, key[0] == top);
            close = close || (has & (has - 1)) != 0;
            const int from = __ffs(has) - 1;
            if (lane == j) {
                chosen = 32 * (EPL - 1 - (int)(top & (EPL - 1))) + from;
                ckey = top & ~(uint32_t)(EPL - 1);
            }
            const bool me = lane == from;
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) key[i] = me ? key[i + 1] : key[i];
            key[EPL - 1] = me ? 0u : key[EPL - 1];
        }
    } else {   // exact keys: K rounds that end on the lowest index among equals
        uint32_t best = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        for (int j = 0; j < a.K; ++j) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            if (top == 0) break;   // uniform: nothing left
            const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(32 * bi + lane) : 0xffffffffu);
            if (lane == j) chosen = e;
            if ((e & 31) == lane) {   // the winner's lane takes its next best
                best = 0;
                const int wi = e >> 5;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    if (i == wi) key[i] = 0u;
                    if (key[i] > best) {
                        best = key[i];
                        bi = i;
                    }
                }
            }
        }
    }
    if (a.bias) {   // neighbours in the order, lane j against lane j + 1
        const float el = chosen >= 0 ? to_f32(row[chosen]) : 0.f, eb = chosen >= 0 ? a.bias[chosen] : 0.f;
        const float v = key_value(ckey), vn = __shfl_down_sync(0xffffffffu, v, 1);
        const float ln = __shfl_down_sync(0xffffffffu, el, 1), bn = __shfl_down_sync(0xffffffffu, eb, 1);
        const int cn = __shfl_down_sync(0xffffffffu, chosen, 1);
        bool tie = false;   // equal inputs: a sure tie
        if (lane < a.K && chosen >= 0 && cn >= 0) {
            tie = el == ln && eb == bn;
            close = close || (!tie && v - vn <= 2.f * err + rel * (fabsf(v) + fabsf(vn)));
        }
        if (__shfl_sync(0xffffffffu, (int)tie, a.K - 1)) {   // at the cut: what comes below the equal ones?
            const float vk = __shfl_sync(0xffffffffu, v, a.K - 1), lk = __shfl_sync(0xffffffffu, el, a.K - 1);
            const float bk = __shfl_sync(0xffffffffu, eb, a.K - 1);
            for (int e = lane; e < E; e += 32) {
                const float le = to_f32(row[e]), be = a.bias[e];
                if (le == -INFINITY || be == -INFINITY || (le == lk && be == bk)) continue;
                const float ce = (a.sigmoid ? fast_sigmoid(le) : __expf(le - m) * rden) + be;
                close = close || fabsf(vk - ce) <= 2.f * err + rel * (fabsf(vk) + fabsf(ce));
            }
        }
        close = __any_sync(0xffffffffu, close);
        if (lane == a.K) chosen = -1;   // the one left out
    }
    if (close) chosen = route_row_f64<TL>(a, row, router_c64 + (size_t)warp * E);   // `close` is uniform
    // weights: lane j holds slot j
    const bool on = chosen >= 0;
    const float lj = on ? to_f32(row[chosen]) : -INFINITY;
    float w;
    if (a.renorm) {
        // ratios to the largest chosen score, so that scores that underflow keep theirs:
        // softmax e^(l - m); sigmoid e^(l - m) / (1 + e^l) when every chosen l < 0
        const float ms = warp_max(lj);
        if (a.sigmoid) w = !on ? 0.f : (ms < 0.f ? expf(lj - ms) / (1.f + expf(lj)) : sigmoid_f32(lj));
        else w = on ? expf(lj - ms) : 0.f;
        const float tot = warp_sum(w);
        w = tot > 0.f ? w / tot : 0.f;
    } else {
        float denom = 1.f;
        if (!a.sigmoid) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) s += l[i] == -INFINITY ? 0.f : expf(l[i] - m);
            denom = warp_sum(s);
        }
        w = !on ? 0.f : (a.sigmoid ? sigmoid_f32(lj) : expf(lj - m) / denom);
    }
    if (lane < a.K) {
        a.ids[(int64_t)t * a.K + lane] = chosen;
        a.weights[(int64_t)t * a.K + lane] = w * a.weight_scale;
        if (a.counts && on) atomicAdd(&a.counts[chosen], 1);
    }
}

// d(loss)/d(logits) from d(loss)/d(weights) at the ids the forward chose (the choice itself
// has no gradient, nor has the bias).  With p_j the weight over weight_scale, G = sum_i g_i p_i:
//   softmax, renormalised : p_j (g_j - G) at the chosen, 0 elsewhere
//   sigmoid, renormalised : p_j (1 - s_j) (g_j - G) at the chosen, 0 elsewhere
//   sigmoid               : g_j s_j (1 - s_j) at the chosen, 0 elsewhere
//   softmax               : s_e ([e chosen] g_e - G) everywhere
// One warp per token; only the last form reads the whole row, the others write zeros and
// the chosen entries.  Bound by the T x E write.
template <typename TL, int EPL>
__global__ void __launch_bounds__(32 * kRouterWarps) route_experts_grad_kernel(RouterGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kRouterWarps + warp;
    if (t >= a.T) return;
    const TL* row = reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.ld;
    TL* out = reinterpret_cast<TL*>(a.dlogits) + (int64_t)t * a.ld_out;
    const int E = a.E;
    int id = -1;
    float g = 0.f;
    if (lane < a.K) {
        id = a.ids[(int64_t)t * a.K + lane];
        if (id < -1 || id >= E) {
            latch_error(LF_ERR_BAD_INDEX);
            id = -1;
        }
        if (id >= 0) g = a.gw[(int64_t)t * a.K + lane] * a.weight_scale;
    }
    const bool on = id >= 0;
    const float lj = on ? to_f32(row[id]) : -INFINITY;
    // a row without slots (a NaN in its logits among the reasons) gets zeros
    const bool dense = !a.sigmoid && !a.renorm && __any_sync(0xffffffffu, on);
    float v;              // the slot's contribution to its entry
    float m = 0.f, inv = 0.f, G = 0.f;
    float l[EPL];
    if (dense) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = 32 * i + lane;
            l[i] = e < E ? to_f32(row[e]) : -INFINITY;
            m = fmaxf(m, l[i]);
        }
        m = warp_max(m);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - m);
            s += l[i];
        }
        s = warp_sum(s);
        inv = s > 0.f ? 1.f / s : 0.f;
        const float sj = on && m > -INFINITY ? expf(lj - m) * inv : 0.f;
        G = warp_sum(g * sj);
        v = g * sj;
    } else if (a.renorm || !a.sigmoid) {   // (softmax here: no slots)
        const float ms = warp_max(lj);
        float r;
        if (!on || ms == -INFINITY) r = 0.f;
        else if (a.sigmoid) r = ms < 0.f ? expf(lj - ms) / (1.f + expf(lj)) : sigmoid_f32(lj);
        else r = expf(lj - ms);
        const float tot = warp_sum(r);
        const float p = tot > 0.f ? r / tot : 0.f;
        G = warp_sum(g * p);
        v = p * (g - G);
        if (a.sigmoid && on) v *= sigmoid_f32(-lj);
        if (!on) v = 0.f;
    } else {
        v = on ? g * sigmoid_f32(lj) * sigmoid_f32(-lj) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = 32 * i + lane;
        if (e < E) out[e] = from_f32<TL>(dense ? -G * (l[i] * inv) : 0.f);
    }
    __syncwarp();   // the entries below are written again after the row
    float sum = 0.f;   // slots that name the same expert add up, in slot order
    for (int j = 0; j < a.K; ++j) {
        const int oj = __shfl_sync(0xffffffffu, id, j);
        const float vj = __shfl_sync(0xffffffffu, v, j);
        if (oj == id) sum += vj;
    }
    if (on) {
        if (dense && m > -INFINITY) sum -= G * (expf(lj - m) * inv);
        out[id] = from_f32<TL>(sum);
    }
}

}  // namespace lf
