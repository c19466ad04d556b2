// dgt_route.cu -- the router's choice of experts, a warp for each token.
//
//   s = softmax(l) or 1 / (1 + e^-l);  c = s + bias, or the order of l itself
//   where there is no bias;  a group's value is the sum of its one or two best
//   c;  the best groups stay, and of their experts the best topk are taken.
//
// Which expert is taken is decided as if in 64 bits: the order is found in
// fp32 with a bound on its error, and a token whose neighbouring values, among
// the chosen, the first one left out and the groups at their border, are not
// further apart than that is decided again in fp64.  Logits alone are compared
// as they are.
#include <cuda_runtime.h>

#include "../../include/dgt.h"
#include "dgt_device.cuh"
#include "dgt_launch.h"

namespace dgt {

constexpr uint32_t RT_WARPS = 4;
constexpr uint32_t RT_MAX_EXPERTS = 1024;

struct RouteArgs {
    const void *logits;
    int64_t stride;
    const float *bias;
    int32_t *ids;
    float *p;
    uint64_t tokens;
    uint32_t experts, topk, groups, group_topk, group_best, f32, sigmoid, renorm;
    float scale;
};

// Whole numbers in the order of the values; a NaN comes behind every number
// (1), what is taken or closed behind that (0).
__device__ __forceinline__ uint32_t order32(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t order64(double v) {
    if (v != v) return 1ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t warp_top(uint32_t k) { return __reduce_max_sync(DGT_FULL, k); }
__device__ __forceinline__ uint64_t warp_top(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(DGT_FULL, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(DGT_FULL, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The best `want` experts in order, lane j's the j-th, from every lane's EPL
// keys of the experts EPL * lane ...; taken keys become 0.  next: the best key
// left.
template <int EPL, typename K>
__device__ __forceinline__ uint32_t take(K (&key)[EPL], uint32_t want, K &mine, K &next) {
    const uint32_t lane = lane_id();
    uint32_t id = 0;
    mine = 0;
    for (uint32_t j = 0;; j++) {
        K best = key[0];
        uint32_t at = 0;
#pragma unroll
        for (int i = 1; i < EPL; i++)
            if (key[i] > best) best = key[i], at = i;
        const K top = warp_top(best);
        if (j == want) {
            next = top;
            return id;
        }
        const uint32_t owner = __ffs(__ballot_sync(DGT_FULL, best == top)) - 1;
        const uint32_t e = __shfl_sync(DGT_FULL, at, owner);
        if (lane == owner) {
#pragma unroll
            for (int i = 0; i < EPL; i++)
                if (i == (int)at) key[i] = 0;
        }
        if (lane == j) id = owner * EPL + e, mine = top;
    }
}

template <int EPL>
__device__ __forceinline__ float logit(const RouteArgs &a, const void *row, uint32_t e) {
    return a.f32 ? static_cast<const float *>(row)[e]
                 : __uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[e] << 16);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(DGT_FULL, v, d));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(DGT_FULL, v, d);
    return v;
}

// e^(l - m) of a softmax: 1 where l is the largest, also when that is
// infinite; 0 for -inf and NaN.
template <typename T>
__device__ __forceinline__ T soft_term(T l, T m) {
    return l == m ? (l == (T)-INFINITY ? (T)0 : (T)1) : l == l ? exp(l - m) : (T)0;
}
template <>
__device__ __forceinline__ float soft_term<float>(float l, float m) {
    return l == m ? (l == -INFINITY ? 0.0f : 1.0f) : l == l ? expf(l - m) : 0.0f;
}
__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ double sigmoid_of(double l) { return 1.0 / (1.0 + exp(-l)); }

// Two values in order that may be the other way round; infinite ones are what they are in any precision.
__device__ __forceinline__ bool near(float hi, float lo, float tol) {
    return fabsf(hi) < INFINITY && fabsf(lo) < INFINITY && hi - lo <= tol;
}

// Groups: lane g gets the value of group g, the sum of its `best` largest of
// v[0 .. per), v in shared memory.
template <typename T>
__device__ __forceinline__ T group_value(const T *v, uint32_t per, uint32_t groups, uint32_t best) {
    const uint32_t lane = lane_id();
    if (lane >= groups) return (T)-INFINITY;
    T one = (T)-INFINITY, two = (T)-INFINITY;
    for (uint32_t i = 0; i < per; i++) {
        const T x = v[lane * per + i];
        if (x > one) two = one, one = x;
        else if (x > two) two = x;
    }
    return best == 2 && per > 1 ? one + two : one;
}
// Which groups stay: bit g.
template <typename K>
__device__ __forceinline__ uint32_t keep_groups(K key, uint32_t groups, uint32_t keep) {
    const uint32_t lane = lane_id();
    uint32_t before = 0;
    for (uint32_t g = 0; g < groups; g++) {
        const K other = __shfl_sync(DGT_FULL, key, g);
        before += other > key || (other == key && g < lane);
    }
    return __ballot_sync(DGT_FULL, lane < groups && before < keep);
}

// A token in fp64 (rare): the same steps.
template <int EPL>
__device__ __noinline__ uint32_t decide64(const RouteArgs &a, const void *row, double *vals) {
    const uint32_t lane = lane_id(), per = a.experts / a.groups;
    double l[EPL], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint32_t e = lane * EPL + i;
        l[i] = e < a.experts ? (double)logit<EPL>(a, row, e) : -INFINITY;
        if (l[i] > m) m = l[i];
    }
    m = (double)warp_max((float)m);
    double z = 0.0;
    uint64_t key[EPL];
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            l[i] = soft_term<double>(l[i], m);
            z += l[i];
        }
        z = warp_sum(z);
        if (z == 0.0) z = 1.0;
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint32_t e = lane * EPL + i;
        key[i] = 0;
        if (e >= a.experts) continue;
        const double x = (double)logit<EPL>(a, row, e);
        const double s = x != x ? x : a.sigmoid ? sigmoid_of(x) : l[i] / z;
        const double c = a.bias ? s + (double)a.bias[e] : s;
        key[i] = order64(a.bias ? c : x);
        if (a.groups > 1) vals[e] = c == c ? c : -INFINITY;
    }
    if (a.groups > 1) {
        __syncwarp();
        const double v = group_value(vals, per, a.groups, a.group_best);
        const uint32_t open = keep_groups(lane < a.groups ? order64(v) : 0ull, a.groups, a.group_topk);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!(open >> ((lane * EPL + i) / per) & 1u)) key[i] = 0;
    }
    uint64_t mine, next;
    return take<EPL>(key, a.topk, mine, next);
}

template <int EPL>
__global__ void __launch_bounds__(RT_WARPS * 32) k_route(RouteArgs a) {
    extern __shared__ __align__(8) uint8_t smem[];
    pdl_trigger();
    pdl_wait();
    const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
    const uint64_t token = (uint64_t)blockIdx.x * RT_WARPS + warp;
    if (token >= a.tokens) return;
    const void *row = a.f32 ? (const void *)(static_cast<const float *>(a.logits) + token * a.stride)
                            : (const void *)(static_cast<const uint16_t *>(a.logits) + token * a.stride);
    double *vals = reinterpret_cast<double *>(smem) + warp * a.experts;   // of the groups' experts
    float l[EPL], c[EPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint32_t e = lane * EPL + i;
        l[i] = e < a.experts ? logit<EPL>(a, row, e) : -INFINITY;
        m = fmaxf(m, l[i]);
    }
    m = warp_max(m);
    float inv = 1.0f;
    if (!a.sigmoid) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            c[i] = soft_term<float>(l[i], m);
            z += c[i];
        }
        z = warp_sum(z);
        inv = z == 0.0f ? 0.0f : 1.0f / z;
    }
    uint32_t key[EPL];
    const bool scored = a.bias || a.groups > 1;   // where scores, not logits, are compared
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint32_t e = lane * EPL + i;
        if (scored) {
            c[i] = a.sigmoid ? sigmoid_of(l[i]) : l[i] != l[i] ? l[i] : c[i] * inv;
            if (a.bias && e < a.experts) c[i] += a.bias[e];
        }
        key[i] = e < a.experts ? order32(a.bias ? c[i] : l[i]) : 0u;
    }
    // How far an fp32 score may be off.  A sigmoid, which is at most 1: expf within 2 units in the last place, a sum
    // and a quotient, below 2^-21.  A softmax, which is at most inv: expf, a sum of EPL + 5 steps, a quotient and a
    // product, below (EPL + 8) 2^-23.  Then half a unit of the sum with the bias.
    const float off = a.sigmoid ? 0x1p-21f : (float)(EPL + 8) * 0x1p-23f * inv;
    bool close = false;
    if (a.groups > 1) {
        const uint32_t per = a.experts / a.groups;
        float *v = reinterpret_cast<float *>(vals);
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const uint32_t e = lane * EPL + i;
            if (e < a.experts) v[e] = c[i] == c[i] ? c[i] : -INFINITY;
        }
        __syncwarp();
        const float gv = group_value(v, per, a.groups, a.group_best);
        const uint32_t gk = lane < a.groups ? order32(gv) : 0u;
        const uint32_t open = keep_groups(gk, a.groups, a.group_topk);
        if (a.group_topk < a.groups) {
            const bool in = open >> lane & 1u;
            const float lo = value32(__reduce_min_sync(DGT_FULL, in ? gk : ~0u));
            const float hi = value32(__reduce_max_sync(DGT_FULL, in ? 0u : gk));
            float big = 0.0f;   // the sums of two may be smaller than what they add
#pragma unroll
            for (int i = 0; i < EPL; i++) big = fmaxf(big, fabsf(c[i]) < INFINITY ? fabsf(c[i]) : 0.0f);
            close = near(lo, hi, 4.0f * off + 0x1p-21f * warp_max(big));
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!(open >> ((lane * EPL + i) / per) & 1u)) key[i] = 0;
        __syncwarp();
    }
    uint32_t mine, next;
    uint32_t id = take<EPL>(key, a.topk, mine, next);
    if (a.bias) {
        const uint32_t after = __shfl_down_sync(DGT_FULL, mine, 1), below = lane + 1 < a.topk ? after : next;
        const float hi = value32(mine), lo = value32(below);
        close |= __any_sync(DGT_FULL, lane < a.topk && below > 1u &&
                                          near(hi, lo, 2.0f * off + 0x1p-23f * (fabsf(lo) + fabsf(hi))));
    }
    if (close) id = decide64<EPL>(a, row, vals);

    // weights
    const bool on = lane < a.topk;
    const float x = on ? logit<EPL>(a, row, id) : -INFINITY;
    float w;
    if (a.renorm) {
        // s / sum s as the quotient of what is left of both by the largest taken logit: nothing is lost to
        // scores below fp32's range
        const float top = warp_max(x);
        float q = soft_term<float>(x, top);
        // e^(l - top) (1 + e^top) / (1 + e^l) for a top below 0, else s itself
        if (a.sigmoid) q = top > 0.0f ? (x == x ? sigmoid_of(x) : 0.0f) : q * (1.0f + expf(top)) / (1.0f + expf(x));
        const float sum = warp_sum(on ? q : 0.0f);
        w = sum > 0.0f ? q / sum : 0.0f;
    } else {
        w = a.sigmoid ? (x == x ? sigmoid_of(x) : 0.0f) : soft_term<float>(x, m) * inv;
    }
    if (on) {
        a.ids[token * a.topk + lane] = (int32_t)id;
        a.p[token * a.topk + lane] = w * a.scale;
    }
}

template <int EPL>
static cudaError_t route_launch(const RouteArgs &a, cudaStream_t st) {
    const uint64_t grid = (a.tokens + RT_WARPS - 1) / RT_WARPS;
    const size_t smem = a.groups > 1 ? (size_t)RT_WARPS * a.experts * 8 : 0;   // 32 KB at most
    return launch_pdl(k_route<EPL>, dim3((unsigned)grid), dim3(RT_WARPS * 32), smem, st, a);
}

}  // namespace dgt

using namespace dgt;

extern "C" int dgt_route(const dgt_router *r, const void *d_logits, int64_t stride, uint64_t tokens, int32_t *d_ids,
                         float *d_p, void *stream) {
    if (!r || r->f32 > 1 || r->sigmoid > 1 || r->renorm > 1) return DGT_ERR_ARG;
    if (r->experts == 0 || r->experts > RT_MAX_EXPERTS || r->topk == 0 || r->topk > 32) return DGT_ERR_SHAPE;
    if (r->groups == 0 || r->groups > 32 || r->experts % r->groups || r->group_topk == 0 ||
        r->group_topk > r->groups || r->topk > r->group_topk * (r->experts / r->groups) || tokens > (1u << 24))
        return DGT_ERR_SHAPE;
    if (r->group_best != 1 && r->group_best != 2) return DGT_ERR_ARG;
    if (tokens == 0) return DGT_OK;
    if (!d_logits || !d_ids || !d_p || ((uintptr_t)d_logits & (r->f32 ? 3 : 1)) ||
        (((uintptr_t)d_ids | (uintptr_t)d_p | (uintptr_t)r->d_bias) & 3))
        return DGT_ERR_ARG;
    const RouteArgs a{d_logits, stride, r->d_bias, d_ids, d_p, tokens, r->experts, r->topk, r->groups,
                      r->group_topk, r->group_best, r->f32, r->sigmoid, r->renorm, r->scale};
    cudaStream_t st = (cudaStream_t)stream;
    const uint32_t epl = (r->experts + 31) / 32;
    const cudaError_t e = epl <= 1   ? route_launch<1>(a, st)
                          : epl <= 2 ? route_launch<2>(a, st)
                          : epl <= 4 ? route_launch<4>(a, st)
                          : epl <= 8 ? route_launch<8>(a, st)
                          : epl <= 16 ? route_launch<16>(a, st)
                                      : route_launch<32>(a, st);
    return e == cudaSuccess ? DGT_OK : DGT_ERR_CUDA;
}
