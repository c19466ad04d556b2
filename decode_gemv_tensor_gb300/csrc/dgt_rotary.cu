// dgt_rotary.cu -- rotary positions with several axes.
//
// A pair's angle is position times frequency.  Both the product and its
// reduction to one revolution are integer arithmetic: the frequency is a 0.64
// fixed-point fraction of a revolution, so position * frequency modulo 2^64 is
// the exact fraction of a revolution, and its high 32 bits (2^-33 revolutions)
// go to sincospif.  No double-precision unit, no loss at far positions.
#include <math.h>

#include "dgt_kv.cuh"

#include "dgt_device.cuh"

namespace dgt {

struct RotateArgs {
    dgt_rotary rot;
    dgt_heads in[2], out[2];
    uint32_t head_dim, heads;   // heads of q and k together
    uint64_t tokens;
    const int32_t *pos;
};

constexpr uint32_t RT_THREADS = 256;
constexpr uint32_t RT_PAIRS = 512;

__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    return (uint32_t)f32_to_bf16_rne(lo) | (uint32_t)f32_to_bf16_rne(hi) << 16;
}

// One CTA per token: its angles' sines and cosines once, in shared memory,
// then every head.
template <bool INTER>
__global__ void __launch_bounds__(RT_THREADS) k_rotate(RotateArgs a) {
    __shared__ float2 cs[RT_PAIRS];
    pdl_trigger();
    pdl_wait();
    const uint32_t tid = threadIdx.x;
    const uint64_t tok = blockIdx.x;
    const uint32_t half = a.rot.rot_dim / 2;
    for (uint32_t i = tid; i < half; i += RT_THREADS) {
        const uint32_t ax = a.rot.d_axis[i];
        const int64_t p = a.pos[(uint64_t)(ax < a.rot.axes ? ax : 0) * a.tokens + tok];
        const uint64_t f = (uint64_t)p * a.rot.d_freq[i];
        float s, c;
        sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();
    // pieces of 16 elements: eight pairs, then 16 unrotated elements
    const uint32_t rp = half / 8, pieces = rp + (a.head_dim - a.rot.rot_dim) / 16;
    for (uint32_t i = tid; i < a.heads * pieces; i += RT_THREADS) {
        const uint32_t h = i / pieces, q = i % pieces;
        const uint32_t side = h >= a.in[0].heads, hh = side ? h - a.in[0].heads : h;
        const dgt_heads &xi = a.in[side], &xo = a.out[side];
        const uint16_t *src = xi.data + (int64_t)tok * xi.token_stride + (int64_t)hh * xi.head_stride;
        uint16_t *dst = xo.data + (int64_t)tok * xo.token_stride + (int64_t)hh * xo.head_stride;
        const uint32_t o0 = q < rp ? (INTER ? 16 * q : 8 * q) : a.rot.rot_dim + 16 * (q - rp);
        const uint32_t o1 = q < rp && !INTER ? half + 8 * q : o0 + 8;
        uint4 u0 = *reinterpret_cast<const uint4 *>(src + o0), u1 = *reinterpret_cast<const uint4 *>(src + o1);
        if (q < rp) {
            uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
            if (INTER) {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float2 r = cs[8 * q + j];
                    const float x = bf16lo(w[j]), y = bf16hi(w[j]);
                    w[j] = round_pair(x * r.x - y * r.y, y * r.x + x * r.y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 r0 = cs[8 * q + 2 * j], r1 = cs[8 * q + 2 * j + 1];
                    const float x0 = bf16lo(w[j]), x1 = bf16hi(w[j]), y0 = bf16lo(w[4 + j]), y1 = bf16hi(w[4 + j]);
                    w[j] = round_pair(x0 * r0.x - y0 * r0.y, x1 * r1.x - y1 * r1.y);
                    w[4 + j] = round_pair(y0 * r0.x + x0 * r0.y, y1 * r1.x + x1 * r1.y);
                }
            }
            u0 = make_uint4(w[0], w[1], w[2], w[3]);
            u1 = make_uint4(w[4], w[5], w[6], w[7]);
        }
        *reinterpret_cast<uint4 *>(dst + o0) = u0;
        *reinterpret_cast<uint4 *>(dst + o1) = u1;
    }
}

}  // namespace dgt

using namespace dgt;

extern "C" int dgt_rotary_freqs(double base, uint32_t rot_dim, uint64_t *out) {
    if (!out || !(base > 1.0) || !isfinite(base)) return DGT_ERR_ARG;
    if (rot_dim == 0 || (rot_dim & 1) || rot_dim > 2 * RT_PAIRS) return DGT_ERR_SHAPE;
    for (uint32_t i = 0; i < rot_dim / 2; i++) {
        // revolutions per position, below 1/6: 2^64 times it fits and rounds in double
        const double f = pow(base, -2.0 * i / rot_dim) / 6.283185307179586476925286766559;
        out[i] = (uint64_t)nearbyint(ldexp(f, 64));
    }
    return DGT_OK;
}

extern "C" int dgt_rotate(const dgt_rotary *rot, const dgt_heads *q, const dgt_heads *k, const dgt_heads *q_out,
                          const dgt_heads *k_out, uint32_t head_dim, uint64_t tokens, const int32_t *d_pos,
                          void *stream) {
    if (!rot || !q || !q_out) return DGT_ERR_ARG;
    if (head_dim == 0 || head_dim > 1024 || (head_dim & 15)) return DGT_ERR_SHAPE;
    if (rot->rot_dim == 0 || (rot->rot_dim & 15) || rot->rot_dim > head_dim) return DGT_ERR_SHAPE;
    if (rot->axes == 0 || rot->axes > 8 || q->heads == 0 || q->heads > 1024) return DGT_ERR_SHAPE;
    if (tokens > KV_MAX_TOKENS) return DGT_ERR_SHAPE;
    if (tokens == 0) return DGT_OK;
    if (!rot->d_freq || !rot->d_axis || !d_pos) return DGT_ERR_ARG;
    RotateArgs a{};
    int rc = heads_check(q, q->heads);
    if (rc == DGT_OK) rc = heads_check(q_out, q->heads);
    if (rc != DGT_OK) return rc;
    a.in[0] = *q;
    a.out[0] = *q_out;
    if (k && k->data) {
        if (k->heads == 0 || k->heads > 1024) return DGT_ERR_SHAPE;
        rc = heads_check(k, k->heads);
        if (rc == DGT_OK) rc = heads_check(k_out, k->heads);
        if (rc != DGT_OK) return rc;
        a.in[1] = *k;
        a.out[1] = *k_out;
    }
    a.rot = *rot;
    a.head_dim = head_dim;
    a.heads = a.in[0].heads + a.in[1].heads;
    a.tokens = tokens;
    a.pos = d_pos;
    auto fn = rot->interleaved ? k_rotate<true> : k_rotate<false>;
    return launch_pdl(fn, dim3((unsigned)tokens), dim3(RT_THREADS), 0, (cudaStream_t)stream, a) == cudaSuccess
               ? DGT_OK
               : DGT_ERR_CUDA;
}
