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
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One CTA per TB tokens.  A piece is 16 elements, eight pairs or what lies past
// rot_dim; a thread keeps one piece's place, for several heads and the CTA's
// tokens.  The elements of the tokens are on their way together, the first
// ones while the angles are found.  Bound by memory: 12873 tokens of 24 heads
// of 128 29 us, 82 % of the measured copy bandwidth (30 us from buffers that
// are not in L2), of 24 heads of 256 53 us, 89 %.
template <bool INTER, uint32_t TB>
__global__ void __launch_bounds__(RT_THREADS) k_rotate(RotateArgs a) {
    __shared__ __align__(16) float2 cs[TB][RT_PAIRS];
    pdl_trigger();
    pdl_wait();
    const uint32_t tid = threadIdx.x;
    const uint64_t tok0 = (uint64_t)blockIdx.x * TB;
    const uint32_t half = a.rot.rot_dim / 2, rp = half / 8, pieces = rp + (a.head_dim - a.rot.rot_dim) / 16;
    const uint32_t q = tid % pieces, h0 = tid / pieces, hs = RT_THREADS / pieces;
    const uint32_t o0 = q < rp ? (INTER ? 16 * q : 8 * q) : a.rot.rot_dim + 16 * (q - rp);
    const uint32_t o1 = q < rp && !INTER ? half + 8 * q : o0 + 8;
    const uint32_t toks = (uint32_t)min((uint64_t)TB, a.tokens - tok0);
    const bool mine = h0 < hs;   // the last threads have no piece
    uint4 u[TB][2];
    auto load = [&](uint32_t h) {
        const uint32_t side = h >= a.in[0].heads;
        const dgt_heads &x = a.in[side];
        const uint16_t *p = x.data + (int64_t)tok0 * x.token_stride + (int64_t)(side ? h - a.in[0].heads : h) * x.head_stride;
#pragma unroll
        for (uint32_t t = 0; t < TB; t++)
            if (t < toks) {
                u[t][0] = *reinterpret_cast<const uint4 *>(p + t * x.token_stride + o0);
                u[t][1] = *reinterpret_cast<const uint4 *>(p + t * x.token_stride + o1);
            }
    };
    if (mine && h0 < a.heads) load(h0);
    for (uint32_t i = tid; i < toks * half; i += RT_THREADS) {
        const uint32_t t = i / half, j = i % half, ax = a.rot.d_axis[j];
        const int64_t p = a.pos[(uint64_t)(ax < a.rot.axes ? ax : 0) * a.tokens + tok0 + t];
        const uint64_t f = (uint64_t)p * a.rot.d_freq[j];
        float s, c;
        sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &s, &c);
        cs[t][j] = make_float2(c, s);
    }
    __syncthreads();
    if (!mine) return;
    for (uint32_t h = h0; h < a.heads; h += hs) {
        if (h != h0) load(h);
        const uint32_t side = h >= a.in[0].heads;
        const dgt_heads &x = a.out[side];
        uint16_t *p = x.data + (int64_t)tok0 * x.token_stride + (int64_t)(side ? h - a.in[0].heads : h) * x.head_stride;
#pragma unroll
        for (uint32_t t = 0; t < TB; t++) {
            if (t >= toks) break;
            uint4 &u0 = u[t][0], &u1 = u[t][1];
            if (q < rp) {
                float2 r[8];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float4 v = *reinterpret_cast<const float4 *>(&cs[t][8 * q + 2 * j]);
                    r[2 * j] = make_float2(v.x, v.y);
                    r[2 * j + 1] = make_float2(v.z, v.w);
                }
                uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                if (INTER) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float e = bf16lo(w[j]), o = bf16hi(w[j]);
                        w[j] = round_pair(e * r[j].x - o * r[j].y, o * r[j].x + e * r[j].y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 r0 = r[2 * j], r1 = r[2 * j + 1];
                        const float x0 = bf16lo(w[j]), x1 = bf16hi(w[j]), y0 = bf16lo(w[4 + j]), y1 = bf16hi(w[4 + j]);
                        w[j] = round_pair(x0 * r0.x - y0 * r0.y, x1 * r1.x - y1 * r1.y);
                        w[4 + j] = round_pair(y0 * r0.x + x0 * r0.y, y1 * r1.x + x1 * r1.y);
                    }
                }
                u0 = make_uint4(w[0], w[1], w[2], w[3]);
                u1 = make_uint4(w[4], w[5], w[6], w[7]);
            }
            *reinterpret_cast<uint4 *>(p + t * x.token_stride + o0) = u0;
            *reinterpret_cast<uint4 *>(p + t * x.token_stride + o1) = u1;
        }
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
    // Four tokens a CTA where one leaves most of its threads without a piece (a piece a thread is 16 elements) and
    // there are CTAs enough.  One and four, 4096 tokens: 576 elements a token 6.6 and 5.0 us, 1152 7.4 and 6.5, 1536
    // 7.4 and 7.0, 2048 8.5 and 9.2, 4096 14.3 and 16.8, 6144 20.6 and 22.9; 2048 tokens of 1536 4.5 and 4.3, 1024 2.8
    // and 3.6.  Between 1536 and 3072 elements one is faster by 6 to 12% at 4096 tokens, four by up to 6% at 12873.
    const bool four = tokens >= 2048 && a.heads * head_dim <= 1536;
    auto fn = rot->interleaved ? (four ? k_rotate<true, 4> : k_rotate<true, 1>)
                               : (four ? k_rotate<false, 4> : k_rotate<false, 1>);
    const unsigned grid = (unsigned)(four ? (tokens + 3) / 4 : tokens);
    return launch_pdl(fn, dim3(grid), dim3(RT_THREADS), 0, (cudaStream_t)stream, a) == cudaSuccess ? DGT_OK
                                                                                                   : DGT_ERR_CUDA;
}
