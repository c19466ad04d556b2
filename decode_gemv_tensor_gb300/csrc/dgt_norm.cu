// dgt_norm.cu -- the norm after a block, its gate, the scaled residual add and
// the norm before the next block, one row at a time in registers:
//   u = y;  u *= r(u) (offset + post);  u *= gate;
//   x' = residual x + scale u;  h = bf16(x' r(x') (offset + pre)),
//   r(v) = 1 / sqrt(mean v^2 + eps).
// Everything is fp32 in between; x' and h are each rounded once, h from x'
// before its rounding.
#include <cuda_runtime.h>

#include "../../include/dgt.h"
#include "dgt_device.cuh"
#include "dgt_launch.h"

namespace dgt {

constexpr uint32_t BN_MAX = 32768;

struct NormArgs {
    dgt_norm io;
    uint64_t rows;
    uint32_t n, rows_cta;   // rows a CTA holds at a time
    float scale, residual, offset, eps;
};

// W neighbouring elements from `at` on, as fp32.
template <int W>
__device__ __forceinline__ void load_row(const void *p, bool f32, uint64_t at, float (&v)[W]) {
    if (W == 8) {
        if (f32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            const float4 a = q[0], b = q[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
        }
    } else {
        v[0] = f32 ? static_cast<const float *>(p)[at]
                   : __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at] << 16);
    }
}
template <int W>
__device__ __forceinline__ void store_row(void *p, bool f32, uint64_t at, const float (&v)[W]) {
    if (W == 8) {
        if (f32) {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                w[i] = f32_to_bf16_rne(v[2 * i]) | (uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else if (f32) {
        static_cast<float *>(p)[at] = v[0];
    } else {
        static_cast<uint16_t *>(p)[at] = f32_to_bf16_rne(v[0]);
    }
}

// The sum over a row's threads: `group` neighbouring lanes, or the whole CTA.
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, uint32_t group, float *part) {
#pragma unroll
    for (uint32_t d = 16; d >= 1; d >>= 1)
        if (CTA || d < group) v += __shfl_xor_sync(DGT_FULL, v, d);
    if (CTA) {
        const uint32_t warps = blockDim.x >> 5;
        if (lane_id() == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane_id() < warps ? part[lane_id()] : 0.0f;
#pragma unroll
        for (uint32_t d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(DGT_FULL, v, d);
    }
    return v;
}

// J vectors of W elements a thread; a row is `group` threads' (CTA: all of
// them).
template <int W, int J, bool CTA>
__global__ void __launch_bounds__(1024) k_block_norm(NormArgs a, uint32_t group) {
    __shared__ float part[2][32];
    pdl_trigger();
    pdl_wait();
    const dgt_norm &io = a.io;
    const uint32_t t = CTA ? threadIdx.x : threadIdx.x % group;
    const uint64_t row = CTA ? blockIdx.x : (uint64_t)blockIdx.x * a.rows_cta + threadIdx.x / group;
    const bool live = row < a.rows;
    const uint64_t r = live ? row : a.rows - 1;   // rows behind the last are computed and not stored
    const bool xf = io.x_f32, yf = io.y_f32;
    auto col = [&](int j) { return (t + j * group) * W; };
    auto in = [&](int j) { return col(j) < a.n; };
    float x[J][W], u[J][W];
    const float inv_n = 1.0f / (float)a.n;
#pragma unroll
    for (int j = 0; j < J; j++) {
#pragma unroll
        for (int i = 0; i < W; i++) u[j][i] = 0.0f;
        if (io.y && in(j)) load_row<W>(io.y, yf, r * io.y_stride + col(j), u[j]);
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
#pragma unroll
        for (int i = 0; i < W; i++) x[j][i] = 0.0f;
        if (in(j)) load_row<W>(io.x, xf, r * io.x_stride + col(j), x[j]);
    }
    if (io.post) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++)
#pragma unroll
            for (int i = 0; i < W; i++) ss = fmaf(u[j][i], u[j][i], ss);
        const float f = 1.0f / sqrtf(row_sum<CTA>(ss, group, part[0]) * inv_n + a.eps);
#pragma unroll
        for (int j = 0; j < J; j++) {
            if (!in(j)) continue;
            float w[W];
            load_row<W>(io.post, false, col(j), w);
#pragma unroll
            for (int i = 0; i < W; i++) u[j][i] = u[j][i] * f * (a.offset + w[i]);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < J; j++) {
        if (!in(j)) continue;
        if (io.gate) {
            float g[W];
            load_row<W>(io.gate, false, r * io.gate_stride + col(j), g);
#pragma unroll
            for (int i = 0; i < W; i++) u[j][i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < W; i++) {
            x[j][i] *= a.residual;
            if (io.y) x[j][i] = fmaf(a.scale, u[j][i], x[j][i]);
            ss = fmaf(x[j][i], x[j][i], ss);
        }
        if (io.x_out && live) store_row<W>(io.x_out, xf, r * io.xo_stride + col(j), x[j]);
    }
    if (io.h) {
        const float f = 1.0f / sqrtf(row_sum<CTA>(ss, group, part[1]) * inv_n + a.eps);
#pragma unroll
        for (int j = 0; j < J; j++) {
            if (!in(j)) continue;
            float w[W];
            load_row<W>(io.pre, false, col(j), w);
#pragma unroll
            for (int i = 0; i < W; i++) w[i] = x[j][i] * f * (a.offset + w[i]);
            if (live) store_row<W>(io.h, false, r * io.h_stride + col(j), w);
        }
    }
}

template <int W, int J>
static cudaError_t norm_launch(NormArgs &a, cudaStream_t st) {
    const uint32_t need = (a.n + W * J - 1) / (W * J);   // threads of a row
    if (need <= 32) {
        uint32_t group = 1;
        while (group < need) group *= 2;
        a.rows_cta = 256 / group;
        const uint64_t grid = (a.rows + a.rows_cta - 1) / a.rows_cta;
        return launch_pdl(k_block_norm<W, J, false>, dim3((unsigned)grid), dim3(256), 0, st, a, group);
    }
    const uint32_t threads = (need + 31) / 32 * 32;
    return launch_pdl(k_block_norm<W, J, true>, dim3((unsigned)a.rows), dim3(threads), 0, st, a, threads);
}

}  // namespace dgt

using namespace dgt;

extern "C" int dgt_block_norm(const dgt_norm *io, uint64_t rows, uint32_t n, float scale, float residual,
                              float offset, float eps, void *stream) {
    if (!io) return DGT_ERR_ARG;
    if (n == 0 || n > BN_MAX || rows > (1u << 24)) return DGT_ERR_SHAPE;
    if (rows == 0) return DGT_OK;
    if (!io->x || (!io->x_out && !io->h)) return DGT_ERR_ARG;
    if ((io->pre == nullptr) != (io->h == nullptr) || ((io->post || io->gate) && !io->y)) return DGT_ERR_ARG;
    if (!(eps >= 0.0f) || io->x_f32 > 1 || io->y_f32 > 1) return DGT_ERR_ARG;
    const uint32_t xs = io->x_f32 ? 4 : 2, ys = io->y_f32 ? 4 : 2;
    if (((uintptr_t)io->x | (uintptr_t)io->x_out) & (xs - 1) || ((uintptr_t)io->y & (ys - 1)) ||
        (((uintptr_t)io->h | (uintptr_t)io->pre | (uintptr_t)io->post | (uintptr_t)io->gate) & 1))
        return DGT_ERR_ARG;
    NormArgs a{*io, rows, n, 0, scale, residual, offset, eps};
    const uintptr_t all = (uintptr_t)io->x | (uintptr_t)io->x_out | (uintptr_t)io->y | (uintptr_t)io->h |
                          (uintptr_t)io->pre | (uintptr_t)io->post | (uintptr_t)io->gate;
    int64_t strides = rows > 1 ? io->x_stride : 0;
    if (rows > 1) {
        if (io->x_out) strides |= io->xo_stride;
        if (io->y) strides |= io->y_stride;
        if (io->h) strides |= io->h_stride;
        if (io->gate) strides |= io->gate_stride;
    }
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    // 16-byte pieces where everything allows them
    if (n % 8 == 0 && (all & 15) == 0 && (strides & 7) == 0)
        e = n <= 8192 ? norm_launch<8, 1>(a, st) : n <= 16384 ? norm_launch<8, 2>(a, st) : norm_launch<8, 4>(a, st);
    else
        e = n <= 4096 ? norm_launch<1, 4>(a, st) : n <= 16384 ? norm_launch<1, 16>(a, st) : norm_launch<1, 32>(a, st);
    return e == cudaSuccess ? DGT_OK : DGT_ERR_CUDA;
}
